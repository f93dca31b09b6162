"""Oracle of the paged step and of token log probabilities (numpy, float64, from the definitions).

TEST INFRASTRUCTURE: used by the test suite only; shares no code with the CUDA path.

  append: head norm and rotation as in tree_step; a row's key and value stand at its position;
  attention: row at position p sees 0 <= j <= p with j > p - window (window > 0) or j < sinks;
  log probabilities: softmax(z / T) of a row, its entropy, its likeliest tokens.
"""
from __future__ import annotations

import numpy as np

from . import kv_commit as KV
from . import tree_step as S

NHD, HND = 0, 1
BAD_SLOT, BAD_RANGE = 5, 8
ROW_NAN, ROW_POSINF, ROW_ALL_NEGINF, ROW_BAD_NODE, ROW_BAD_TOKEN = 1, 2, 4, 8, 16


def norm_rope(x, w, eps, inv_freq, pos, pairs):
    """x [T, H, D] float64 at positions pos [T]."""
    return S.norm_rope(x[None], w, eps, inv_freq, np.asarray(pos)[None], pairs)[0]


def fp8_values(codes, e4m3):
    """What the codes of an 8-bit cache stand for, over the tensor scale."""
    table = KV._fp8_table(KV.FP8_E4M3 if e4m3 else KV.FP8_E5M2)
    return table[np.asarray(codes, np.uint8)]


def visible(p, n, window, sinks):
    """Which of positions 0 .. n - 1 a row at position p sees."""
    j = np.arange(n)
    ok = j <= p
    if window > 0:
        ok &= (j > p - window) | (j < sinks)
    return ok


def attention(q, k, v, pos, there, scale, window, sinks):
    """q [n, Hq, D], k, v [L, H, D] float64; rows at positions pos[i]; there [L]: positions whose
    block exists. -> dict(out, lse, A, X): results, the weighted mean of |v|, and the largest
    sum of |q k| scale log2(e) among the keys seen."""
    n, Hq, D = q.shape
    L, H, _ = k.shape
    G = Hq // H
    out, A = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, X = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for i in range(n):
        see = visible(pos[i], L, window, sinks) & there
        if not see.any():
            continue
        for h in range(Hq):
            kk, vv = k[see, h // G], v[see, h // G]
            with np.errstate(invalid="ignore", over="ignore"):
                z = kk @ q[i, h] * scale
                m = z.max()
                e = np.exp(z - m)
                out[i, h] = (e[:, None] * vv).sum(0) / e.sum()
                A[i, h] = (e[:, None] * np.abs(vv)).sum(0) / e.sum()
                lse[i, h] = m + np.log(e.sum())
                X[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * scale * np.log2(np.e)
    return dict(out=out, lse=lse, A=A, X=X)


def logprobs(row, temperature, tokens, top):
    """One row of logits (float64). -> dict(flags, logprob [C], entropy, ids, top)."""
    C, V = len(tokens), len(row)
    nan = np.isnan(row).any()
    flags = (ROW_NAN if nan else 0) | (ROW_POSINF if (row == np.inf).any() else 0)
    if not nan and (row == -np.inf).all():
        flags |= ROW_ALL_NEGINF
    tokens = np.asarray(tokens, np.int64)
    out = dict(logprob=np.full(C, np.nan), entropy=np.nan, ids=np.full(top, -1),
               top=np.full(top, np.nan))
    odd = (tokens < -1) | (tokens >= V)
    if flags == 0:
        z = row / temperature
        z = z - z.max()
        e = np.exp(z)
        lp = z - np.log(e.sum())
        p = e / e.sum()
        out["entropy"] = -(p[p > 0] * lp[p > 0]).sum()
        out["logprob"] = np.where(odd, np.nan, lp[np.clip(tokens, 0, V - 1)])
        order = np.argsort(-row, kind="stable")[:top]
        order = order[row[order] > -np.inf]
        out["ids"][:len(order)] = order
        out["top"][:] = -np.inf
        out["top"][:len(order)] = lp[order]
    out["logprob"][tokens == -1] = 0.0
    out["flags"] = flags | (ROW_BAD_TOKEN if odd.any() else 0)
    return out
