"""Oracle of the tree step over a 4-bit cache (numpy, float64, written from the definitions).

TEST INFRASTRUCTURE: used by the test suite only; shares no code with the CUDA path.

  head norm and rotation: y = x / sqrt(mean(x^2) + eps) * w, then each pair (a, c) of the
      rotated elements becomes (a cos t - c sin t, c cos t + a sin t), t = position * inv_freq;
  4-bit cache: 16 elements share an e4m3 scale, elements are e2m1; the stored scale is
      e4m3(max|x| * RN(r * RN(1/6))) and a code e2m1(x * RN(RN(1/s) * r)), r = RN(1 / tensor
      scale), RN = rounding to float32, products rounded to float32;
  tree attention: softmax over the positions 0..ctx-1 and the nodes in the mask.
"""
from __future__ import annotations

import numpy as np

from . import kv_commit as KV

NHD, HND = 0, 1
BAD_SLOT = 5
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def norm_rope(x, w, eps, inv_freq, pos, pairs):
    """x [B, N, H, D] float64, w [D] or None, inv_freq float32 [rot/2], pos int [B, N]."""
    y = np.array(x, dtype=np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    half = len(inv_freq)
    if half:
        t = np.asarray(pos, np.float64)[..., None] * np.asarray(inv_freq, np.float64)
        cos, sin = np.cos(t)[:, :, None], np.sin(t)[:, :, None]
        a = np.arange(half) * (2 if pairs else 1)
        c = a + (1 if pairs else half)
        ya, yc = y[..., a].copy(), y[..., c].copy()
        y[..., a], y[..., c] = ya * cos - yc * sin, yc * cos + ya * sin
    return y


def _nearest(a, grid):
    """Index of the grid value nearest to each a >= 0; ties to the even index."""
    a = np.minimum(a, grid[-1])
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


E4M3 = KV._fp8_table(KV.FP8_E4M3)


def quantise(x, tensor_scale=1.0):
    """float32 values [..., D] -> (codes uint8 [..., D] (0..15), scales uint8 [..., D/16])."""
    f32 = np.float32
    x = np.asarray(x, f32)
    blocks = x.reshape(x.shape[:-1] + (-1, 16))
    r = f32(1) / f32(tensor_scale)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        amax = np.abs(blocks).max(-1)
        want = (amax * f32(r * f32(1.0 / 6.0))).astype(f32).astype(np.float64)
        sf = np.where(np.isnan(want), 0x7F, _nearest(np.nan_to_num(want, nan=0.0), E4M3[:0x7F]))
        s = E4M3[sf].astype(f32)
        m = np.where(s > 0, ((f32(1) / s).astype(f32) * r).astype(f32), f32(0))
        y = np.where(m[..., None] > 0, (blocks * m[..., None]).astype(f32), f32(0))
    code = _nearest(np.abs(y).astype(np.float64), E2M1) + 8 * (y < 0)
    return code.reshape(x.shape).astype(np.uint8), sf.astype(np.uint8)


def values(codes, sf, tensor_scale=1.0):
    """The float64 values of codes [..., D] under scales [..., D/16]."""
    v = np.where(codes >= 8, -E2M1[codes & 7], E2M1[codes & 7])
    v = v.reshape(codes.shape[:-1] + (-1, 16)) * E4M3[sf][..., None]
    return v.reshape(codes.shape) * np.float64(np.float32(tensor_scale))


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(b):
    out = np.empty(b.shape[:-1] + (2 * b.shape[-1],), np.uint8)
    out[..., 0::2], out[..., 1::2] = b & 15, b >> 4
    return out


def place(table, num_blocks, block_size, b, p):
    """(block, offset) of position p of request b, or None outside the table or the cache."""
    if p < 0 or p // block_size >= table.shape[1]:
        return None
    blk = int(table[b, p // block_size])
    return (blk, p % block_size) if 0 <= blk < num_blocks else None


def commit(src, cache, sf, layout, block_size, table, seq_pos, tensor_scale=1.0, kv=None,
           last=None):
    """Rows src [B, N, H, D] (float32 values) into copies of cache (codes, one per byte,
    [..., D]) and sf. Returns (cache, sf, status)."""
    cache, sf = cache.copy(), sf.copy()
    B, N = src.shape[:2]
    status = np.zeros(B, np.int32)
    for b in range(B):
        if kv is not None and kv[b, 0] < 0:
            continue
        n = N - 1 if last is None else min(int(last[b]), N - 1)
        for j in range(n + 1):
            node = j if kv is None else int(kv[b, j])
            at = place(table, cache.shape[0], block_size, b, int(seq_pos[b]) + j)
            if at is None or not 0 <= node < N:
                status[b] = BAD_SLOT
                continue
            c, s = quantise(src[b, node], tensor_scale)
            if layout == NHD:
                cache[at], sf[at] = c, s
            else:
                cache[at[0], :, at[1]], sf[at[0], :, at[1]] = c, s
    return cache, sf, status


def read(cache, sf, layout, block_size, table, b, p, tensor_scale=1.0):
    """Values [H, D] of position p of request b, or None."""
    at = place(table, cache.shape[0], block_size, b, p)
    if at is None:
        return None
    if layout == NHD:
        return values(cache[at], sf[at], tensor_scale)
    return values(cache[at[0], :, at[1]], sf[at[0], :, at[1]], tensor_scale)


def attend(q, tk, tv, keys, vals, mask, scale):
    """One request: q [N, Hq, D]; tree rows tk, tv [N, H, D]; context keys, vals [L, H, D];
    mask uint64 [N]. Returns (out [N, Hq, D], lse [N, Hq], weight of |v| [N, Hq, D], largest
    sum of |q k| scale [N, Hq]): the last two for error bounds."""
    N, Hq, D = q.shape
    H = tk.shape[1]
    G = Hq // H
    out, lse = np.zeros((N, Hq, D)), np.full((N, Hq), -np.inf)
    size, big = np.zeros((N, Hq, D)), np.zeros((N, Hq))
    for n in range(N):
        sel = [j for j in range(N) if (int(mask[n]) >> j) & 1]
        for h in range(Hq):
            k = np.concatenate((keys[:, h // G], tk[sel, h // G]))
            v = np.concatenate((vals[:, h // G], tv[sel, h // G]))
            if not len(k):
                continue
            with np.errstate(invalid="ignore", over="ignore"):
                z = k @ q[n, h] * scale
                m = z.max()
                p = np.exp(z - m)
                out[n, h] = (p[:, None] * v).sum(0) / p.sum()
                lse[n, h] = m + np.log(p.sum())
                size[n, h] = (p[:, None] * np.abs(v)).sum(0) / p.sum()
                big[n, h] = (np.abs(k) @ np.abs(q[n, h])).max() * scale
    return out, lse, size, big
