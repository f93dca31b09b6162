"""Log probabilities of tokens against the float64 oracle (needs a GB300).

Tolerances. With t = (z - m) / T, in natural units: t is a float32 difference and product (2^-23 |t|),
2^t's exponential is within 2^-21 of itself beyond what t's rounding gives it, a sum of V / 256 terms
in chains adds V 2^-33 of itself. The sum S of the exponentials so errs by 2^-21 + 2^-23 E + V 2^-33 of
itself, E = sum p |t|, a log p by that, 2^-23 |t| and 2^-23 |log S|; the entropy's sum E by (2^-21 +
2^-22 max(1, |t| where p counts, below 2^5) + V 2^-33) E.
"""
import numpy as np
import pytest
import torch

from oracle import paged_step as S
from speculative_decoding_tree_mask_gb300 import binding as G

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def h():
    G.load()
    with G.Handle(64, 64, 1 << 21, 0) as handle:
        yield handle


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def check(got, logits, node, tokens, temperature, top):
    """Every slot of a call against the oracle. logits [B, N, V] float64."""
    got = {k: v.cpu().numpy() for k, v in got.items()}
    B, N, V = logits.shape
    P = node.shape[1]
    tokens = None if tokens is None else tokens.reshape(B, P, -1)
    for b in range(B):
        for j in range(P):
            n, at = int(node[b, j]), (b, j)
            tok = np.zeros(0, np.int64) if tokens is None else tokens[b, j]
            lp = got["logprob"].reshape(B, P, -1)[at] if tokens is not None else np.zeros(0)
            ids, tlp = got["top_ids"][at], got["top_logprobs"][at]
            if n == -1:
                assert got["flags"][at] == 0 and got["entropy"][at] == 0 and (lp == 0).all()
                assert (ids == -1).all() and (tlp == -np.inf).all()
                continue
            if not 0 <= n < N:
                assert got["flags"][at] == S.ROW_BAD_NODE and np.isnan(got["entropy"][at])
                assert np.isnan(lp).all() and (ids == -1).all() and np.isnan(tlp).all()
                continue
            r = S.logprobs(logits[b, n], temperature, tok, top)
            assert got["flags"][at] == r["flags"], (at, got["flags"][at], r["flags"])
            assert np.array_equal(ids, r["ids"]), (at, ids, r["ids"])
            for x, y in ((lp, r["logprob"]), (tlp, r["top"]), (got["entropy"][at], r["entropy"])):
                assert np.array_equal(np.isnan(x), np.isnan(y))
            if r["flags"] & ~S.ROW_BAD_TOKEN:
                continue
            z = (logits[b, n] - logits[b, n].max()) / temperature
            p = np.exp(z)
            log_s = np.log(p.sum())
            E = (p[p > 0] * -z[p > 0]).sum() / p.sum()
            rel = 2.0 ** -21 + 2.0 ** -23 * E + V * 2.0 ** -33
            for x, y in ((lp, r["logprob"]), (tlp, r["top"])):
                ok = np.isfinite(y)
                assert np.array_equal(x[~ok & ~np.isnan(y)], y[~ok & ~np.isnan(y)])
                # |t| = |y + log S|
                tol = rel + 2.0 ** -23 * (np.abs(y[ok] + log_s) + log_s + np.abs(y[ok]))
                assert np.all(np.abs(x[ok] - y[ok]) <= tol)
            tol = rel + 2.0 ** -23 * log_s + (2.0 ** -17 + V * 2.0 ** -33) * E
            assert abs(got["entropy"][at] - r["entropy"]) <= tol


def rows(rng, B, N, V, dt, std=2.5):
    t = torch.from_numpy((rng.standard_normal((B, N, V)) * std).astype(np.float32)).to(TDT[dt])
    return t.to(DEV), t.double().numpy()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,V,C,top,temperature", [
    (1, 1, 1, 1, 1, 1.0), (2, 3, 2, 2, 2, 0.5), (1, 2, 7, 1, 32, 1.0), (3, 2, 8, 3, 5, 2.0),
    (2, 2, 31, 64, 31, 1.0), (1, 5, 257, 1, 0, 0.1), (4, 3, 1000, 2, 20, 1.0),
    (2, 9, 4099, 1, 32, 0.7), (1, 1, 50257, 4, 8, 1.0), (1, 1, 152064, 1, 20, 1.3),
    (40, 30, 300, 1, 3, 1.0), (1, 2, 2097152, 1, 5, 1.0)])
def test_every_row(h, dt, B, N, V, C, top, temperature):
    rng = np.random.default_rng(V + C)
    t, x = rows(rng, B, N, V, dt)
    tokens = rng.integers(0, V, (B, N, C)).astype(np.int32)
    got = G.token_logprobs(h, t, gpu(tokens), temperature=temperature, top=top)
    check(got, x, np.tile(np.arange(N), (B, 1)), tokens, temperature, top)
    if C == 1:
        two = G.token_logprobs(h, t, gpu(tokens[..., 0]), temperature=temperature, top=top)
        assert torch.equal(two["logprob"], got["logprob"][..., 0])
    none = G.token_logprobs(h, t, temperature=temperature, top=top)
    assert "logprob" not in none and torch.equal(none["top_ids"], got["top_ids"])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", [100, 4103, 60000])
def test_rows_that_are_hard_to_order(h, dt, V):
    """Ties everywhere, masks by -inf and by the type's lowest value, zeros of both signs, one token
    far above, all large values in one thread's share, rising and falling rows."""
    rng = np.random.default_rng(V)
    low = torch.finfo(TDT[dt]).min
    x = np.zeros((1, 12, V))
    x[0, 1] = 3.0
    x[0, 2, ::2] = -0.0
    x[0, 3] = -np.inf
    x[0, 3, [V - 1, 5, 17]] = [1.0, 2.0, 1.0]
    x[0, 4] = low
    x[0, 4, [40, 3, V // 2]] = [0.5, -1.0, 0.5]
    x[0, 5] = rng.integers(-3, 3, V)
    x[0, 6] = rng.standard_normal(V)
    x[0, 6, V // 3] = 200.0
    x[0, 7] = -rng.random(V)
    x[0, 7, ::2048 if V > 4096 else 16] = rng.random(len(x[0, 7, ::2048 if V > 4096 else 16]))
    x[0, 8] = np.arange(V) / V * 20
    x[0, 9] = -np.arange(V) / V * 20
    x[0, 10] = np.where(np.arange(V) % 256 < 8, 1.0 + rng.random(V), 0.0)
    x[0, 11] = rng.standard_normal(V) * 1e4
    t = torch.from_numpy(x.astype(np.float32)).to(TDT[dt])
    x = t.double().numpy()
    tokens = np.tile(np.array([5, V - 1, 0], np.int32), (1, 12, 1))
    for top in (1, 20, 32):
        got = G.token_logprobs(h, t.to(DEV), gpu(tokens), top=top)
        check(got, x, np.arange(12)[None], tokens, 1.0, top)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", [9, 3001])
def test_rows_and_tokens_that_cannot_be_scored(h, dt, V):
    rng = np.random.default_rng(V)
    t, x = rows(rng, 2, 5, V, dt)
    for at, value in (((0, 0, 3), np.nan), ((0, 1, V - 1), np.inf), ((0, 2), -np.inf),
                      ((1, 4, 0), -np.inf)):
        t[at], x[at] = value, value
    node = np.array([[0, 1, 2, 3, -1, 5, -2], [4, 0, -1, 4, 3, 2 ** 31 - 1, -2 ** 31]], np.int32)
    tokens = rng.integers(0, V, (2, 7, 3)).astype(np.int32)
    tokens[0, :, 1], tokens[1, 0], tokens[1, 3] = -1, [V, -2, 0], [0, 2 ** 31 - 1, -1]
    got = G.token_logprobs(h, t, gpu(tokens), gpu(node), top=4)
    check(got, x, node, tokens, 1.0, 4)


def test_an_accepted_path(h):
    """What a verify call answers, scored by the rows that chose it; slots past it add nothing."""
    rng = np.random.default_rng(2)
    B, N, V = 6, 12, 1003
    t, x = rows(rng, B, N, V, "bf16", 1.0)
    parent = np.array([[-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, N)]
                       for _ in range(B)], np.int32)
    token = np.zeros((B, N), np.int32)
    for b in range(B):
        for i in range(1, N):          # half of the drafts are what the target likes best
            token[b, i] = x[b, parent[b, i]].argmax() if i % 2 else rng.integers(0, V)
    res = G.verify_greedy(h, t, gpu(token), gpu(parent))
    got = G.token_logprobs(h, t, res["out_tokens"], res["kv_commit"], top=1)
    check(got, x, res["kv_commit"].cpu().numpy(), res["out_tokens"].cpu().numpy(), 1.0, 1)
    live = res["kv_commit"] >= 0
    assert torch.equal(got["top_ids"][..., 0][live], res["out_tokens"][live])     # greedy answers


@pytest.mark.parametrize("B,N", [(1, 2), (64, 20)])
def test_repeated_and_captured(h, B, N):
    rng = np.random.default_rng(B)
    t, _ = rows(rng, B, N, 20011, "bf16")
    tokens = gpu(rng.integers(0, 20011, (B, N)).astype(np.int32))
    first = G.token_logprobs(h, t, tokens, top=16)
    for _ in range(4):
        again = G.token_logprobs(h, t, tokens, top=16)
        assert all(torch.equal(first[k], again[k]) for k in first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = G.token_logprobs(h, t, tokens, top=16)
    t.copy_(t.flip(0).clone() if B > 1 else t * 0.5)
    g.replay()
    again = G.token_logprobs(h, t, tokens, top=16)
    assert all(torch.equal(held[k], again[k]) for k in held)


@pytest.mark.parametrize("kw", [dict(temperature=0.0), dict(temperature=-1.0), dict(top=33),
                                dict(temperature=float("nan")), dict(temperature=1e-40), dict(B=65),
                                dict(C=65)])
def test_library_refusals(h, kw):
    B = kw.get("B", 1)
    t = torch.zeros((B, 2, 50), device=DEV)
    tokens = torch.zeros((B, 2, kw.get("C", 1)), dtype=torch.int32, device=DEV)
    with pytest.raises(G.SpecError):
        G.token_logprobs(h, t, tokens, temperature=kw.get("temperature", 1.0), top=kw.get("top", 1))
    torch.cuda.synchronize()


def test_an_empty_batch(h):
    got = G.token_logprobs(h, torch.zeros((0, 2, 50), device=DEV), top=3)
    assert got["top_ids"].shape == (0, 2, 3)
