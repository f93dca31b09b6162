"""Tree attention where float32, and the 16-bit probabilities, come to their limits (needs a GB300):
weights far below a row's largest, scale factors at the ends of float32, scores of any size."""
import numpy as np
import pytest
import torch

import test_gpu_tree_step as T
from oracle import tree_step as S
from speculative_decoding_tree_mask_gb300 import binding as G

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# one warp-kernel and tcgen05 shape of each kind: groups of rows, items of up to 128 rows, of 256
SHAPES = [(1, 4, 64), (6, 4, 128), (16, 1, 256), (40, 2, 64), (64, 1, 128), (64, 4, 128),
          (64, 4, 64)]


@pytest.fixture(scope="module")
def h():
    G.load()
    with G.Handle(64, 64, 1 << 10, 0) as handle:
        yield handle


class Flat:
    """One request over `ctx` positions in order, one K/V head, a K of one element (the first) that
    the caller chooses per position, and V codes of [ctx, D] under block scales of 1."""

    def __init__(self, rng, N, Gq, D, dt, ctx, k_code, bs=64):
        pages = (ctx + bs - 1) // bs
        self.N, self.Gq, self.D, self.dt, self.ctx = N, Gq, D, dt, ctx
        self.cache = T.empty_cache(S.NHD, pages, bs, 1, D, fill=0x38)     # block scales: 1
        codes = np.zeros((pages * bs, D), np.uint8)
        codes[:ctx, 0] = k_code
        self.k0 = np.where(k_code >= 8, -1, 1) * S.E2M1[k_code & 7]
        self.cache.k.copy_(T.gpu(S.pack(codes)).view(self.cache.k.shape))
        codes = rng.integers(1, 8, (pages * bs, D)).astype(np.uint8)
        self.v = S.E2M1[codes[:ctx]]
        self.cache.v.copy_(T.gpu(S.pack(codes)).view(self.cache.v.shape))
        self.table = T.gpu(np.arange(pages, dtype=np.int32)[None])
        self.q = torch.zeros((1, N, Gq, D), dtype=T.TDT[dt], device=DEV)
        self.tk = torch.zeros((1, N, 1, D), dtype=T.TDT[dt], device=DEV)
        self.tv = T.rows(rng, 1, N, 1, D, dt)[0].abs()
        self.mask = np.uint64([(1 << (i + 1)) - 1 for i in range(N)])      # a chain

    def run(self, h, scale):
        out, lse = G.tree_attention_fp4(h, self.q, self.tk, self.tv, self.cache, self.table,
                                        T.gpu(np.int32([self.ctx])),
                                        T.gpu(self.mask.view(np.int64)[None]), scale)
        return out[0].double().cpu().numpy(), lse[0].double().cpu().numpy()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("N,Gq,D", SHAPES)
@pytest.mark.parametrize("octaves,every", [(20.3, 32), (24.5, 32), (25.01, 32), (25.01, 20011)])
def test_many_keys_far_below_the_largest(h, dt, N, Gq, D, octaves, every):
    """Keys with values of zero that outweigh all others by 2^octaves: what remains of the others
    is the whole result. A probability is held in 16 bits with the row's largest at 2^7 or more
    when the others meet it: 2^(7 - 25.01) errs by half of 2^-24, 2^-7 of itself, whatever the
    number of keys. Then the scores' and sums' 2^-14 (|x| is at most 26) and the result's
    rounding; a float16 result below 2^-14 errs by half of 2^-24."""
    rng = np.random.default_rng(int(octaves * 10))
    ctx = 20011
    code = np.zeros(ctx, np.int64)
    code[::every] = 7                                          # 6 under a scale of 1
    c = Flat(rng, N, Gq, D, dt, ctx, code)
    c.q[..., 0] = 1.0
    sink = code == 7
    pages = c.cache.v.view(-1, D // 2)
    pages[:ctx][T.gpu(sink)] = 0
    c.v[sink] = 0
    scale = octaves * np.log(2) / 6
    got, gl = c.run(h, scale)
    tv = c.tv[0, :, 0].double().cpu().numpy()
    tail = 2.0 ** -octaves
    top = sink.sum()
    rest = (ctx - top + 1 + np.arange(N)) * tail
    ref = (c.v.sum(0) + np.cumsum(tv, 0)) * tail / (top + rest)[:, None]
    tol = (2.0 ** -7 + 2.0 ** -14 + torch.finfo(T.TDT[dt]).eps / 2) * ref
    tol += 2.0 ** -25 if dt == "f16" else 0.0
    assert np.all(np.abs(got - ref[:, None]) <= tol[:, None]), np.abs(got / ref[:, None] - 1).max()
    want = octaves * np.log(2) + np.log(top + rest)
    assert np.all(np.abs(gl - want[:, None]) <= 2.0 ** -20 * 32)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("N,Gq,D", SHAPES)
@pytest.mark.parametrize("log_ks,log_q,scale", [(-100, 0, None), (-30, 0, None), (100, -100, None),
                                                (0, 0, 1e-30), (0, 0, 1e-44)])
def test_scale_factors_at_the_ends_of_float32(h, dt, N, Gq, D, log_ks, log_q, scale):
    """Rows of zeros among others, under tensor scales and a `scale` that bring the factor of the
    scores out of float32's range: the scores are numbers, so the results are."""
    if dt == "f16" and log_q < 0:
        log_q = -14                    # its range; the scores are then large, but numbers
        log_ks = 14
    rng = np.random.default_rng(N + D)
    c = T.Case(rng, 2, N, 1, Gq, D, dt, S.NHD, 16, [300, 1])
    c.scales = (2.0 ** log_ks, c.scales[1])
    c.cache.k_scale.fill_(2.0 ** log_ks)
    c.q.mul_(2.0 ** log_q)
    c.q[:, ::3] = 0
    if log_ks == 100:
        c.tk.mul_(2.0 ** 100)
        c.tk64 = c.tk.double().cpu().numpy()
    c.q64 = c.q.double().cpu().numpy()
    if scale is not None:
        c.scale = scale
    c.check(h)


@pytest.mark.parametrize("N,Gq,D", SHAPES)
def test_large_queries_and_keys_of_zeros(h, N, Gq, D):
    """Rows of 2^100 under a K scale of 2^100 over keys of zeros: all scores are zero."""
    rng = np.random.default_rng(N + D)
    c = T.Case(rng, 2, N, 1, Gq, D, "bf16", S.HND, 16, [300, 1])
    c.codes[0][:] = 0
    c.cache.k.zero_()
    c.scales = (2.0 ** 100, c.scales[1])
    c.cache.k_scale.fill_(2.0 ** 100)
    c.q.mul_(2.0 ** 100)
    c.tk.zero_()
    c.q64, c.tk64 = c.q.double().cpu().numpy(), c.tk.double().cpu().numpy()
    # the oracle's bound counts |q k|: zero
    c.check(h)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("N,Gq,D", SHAPES)
@pytest.mark.parametrize("log_q", [14, 15])
@pytest.mark.parametrize("scale", [0.1, 1e5, 3e9, 7e12, 1.3e20, 1e25, 1e33])
def test_scores_of_any_size(h, dt, N, Gq, D, log_q, scale):
    """Scores so large that float32 steps between them pass 2^5: the keys of the largest share the
    weight evenly. They are equal as products, so they are equal as probabilities: half a step
    of the result's type, the 2^-11 of the probabilities and the sums."""
    rng = np.random.default_rng(N + D)
    ctx = 700
    code = rng.integers(0, 7, ctx)
    best = rng.permutation(ctx)[:5]
    code[best] = 7
    c = Flat(rng, N, Gq, D, dt, ctx, code)
    c.q[..., 0] = 2.0 ** log_q
    c.tk[..., 0] = -1.0
    got, gl = c.run(h, scale)
    ref = c.v[best].mean(0)
    tol = (torch.finfo(T.TDT[dt]).eps / 2 * (1 + 2.0 ** -7) + 2.0 ** -11 + 2.0 ** -18) * ref
    assert np.all(np.abs(got - ref) <= tol)
    want = 6 * 2.0 ** log_q * float(np.float32(scale)) + np.log(5)
    assert np.all(np.abs(gl - want) <= 2.0 ** -21 * want)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("N,Gq,D", SHAPES)
@pytest.mark.parametrize("scale", [0.1, 1e20, 1e28, 1e33])
def test_large_negative_scores(h, dt, N, Gq, D, scale):
    """Every key's score is the same negative number, however large: the weights are even."""
    rng = np.random.default_rng(N + D)
    ctx = 300
    c = Flat(rng, N, Gq, D, dt, ctx, np.full(ctx, 15))
    c.q[..., 0] = 64.0
    c.tk[..., 0] = -6.0
    got, gl = c.run(h, scale)
    tv = c.tv[0, :, 0].double().cpu().numpy()
    keys = (ctx + 1 + np.arange(N))[:, None]
    ref = (c.v.sum(0) + np.cumsum(tv, 0)) / keys
    tol = (torch.finfo(T.TDT[dt]).eps / 2 * (1 + 2.0 ** -7) + 2.0 ** -11 + 2.0 ** -18) * ref
    assert np.all(np.abs(got - ref[:, None]) <= tol[:, None])
    want = -384 * float(np.float32(scale)) + np.log(keys)
    assert np.all(np.abs(gl - want) <= 2.0 ** -21 * np.abs(want))
