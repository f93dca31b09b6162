"""Attention of new tokens over the paged cache against the float64 oracle (needs a GB300).

Tolerances. A score in powers of two is a float32 sum of products (and the matrix unit may cut
rather than round), within 2^-20 X for sums of |q k| up to X; p = 2^x errs by as much and 2^-20, in
numerator and denominator; p is rounded to 16 bits (bfloat16 2^-8, half 2^-11, below 2^-14 by 2^-25
at most, with a row sum of at least 1). The result is rounded once, by finfo(t).eps / 2 of itself
(in half's subnormals by 2^-25). So an output errs by
  (u_P + 2 2^-20 (2 + X)) A + 2^-24 L max|v| + eps / 2 |out|,
A the p-weighted mean of |v|, L the keys; log sum exp by 2 2^-20 (2 + X) + 2^-24 L + 2^-22 |lse|.
"""
import numpy as np
import pytest
import torch

from oracle import paged_step as S
from speculative_decoding_tree_mask_gb300 import binding as G

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TDT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16,
       "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.fixture(scope="module")
def h():
    G.load()
    with G.Handle(64, 64, 1 << 10, 0) as handle:
        yield handle


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def typed(x, dt):
    """float array -> (tensor of the type on the GPU, its values in float64)."""
    t = torch.from_numpy(np.asarray(x, np.float32)).to(TDT[dt])
    if t.element_size() == 1:
        return t.to(DEV), S.fp8_values(t.view(torch.uint8).numpy(), dt == "e4m3")
    return t.to(DEV), t.double().numpy()


class Case:
    """A batch: counts[b] new tokens at pos[b], a cache whose unused places hold `junk`."""

    def __init__(self, rng, counts, pos, H, Gq, D, dt, cache="same", layout=S.NHD, bs=16, window=0,
                 sinks=0, pad=0, spare=0, junk=np.nan, apart=False, std=1.0):
        self.dt, self.kind = dt, dt if cache == "same" else cache
        self.H, self.Hq, self.D, self.bs, self.layout = H, H * Gq, D, bs, layout
        self.window, self.sinks = window, sinks
        self.counts, self.pos = list(counts), list(pos)
        B = len(counts)
        T = sum(counts) + spare
        q = rng.standard_normal((T, self.Hq * D + 2 * pad)) * 1.5 * std
        t, v64 = typed(q, dt)
        self.q = t[:, pad:pad + self.Hq * D].unflatten(1, (self.Hq, D))
        self.q64 = v64[:, pad:pad + self.Hq * D].reshape(T, self.Hq, D)
        self.start = np.cumsum([0] + self.counts).astype(np.int32)
        last = [max(0, p + n) for p, n in zip(pos, counts)]
        width = max(1, max((n + bs - 1) // bs for n in last))
        nb = B * width + 3
        self.table = rng.permutation(nb)[:B * width].reshape(B, width).astype(np.int32)
        shape = (nb, bs, H, D) if layout == S.NHD else (nb, H, bs, D)
        self.scales = (0.25, 0.5) if len(self.kind) == 4 and self.kind[0] == "e" else (1.0, 1.0)
        self.k64, self.v64, raw = [], [], [np.full(shape, junk), np.full(shape, junk)]
        for b, n in enumerate(last):
            for to, out, scale, f in ((raw[0], self.k64, self.scales[0], std),
                                      (raw[1], self.v64, self.scales[1], 1.0)):
                x = rng.standard_normal((n, H, D)) * f / scale
                for p in range(n):
                    blk, off = self.table[b, p // bs], p % bs
                    if layout == S.NHD:
                        to[blk, off] = x[p]
                    else:
                        to[blk, :, off] = x[p]
                out.append(x)
        kv = [typed(x, self.kind)[0] for x in raw]
        if apart:     # K and V of a block side by side in one tensor
            both = torch.stack([t.view(torch.uint8) for t in kv], 1).view(TDT[self.kind])
            kv = [both[:, 0], both[:, 1]]
        self.k, self.v = kv
        self.k64 = [typed(x, self.kind)[1] * self.scales[0] for x in self.k64]
        self.v64 = [typed(x, self.kind)[1] * self.scales[1] for x in self.v64]
        self.scale = D ** -0.5

    def cache(self):
        sc = [None if s == 1.0 else torch.tensor([s], device=DEV) for s in self.scales]
        return G.KvCache(self.k, self.v, self.layout, *sc)

    def run(self, h, status=None, max_new=0, start="given", **kw):
        return G.paged_attention(
            h, self.q, self.cache(), gpu(self.table), gpu(np.array(self.pos, np.int32)), self.scale,
            gpu(self.start) if isinstance(start, str) else start, max_new=max_new,
            window=self.window, sinks=self.sinks, status=status, **kw)

    def check(self, out, lse):
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        nb = self.k.shape[0]
        eps = torch.finfo(TDT[self.dt]).eps / 2
        up = 2.0 ** -8 if self.dt == "bf16" and self.kind == "bf16" else 2.0 ** -11
        for b, n in enumerate(self.counts):
            rows = slice(self.start[b], self.start[b] + n)
            L = len(self.k64[b])
            there = np.array([0 <= self.table[b, p // self.bs] < nb for p in range(L)], bool)
            r = S.attention(self.q64[rows], self.k64[b], self.v64[b], self.pos[b] + np.arange(n),
                            there, self.scale, self.window, self.sinks)
            big = np.abs(self.v64[b][np.isfinite(self.v64[b])]).max() if L else 0.0
            soft = 2 * 2.0 ** -20 * (2 + r["X"])
            tol = (up + soft[..., None]) * r["A"] + 2.0 ** -24 * L * big + eps * np.abs(r["out"])
            tol += 2.0 ** -25 if self.dt == "f16" else 0.0
            fine = np.isfinite(r["out"])
            assert np.array_equal(np.isnan(out[rows]), np.isnan(r["out"]))
            assert np.array_equal(out[rows][~fine & ~np.isnan(r["out"])],
                                  r["out"][~fine & ~np.isnan(r["out"])])
            err = np.abs(out[rows][fine] - r["out"][fine])
            assert np.all(err <= tol[fine]), (b, (err / tol[fine]).max())
            none = r["lse"] == -np.inf
            assert np.array_equal(lse[rows] == -np.inf, none)
            ref = r["lse"][~none]
            ltol = soft[~none] + 2.0 ** -24 * L + 2.0 ** -22 * np.abs(ref)
            assert np.all(np.abs(lse[rows][~none] - ref) <= ltol)


SIZES = [
    # counts, pos, H, Gq, D
    ([1], [0], 1, 1, 64), ([1, 1, 1], [0, 127, 128], 2, 4, 128), ([1, 0, 1], [300, 5, 31], 1, 16, 64),
    ([3, 1, 5], [0, 500, 1], 2, 3, 128), ([2], [1000], 2, 8, 96), ([1, 2], [40, 700], 2, 5, 256),
    ([4], [259], 1, 7, 80), ([20], [0], 2, 4, 256), ([1], [3000], 1, 20, 128),
]


@pytest.mark.parametrize("dt,cache", [("bf16", "same"), ("f16", "same"), ("bf16", "e4m3"),
                                      ("f16", "e5m2"), ("f16", "e4m3"), ("bf16", "e5m2")])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s[0])) + f"-D{s[4]}-G{s[3]}")
@pytest.mark.parametrize("layout,bs,window,sinks", [(S.NHD, 16, 0, 0), (S.HND, 8, 20, 3),
                                                    (S.NHD, 48, 129, 0), (S.HND, 64, 1, 200)])
def test_few_rows(h, dt, cache, size, layout, bs, window, sinks):
    counts, pos, H, Gq, D = size
    rng = np.random.default_rng(D + bs)
    c = Case(rng, counts, pos, H, Gq, D, dt, cache, layout, bs, window, sinks, pad=8)
    st = torch.full((len(counts),), 9, dtype=torch.int32, device=DEV)
    out, lse = c.run(h, st, max_new=max(counts))
    assert st.tolist() == [0] * len(counts)
    c.check(out, lse)


MANY = [
    ([33], [0], 1, 1, 64), ([70], [0], 1, 4, 128), ([300], [0], 1, 1, 128), ([65], [190], 2, 4, 64),
    ([1, 140, 0, 2], [700, 100, 3, 0], 2, 2, 128), ([257], [1], 1, 3, 96), ([90], [600], 1, 5, 80),
    ([129, 64], [0, 64], 1, 2, 48),
]


@pytest.mark.parametrize("dt,cache", [("bf16", "same"), ("f16", "same"), ("bf16", "e4m3"),
                                      ("f16", "e5m2"), ("f16", "e4m3"), ("bf16", "e5m2")])
@pytest.mark.parametrize("size", MANY, ids=lambda s: "x".join(map(str, s[0])) + f"-D{s[4]}-G{s[3]}")
@pytest.mark.parametrize("layout,bs,window,sinks", [(S.NHD, 16, 0, 0), (S.HND, 8, 20, 3),
                                                    (S.NHD, 48, 129, 0), (S.HND, 64, 100, 140)])
def test_many_rows(h, dt, cache, size, layout, bs, window, sinks):
    counts, pos, H, Gq, D = size
    rng = np.random.default_rng(D + bs + 1)
    c = Case(rng, counts, pos, H, Gq, D, dt, cache, layout, bs, window, sinks, pad=8)
    st = torch.full((len(counts),), 9, dtype=torch.int32, device=DEV)
    out, lse = c.run(h, st)
    assert st.tolist() == [0] * len(counts)
    c.check(out, lse)
