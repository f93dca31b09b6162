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
            assert np.array_equal(np.isnan(lse[rows]), np.isnan(r["lse"]))
            some = np.isfinite(r["lse"])
            ref = r["lse"][some]
            ltol = soft[some] + 2.0 ** -24 * L + 2.0 ** -22 * np.abs(ref)
            assert np.all(np.abs(lse[rows][some] - ref) <= ltol)


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
    ([129, 64], [0, 64], 1, 2, 48), ([100], [50], 1, 2, 256), ([130, 20], [300, 0], 2, 4, 192),
    ([17], [900], 1, 2, 256), ([5, 0, 70], [40, 7, 0], 1, 8, 256),
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


def place(c, b, p):
    """The block and offset of position p of request b."""
    return int(c.table[b, p // c.bs]), p % c.bs


def put(c, which, b, p, head, d, value):
    """Sets an element of the cache and of the oracle's copy."""
    blk, off = place(c, b, p)
    t = (c.k, c.v)[which]
    at = (blk, off, head, d) if c.layout == S.NHD else (blk, head, off, d)
    if t.element_size() == 1:       # the code of a NaN or an infinity
        code = 0x7F if c.kind == "e4m3" else 0x7C if value == np.inf else 0x7E
        t.view(torch.uint8)[at] = code
        value = np.nan if c.kind == "e4m3" else value
    else:
        t[at] = value
    (c.k64, c.v64)[which][b][p, head, d] = value


@pytest.mark.parametrize("dt,cache", [("bf16", "same"), ("f16", "same"), ("bf16", "e4m3"),
                                      ("f16", "e5m2")])
@pytest.mark.parametrize("counts,pos,Gq,D,window,sinks", [
    ([5, 3], [100, 0], 2, 64, 0, 0), ([6, 1], [400, 30], 2, 128, 37, 5), ([3], [200], 1, 256, 50, 2),
    ([130, 40], [60, 0], 2, 64, 0, 0), ([70, 100], [700, 300], 2, 128, 260, 3),
    ([70, 33], [300, 0], 2, 256, 90, 3)])
def test_values_that_are_no_numbers(h, dt, cache, counts, pos, Gq, D, window, sinks):
    """NaN and infinities in K and V reach the rows that see them, and no others."""
    rng = np.random.default_rng(D + len(counts))
    c = Case(rng, counts, pos, 2, Gq, D, dt, cache, S.HND, 16, window, sinks)
    for b, n in enumerate(counts):
        last = pos[b] + n - 1
        put(c, 1, b, last, 0, 3, np.inf)                  # the last row alone sees it
        put(c, 1, b, pos[b] + n // 2, 1, D - 1, np.nan)   # about half of the rows
        put(c, 0, b, last, 1, 5, np.nan)                  # a key: the whole last row
        if window and pos[b] > window + n:
            put(c, 1, b, pos[b] - window + n // 2, 0, 7, np.inf)     # leaves the window on the way
    out, lse = c.run(h)
    c.check(out, lse)


@pytest.mark.parametrize("n,Gq", [(3, 2), (90, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 4)])
def test_blocks_outside_the_cache(h, n, Gq, window, sinks):
    rng = np.random.default_rng(5)
    c = Case(rng, [n, n, 1], [300, 0, 600], 2, Gq, 64, "bf16", "same", S.NHD, 16, window, sinks)
    c.table[0, 18] = -1
    c.table[1, 0] = c.k.shape[0]
    c.table[2, 3] = 2 ** 31 - 1        # outside the window if there is one
    st = torch.full((3,), 9, dtype=torch.int32, device=DEV)
    out, lse = c.run(h, st)
    assert st.tolist() == [S.BAD_SLOT, S.BAD_SLOT, 0 if window else S.BAD_SLOT]
    c.check(out, lse)


@pytest.mark.parametrize("n,Gq", [(2, 2), (70, 4)])
def test_rows_of_no_request_stay(h, n, Gq):
    """Rows behind the last request, of requests out of range and of those over max_new are left."""
    rng = np.random.default_rng(7)
    c = Case(rng, [n, n, n], [10, 20, 30], 1, Gq, 64, "f16", spare=5)
    T = 3 * n + 5
    work = torch.empty(G.spec_paged_attention_workspace(h, 3, T, n, Gq, 1, 64), dtype=torch.uint8,
                       device=DEV)

    def call(start, max_new=n, pos=(10, 20, 30)):
        out = torch.full((T, Gq, 64), 7.0, dtype=torch.float16, device=DEV)
        lse = torch.full((T, Gq), 7.0, device=DEV)
        st = torch.full((3,), 9, dtype=torch.int32, device=DEV)
        G.spec_paged_attention(h, c.q, c.cache(), gpu(c.table), gpu(np.array(pos, np.int32)),
                               c.scale, out, work, gpu(np.array(start, np.int32)),
                               max_new=max_new, lse=lse, status=st)
        return out, lse, st.tolist()

    out, lse, st = call([0, n, 2 * n, 3 * n])
    assert st == [0, 0, 0] and (out[3 * n:] == 7).all() and (lse[3 * n:] == 7).all()
    assert not (lse[:3 * n] == 7).any()
    out, lse, st = call([-1, n, 2 * n, T + 1])
    assert st == [S.BAD_RANGE, 0, S.BAD_RANGE]
    assert (out[:n] == 7).all() and (out[2 * n:] == 7).all() and not (lse[n:2 * n] == 7).any()
    out, lse, st = call([0, n, n - 1, 2 * n - 1])
    assert st == [0, S.BAD_RANGE, 0]
    out, lse, st = call([0, n + 1, n + 1, 2 * n + 1])
    assert st == [S.BAD_RANGE, 0, 0] and (lse[:n + 1] == 7).all()


@pytest.mark.parametrize("n", [4, 80])
def test_positions_outside_the_table(h, n):
    """Rows before position 0 see nothing; rows past the table see what is in it."""
    rng = np.random.default_rng(8)
    c = Case(rng, [n, n], [-3, 40], 2, 2, 64, "bf16")
    pages = c.table.shape[1]
    st = torch.full((2,), 9, dtype=torch.int32, device=DEV)
    out, lse = c.run(h, st)
    assert st.tolist() == [S.BAD_SLOT, 0]
    c.check(out, lse)
    assert (out[:3] == 0).all() and (lse[:3] == -np.inf).all()
    c.pos = [-(2 ** 31), 2 ** 31 - 1]
    out, lse = c.run(h, st)
    assert st.tolist() == [S.BAD_SLOT, S.BAD_SLOT]
    assert (out[:n] == 0).all() and (lse[:n] == -np.inf).all()
    assert torch.isfinite(lse[n:]).all() or pages * 16 > 40 + n     # unused pages hold NaN


@pytest.mark.parametrize("B,n,Gq,D", [(3, 1, 4, 64), (2, 50, 2, 128), (64, 1, 1, 128)])
def test_equal_rows_without_row_start(h, B, n, Gq, D):
    rng = np.random.default_rng(B + n)
    c = Case(rng, [n] * B, list(rng.integers(0, 400, B)), 2, Gq, D, "bf16", "same", S.HND, 32)
    a = c.run(h, start=None, max_new=n)
    b = c.run(h, max_new=n)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    c.check(*a)


@pytest.mark.parametrize("dt,cache", [("bf16", "same"), ("f16", "e4m3")])
def test_few_and_many_rows_of_one_batch(h, dt, cache):
    """Requests of one token beside chunks, K and V of a block side by side: each kernel takes its
    own."""
    rng = np.random.default_rng(11)
    counts = [1, 40, 0, 1, 9, 130, 1, 16, 17, 2]
    pos = [900, 0, 5, 0, 250, 20, 131, 64, 3000, 1]
    c = Case(rng, counts, pos, 2, 2, 128, dt, cache, S.NHD, 16, apart=True)
    st = torch.full((10,), 9, dtype=torch.int32, device=DEV)
    out, lse = c.run(h, st, max_new=130)
    assert st.tolist() == [0] * 10
    c.check(out, lse)


@pytest.mark.parametrize("counts", [[40, 40, 1], [40, 40, 2], [40, 0, 40], [40, 39], [33, 1], [1, 33]])
@pytest.mark.parametrize("Gq", [1, 8])
def test_the_fewest_rows_that_a_batch_may_hold(h, counts, Gq):
    """Where the sizes given leave room for a request of few rows, and where they do not."""
    c = Case(np.random.default_rng(len(counts)), counts, [70] * len(counts), 1, Gq, 64, "f16")
    c.check(*c.run(h, max_new=max(counts)))


@pytest.mark.parametrize("counts,Gq", [([1, 1, 1], 8), ([200, 1, 30], 4)])
def test_repeated_and_captured(h, counts, Gq):
    """The same bits every time, on a stream of the caller's, and from two graphs that share a
    workspace; a replay follows new lengths."""
    rng = np.random.default_rng(13)
    pos = [2000, 700, 90]
    c = Case(rng, counts, pos, 2, Gq, 128, "bf16")
    T, B = sum(counts), 3
    first = c.run(h)
    for _ in range(5):
        assert all(torch.equal(x, y) for x, y in zip(first, c.run(h)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = c.run(h, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    work = torch.empty(G.spec_paged_attention_workspace(h, B, T, 0, 2 * Gq, 2, 128),
                       dtype=torch.uint8, device=DEV)
    table, at, start = gpu(c.table), gpu(np.array(pos, np.int32)), gpu(c.start)
    outs = [(torch.zeros_like(first[0]), torch.zeros_like(first[1])) for _ in range(2)]
    graphs = []
    for out, lse in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            G.spec_paged_attention(h, c.q, c.cache(), table, at, c.scale, out, work, start, lse=lse)
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(x, y) for x, y in zip(first, o))
    c.pos = [1500, 3, 90]
    at.copy_(gpu(np.array(c.pos, np.int32)))
    graphs[0].replay()
    assert all(torch.equal(x, y) for x, y in zip(c.run(h), outs[0]))


@pytest.mark.parametrize("n,Gq", [(1, 4), (60, 2)])
def test_blocks_beyond_four_gigabytes(h, n, Gq):
    """A cache of more than 2^32 bytes, its last blocks in use."""
    rng = np.random.default_rng(17)
    c = Case(rng, [n], [300], 1, Gq, 128, "bf16")
    nb = (2 ** 32 + 2 ** 28) // (16 * 128 * 2)
    small_k, small_v, table, m = c.k, c.v, c.table, c.k.shape[0]
    c.k = torch.empty((nb, 16, 1, 128), dtype=torch.bfloat16, device=DEV)
    c.v = torch.empty((nb, 16, 1, 128), dtype=torch.bfloat16, device=DEV)
    c.k[nb - m:], c.v[nb - m:] = small_k, small_v
    c.table = table + (nb - m)
    out, lse = c.run(h)
    c.check(out, lse)


@pytest.mark.parametrize("std", [1e-30, 30.0, 3e3])
@pytest.mark.parametrize("n,Gq", [(3, 4), (80, 2)])
def test_scores_of_any_size(h, n, Gq, std):
    """Tiny scores weigh all keys alike; huge ones leave one key: numbers, and lse near its score."""
    rng = np.random.default_rng(19)
    c = Case(rng, [n], [500], 2, Gq, 64, "bf16", std=std)
    out, lse = c.run(h)
    r = S.attention(c.q64, c.k64[0], c.v64[0], 500 + np.arange(n), np.ones(500 + n, bool), c.scale, 0,
                    0)
    assert torch.isfinite(out).all()
    got = lse.double().cpu().numpy()
    tol = 2 * 2.0 ** -20 * (2 + r["X"]) + 2.0 ** -24 * 600 + 2.0 ** -22 * np.abs(r["lse"])
    assert np.all(np.abs(got - r["lse"]) <= tol)
    if std < 1:
        c.check(out, lse)


def test_an_empty_batch(h):
    c = Case(np.random.default_rng(1), [1], [3], 1, 1, 64, "bf16")
    none = torch.zeros((0, 1, 64), dtype=torch.bfloat16, device=DEV)
    out, lse = G.paged_attention(h, none, c.cache(), gpu(c.table), gpu(np.zeros(1, np.int32)), 1.0,
                                 gpu(np.zeros(2, np.int32)))
    assert out.shape == (0, 1, 64) and lse.shape == (0, 1)
    out, lse = G.paged_attention(h, none, c.cache(), gpu(c.table[:0]), gpu(np.zeros(0, np.int32)), 1.0)
    assert out.shape == (0, 1, 64)


@pytest.mark.parametrize("kw", [
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(window=-1), dict(sinks=-1), dict(max_new=-1), dict(D=24), dict(D=272), dict(Hq=3),
    dict(B=65), dict(work=0), dict(work="off"), dict(dtype="f32")])
def test_library_refusals(h, kw):
    dt = torch.float32 if kw.get("dtype") else torch.bfloat16
    D, Hq, B = kw.get("D", 64), kw.get("Hq", 4), kw.get("B", 2)
    q = torch.zeros((B, Hq, D), dtype=dt, device=DEV)
    cache = G.KvCache.empty(4, 16, 2, D, dt, DEV)
    work = torch.empty(32 << 20, dtype=torch.uint8, device=DEV)
    work = {"off": work[16:], 0: work[:0]}.get(kw.get("work"), work)
    one = torch.zeros(B, dtype=torch.int32, device=DEV)
    with pytest.raises(G.SpecError):
        G.spec_paged_attention(h, q, cache, torch.zeros((B, 4), dtype=torch.int32, device=DEV), one,
                               kw.get("scale", 0.1), torch.empty_like(q), work,
                               max_new=kw.get("max_new", 0), window=kw.get("window", 0),
                               sinks=kw.get("sinks", 0))
    torch.cuda.synchronize()


def test_rows_that_do_not_divide(h):
    q = torch.zeros((5, 2, 64), dtype=torch.bfloat16, device=DEV)
    cache = G.KvCache.empty(4, 16, 2, 64, torch.bfloat16, DEV)
    with pytest.raises(G.SpecError):
        G.paged_attention(h, q, cache, torch.zeros((2, 4), dtype=torch.int32, device=DEV),
                          torch.zeros(2, dtype=torch.int32, device=DEV), 0.1)
