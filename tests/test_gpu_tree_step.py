"""The tree step over a 4-bit cache against the float64 oracle through the C ABI (needs a GB300).

Tolerances. One rounding to the output type is half a step, finfo(t).eps / 2 of the value.
Before it, float32 arithmetic:
  rotation: angle within 2 pi (2^-32 + 2^-25), sincospi within 2 steps, three products and a
      sum, the norm's sum of up to 256 squares in chains of at most 32, its root and two
      products: together below 2^-19 (|a| + |c|) for a pair;
  attention: a score is a float32 sum of products (and the matrix unit may cut rather than
      round), within 2^-20 X for sums of |q k| up to X; p = 2^x errs by as much and 2^-20, in
      numerator and denominator; p is rounded to a half (2^-11), or below 2^-14 by 2^-25 at
      most, with a row sum of at least 1. So an output errs by
      (2^-11 + 2 2^-20 (2 + X)) A + 2^-24 L max|v|, A the p-weighted mean of |v|, L the keys.
Cache codes are compared by the values they stand for, exactly.
"""
import numpy as np
import pytest
import torch

from oracle import tree_step as S
from speculative_decoding_tree_mask_gb300 import binding as G
from speculative_decoding_tree_mask_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TDT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def h():
    G.load()
    with G.Handle(64, 64, 1 << 10, 0) as handle:
        yield handle


def rows(rng, B, N, H, D, dt, pad=0, std=1.0):
    """Rows [B, N, H, D] of a type: values exactly representable, and the tensor on the GPU
    (inside a wider matrix when pad > 0, starting `pad` elements in)."""
    x = torch.from_numpy((rng.standard_normal((B, N, H * D + 2 * pad)) * std).astype(np.float32))
    t = x.to(TDT[dt]).to(DEV)
    t = t[:, :, pad:pad + H * D].unflatten(2, (H, D)) if pad else t.view(B, N, H, D)
    return t, t.double().cpu().numpy()


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


# ---- head norm and rotation --------------------------------------------------------------

@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D,rot,pairs,norm,pad", [
    (128, 128, False, True, 0), (128, 96, False, True, 8), (64, 64, True, True, 0),
    (64, 0, False, True, 0), (80, 42, False, True, 0), (80, 80, True, False, 4),
    (256, 256, False, True, 0), (128, 64, True, True, 3), (7, 4, False, True, 0),
    (1, 0, False, True, 1), (33, 32, True, True, 0), (512, 128, False, True, 0)])
def test_norm_rope(h, dt, D, rot, pairs, norm, pad):
    rng = np.random.default_rng(D * 1000 + rot)
    B, N, Hq, Hk = 3, 5, 6, 2
    q, q64 = rows(rng, B, N, Hq, D, dt, pad, 3.0)
    k, k64 = rows(rng, B, N, Hk, D, dt, pad, 0.01)
    q0, k0 = q.clone(), k.clone()
    f = (10000.0 ** -(np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    pos = np.array([0, 131071, 2000000000], np.int32)
    depth = rng.integers(-1, 5, (B, N)).astype(np.int32)
    wq = torch.from_numpy(rng.uniform(0.5, 2, D).astype(np.float32)).to(TDT[dt])
    wk = torch.from_numpy(rng.uniform(0.5, 2, D).astype(np.float32)).to(TDT[dt])
    qo, ko = G.qk_norm_rope(h, q, k, gpu(f) if rot else None, gpu(pos), gpu(depth),
                            wq.to(DEV) if norm else None, wk.to(DEV) if norm else None, 1e-5,
                            G.SPEC_ROPE_PAIRS if pairs else G.SPEC_ROPE_HALVES)
    torch.cuda.synchronize()
    assert torch.equal(q, q0) and torch.equal(k, k0)
    where = pos[:, None].astype(np.int64) + depth
    for got, x, w in ((qo, q64, wq), (ko, k64, wk)):
        w64 = w.double().numpy() if norm else None
        ref = S.norm_rope(x, w64, 1e-5, f, where, pairs)
        plain = np.abs(S.norm_rope(x, w64, 1e-5, f[:0], where, pairs))
        size = plain.copy()
        a = np.arange(rot // 2) * (2 if pairs else 1)
        c = a + (1 if pairs else rot // 2)
        size[..., a] = size[..., c] = plain[..., a] + plain[..., c]
        tol = torch.finfo(TDT[dt]).eps / 2 * np.abs(ref) + 2.0 ** -19 * size
        tol += 2.0 ** -25 if dt == "f16" else 0.0      # half a step of its subnormals
        assert np.all(np.abs(got.double().cpu().numpy() - ref) <= tol)
    # in place, and depth None = n itself
    q1, k1 = G.qk_norm_rope(h, q, k, gpu(f) if rot else None, gpu(pos), None,
                            wq.to(DEV) if norm else None, wk.to(DEV) if norm else None, 1e-5,
                            G.SPEC_ROPE_PAIRS if pairs else G.SPEC_ROPE_HALVES)
    G.spec_qk_norm_rope(h, q, k, gpu(f) if rot else None, gpu(pos),
                        gpu(np.tile(np.arange(N, dtype=np.int32), (B, 1))), q, k,
                        wq.to(DEV) if norm else None, wk.to(DEV) if norm else None, 1e-5,
                        G.SPEC_ROPE_PAIRS if pairs else G.SPEC_ROPE_HALVES)
    torch.cuda.synchronize()
    assert torch.equal(q1, q) and torch.equal(k1, k)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D,rot,pad", [(128, 90, 0), (64, 2, 8), (512, 250, 0), (256, 254, 16),
                                       (72, 70, 0), (16, 14, 0), (8, 6, 8)])
def test_rotation_across_vectors(h, dt, D, rot, pad):
    """Halves whose length is no multiple of a 16-byte vector, in place, with one head and many."""
    rng = np.random.default_rng(D + rot)
    B, N, Hq, Hk = 2, 3, 9, 1
    q, q64 = rows(rng, B, N, Hq, D, dt, pad, 2.0)
    k, k64 = rows(rng, B, N, Hk, D, dt, pad)
    f = (10000.0 ** -(np.arange(rot // 2) / (rot // 2))).astype(np.float32)
    pos = np.array([7, 500000], np.int32)
    w = torch.from_numpy(rng.uniform(0.5, 2, D).astype(np.float32)).to(TDT[dt])
    G.spec_qk_norm_rope(h, q, k, gpu(f), gpu(pos), None, q, k, w.to(DEV), w.to(DEV), 1e-6)
    torch.cuda.synchronize()
    where = pos[:, None].astype(np.int64) + np.arange(N)
    for got, x in ((q, q64), (k, k64)):
        ref = S.norm_rope(x, w.double().numpy(), 1e-6, f, where, False)
        plain = np.abs(S.norm_rope(x, w.double().numpy(), 1e-6, f[:0], where, False))
        size = plain.copy()
        a = np.arange(rot // 2)
        size[..., a] = size[..., a + rot // 2] = plain[..., a] + plain[..., a + rot // 2]
        tol = torch.finfo(TDT[dt]).eps / 2 * np.abs(ref) + 2.0 ** -19 * size
        tol += 2.0 ** -25 if dt == "f16" else 0.0
        assert np.all(np.abs(got.double().cpu().numpy() - ref) <= tol)


def test_norm_rope_many_tokens_and_special_values(h):
    """A prompt longer than the handle's trees; a NaN stays in its head; a row of zeros is zero."""
    rng = np.random.default_rng(5)
    B, N, Hq, Hk, D = 2, 700, 8, 1, 64
    q, q64 = rows(rng, B, N, Hq, D, "bf16")
    k, _ = rows(rng, B, N, Hk, D, "bf16")
    q[1, 5, 3, 7] = float("nan")
    q[0, 2, 1] = 0
    f = (10000.0 ** -(np.arange(32) / 32)).astype(np.float32)
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    qo, _ = G.qk_norm_rope(h, q, k, gpu(f), gpu(np.int32([3, 900])), None, w, w)
    got = qo.double().cpu().numpy()
    bad = np.isnan(got)
    assert bad[1, 5, 3].all() and bad.sum() == D
    assert np.all(got[0, 2, 1] == 0)
    q64[0, 2, 1] = 0
    ref = S.norm_rope(q64, np.ones(D), 1e-6, f, np.int64([[3], [900]]) + np.arange(N), False)
    ok = ~bad
    assert np.all(np.abs(got - ref)[ok] <= 2.0 ** -8 * np.abs(ref)[ok] + 2.0 ** -19 * 16)


# ---- the 4-bit cache ------------------------------------------------------------------------

def empty_cache(layout, blocks, bs, H, D, ks=1.0, vs=1.0, fill=0x55):
    c = G.Fp4Cache.empty(blocks, bs, H, D, DEV, layout,
                         torch.tensor([ks], device=DEV), torch.tensor([vs], device=DEV))
    for t in (c.k, c.v, c.k_sf, c.v_sf):
        t.fill_(fill)
    return c


def same_values(c, key, codes, sf):
    got = S.values(S.unpack(getattr(c, key).cpu().numpy()), getattr(c, key + "_sf").cpu().numpy())
    ref = S.values(codes, sf)
    assert np.array_equal(getattr(c, key + "_sf").cpu().numpy(), sf)
    assert np.array_equal(got, ref, equal_nan=True)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("layout", [S.NHD, S.HND])
@pytest.mark.parametrize("H,D,bs,path,pad", [(4, 128, 16, True, 0), (1, 16, 1, True, 16),
                                             (3, 80, 7, True, 8), (33, 256, 8, True, 0),
                                             (2, 48, 5, False, 1), (5, 64, 16, False, 0)])
def test_commit_and_load(h, dt, layout, H, D, bs, path, pad):
    rng = np.random.default_rng(H * D + bs)
    B, N = 13, 9
    src_k, k64 = rows(rng, B, N, H, D, dt, pad, 2.0)
    src_v, v64 = rows(rng, B, N, H, D, dt, pad, 0.3)
    width = (2 * bs + N - 1) // bs + 1
    blocks = B * width + 2
    table = rng.permutation(blocks)[:B * width].reshape(B, width).astype(np.int32)
    pos = rng.integers(0, bs, B).astype(np.int32)
    last = rng.integers(0, N, B).astype(np.int32)
    kv = None
    if path:
        kv = np.full((B, N), -1, np.int32)
        for b in range(B):
            kv[b, :last[b] + 1] = np.concatenate(
                ([0], 1 + np.sort(rng.permutation(N - 1)[:last[b]])))
        kv[4] = -1                                     # its verification failed
    else:
        last[4] = -1                                   # nothing to write
    last[6] = last[7] = last[8] = 2
    if path:
        kv[6:9, :3] = [0, 1, 2]
        kv[8, 1] = N                                   # no such node
    pos[6] = width * bs - 1                            # runs out of the table
    table[7, (int(pos[7]) + 1) // bs] = blocks         # a block outside the cache
    pos[9], last[9] = -1, max(last[9], 1)              # begins before the sequence
    if path:
        kv[9, :2] = [0, 1]
        kv[9, 2:last[9] + 1] = np.arange(2, last[9] + 1)
    c = empty_cache(layout, blocks, bs, H, D, 0.75, 2.0 ** -4)
    st = torch.full((B,), -7, dtype=torch.int32, device=DEV)
    G.spec_kv_commit_fp4(h, src_k, src_v, c, gpu(table), gpu(pos), None if kv is None else gpu(kv),
                         gpu(last), st)
    torch.cuda.synchronize()
    shape = (blocks, bs, H) if layout == S.NHD else (blocks, H, bs)
    c0 = np.full(shape + (D,), 5, np.uint8)
    f0 = np.full(shape + (D // 16,), 0x55, np.uint8)
    rk, rkf, rst = S.commit(k64, c0, f0, layout, bs, table, pos, 0.75, kv, last)
    rv, rvf, _ = S.commit(v64, c0, f0, layout, bs, table, pos, 2.0 ** -4, kv, last)
    assert st.cpu().numpy().tolist() == rst.tolist()
    assert rst[6] == rst[7] == rst[9] == S.BAD_SLOT and (not path or rst[8] == S.BAD_SLOT)
    same_values(c, "k", rk, rkf)
    same_values(c, "v", rv, rvf)
    # and back: counts from none to more than there is
    most = N + 2
    count = np.minimum(last + 1, most).astype(np.int32)
    count[1] = 0
    count[2] = most + 1
    out_k, out_v = (torch.full((B, most, H, D), 9.0, dtype=TDT[dt], device=DEV) for _ in range(2))
    st.fill_(-7)
    G.spec_kv_load_fp4(h, c, gpu(table), gpu(pos), gpu(count), out_k, out_v, st)
    torch.cuda.synchronize()
    want = np.zeros(B, np.int32)
    for out, codes, sf, ts in ((out_k, rk, rkf, 0.75), (out_v, rv, rvf, 2.0 ** -4)):
        got = out.cpu()
        for b in range(B):
            want[b] |= S.BAD_SLOT if count[b] > most or count[b] < 0 else 0
            for i in range(most):
                x = None
                if i < count[b]:
                    x = S.read(codes, sf, layout, bs, table, b, int(pos[b]) + i, ts)
                    want[b] |= S.BAD_SLOT if x is None else 0
                x = np.zeros((H, D)) if x is None else x
                # six significant bits times 0.75 or a power of two: exact in all three types
                # but for the halves' subnormals, which round once
                x = torch.from_numpy(x).to(TDT[dt])
                assert torch.equal(got[b, i], x), (b, i)
    assert st.cpu().numpy().tolist() == want.tolist()


def test_commit_rounding_and_special_values(h):
    """Values on and beside every rounding boundary of codes and scales, zeros, infinities, NaN
    and blocks too small or too large for a scale: the stored values equal the oracle's."""
    rng = np.random.default_rng(11)
    n = 4096
    x = np.zeros((n, 16), np.float32)
    grid = (S.E2M1[1:] + S.E2M1[:-1]) / 2
    for i in range(n):
        s = S.E4M3[rng.integers(1, 0x7F)]
        v = grid[rng.integers(0, 7, 16)] * s
        v = (v.astype(np.float32).view(np.int32) + rng.integers(-2, 3, 16)).astype(
            np.int32).view(np.float32)
        x[i] = v * rng.choice([-1, 1], 16)
        x[i, rng.integers(0, 16)] = 6 * s
    x[0] = 0
    x[1, 3] = np.nan
    x[2, 5] = np.inf
    x[3, 1] = -np.inf
    x[4] = 1e-9
    x[5] = 1e9
    x[6, :] = -0.0
    x[7] = np.float32(1e-40)
    N, D = 64, 64
    src = torch.from_numpy(x.reshape(n * 16 // (N * D), N, 1, D)).to(DEV)
    B = src.shape[0]
    for ts in (1.0, 0.3):
        c = empty_cache(S.NHD, B, N, 1, D, ts, ts, 0)
        G.spec_kv_commit_fp4(h, src, src, c, gpu(np.arange(B, dtype=np.int32)[:, None]),
                             gpu(np.zeros(B, np.int32)))
        codes, sf = S.quantise(x.reshape(B, N, 1, D), ts)
        same_values(c, "k", codes, sf)
        same_values(c, "v", codes, sf)


def test_cache_offsets_past_32_bits(h):
    """Blocks whose codes lie more than 4 GiB into the cache (its memory is not initialised:
    only the pages written are read)."""
    H, D, bs = 8, 128, 16
    blocks = (5 << 30) // (bs * H * (D // 2))
    shape = (blocks, bs, H)
    t = [torch.empty(shape + (m,), dtype=torch.uint8, device=DEV)
         for m in (D // 2, D // 2, D // 16, D // 16)]
    c = G.Fp4Cache(*t)
    table = np.int32([[blocks - 1, 3, blocks // 2 + 7, blocks - 2]])
    rng = np.random.default_rng(12)
    src, x = rows(rng, 1, 60, H, D, "bf16")
    G.spec_kv_commit_fp4(h, src, src, c, gpu(table), gpu(np.int32([2])))
    k, v = G.kv_load_fp4(h, c, gpu(table), gpu(np.int32([2])), gpu(np.int32([60])), 60,
                         torch.float32)
    ref = S.values(*S.quantise(x))
    assert np.array_equal(k.cpu().numpy(), ref) and np.array_equal(v.cpu().numpy(), ref)
    q, q64 = rows(rng, 1, 1, 16, D, "bf16", 0, 2.0)
    tk, tk64 = rows(rng, 1, 1, H, D, "bf16")
    out, _ = G.tree_attention_fp4(h, q, tk, tk, c, gpu(table), gpu(np.int32([62])),
                                  gpu(np.int64([[1]])), 0.1)
    # positions 0 and 1 were never written: rows of zeros there
    G.spec_kv_commit_fp4(h, torch.zeros_like(src), torch.zeros_like(src), c, gpu(table),
                         gpu(np.int32([0])), accept_len=gpu(np.int32([1])))
    out, lse = G.tree_attention_fp4(h, q, tk, tk, c, gpu(table), gpu(np.int32([62])),
                                    gpu(np.int64([[1]])), 0.1)
    ctx = np.concatenate((np.zeros((2, H, D)), ref[0]))
    check_attention(out, lse, [(q64[0], tk64[0], tk64[0], ctx, ctx, np.uint64([1]))], 0.1, "bf16")


# ---- attention ------------------------------------------------------------------------------

def check_attention(out, lse, requests, scale, dt):
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, (q, tk, tv, keys, vals, mask) in enumerate(requests):
        ref, rl, size, big = S.attend(q, tk, tv, keys, vals, mask, scale)
        vmax = max([np.abs(v).max() for v in (tv, vals) if v.size] + [0.0])
        f = 2.0 ** -20 * (2 + big)
        tol = torch.finfo(TDT[dt]).eps / 2 * np.abs(ref) * (1 + 2.0 ** -7) + \
            (2.0 ** -11 + 2 * f)[..., None] * size + 2.0 ** -24 * (len(keys) + len(tk)) * vmax
        tol += 2.0 ** -25 if dt == "f16" else 0.0
        assert np.all(np.abs(got[b] - ref) <= tol), (b, np.abs(got[b] - ref).max())
        seen = np.isfinite(rl)
        assert np.array_equal(np.isfinite(gl[b]), seen) and np.all(gl[b][~seen] == -np.inf)
        assert np.all(np.abs(gl[b][seen] - rl[seen]) <=
                      2 * f[seen] + 2.0 ** -22 * np.abs(rl[seen]) + 2.0 ** -20)


class Case:
    """A batch: a cache with values everywhere, a tree per request, and the oracle's view."""

    def __init__(self, rng, B, N, H, Gq, D, dt, layout, bs, ctx, chain=False, pad=0):
        self.B, self.N, self.H, self.D, self.dt, self.layout, self.bs = B, N, H, D, dt, layout, bs
        self.ctx = np.array(ctx, np.int32)
        width = max(1, (int(max(ctx)) + bs - 1) // bs)
        blocks = B * width + 1
        self.table = rng.permutation(blocks)[:B * width].reshape(B, width).astype(np.int32)
        shape = (blocks, bs, H) if layout == S.NHD else (blocks, H, bs)
        self.scales = (0.75, 0.125)
        self.cache = empty_cache(layout, blocks, bs, H, D, *self.scales)
        self.codes, self.sf = [], []
        for key, ts, std in (("k", 0.75, 1.0), ("v", 0.125, 0.5)):
            x = rng.standard_normal(shape + (D,)) * std * 10.0 ** rng.uniform(-1, 0.5, (D,))
            c, s = S.quantise(x.astype(np.float32), ts)
            self.codes.append(c)
            self.sf.append(s)
            getattr(self.cache, key).copy_(gpu(S.pack(c)))
            getattr(self.cache, key + "_sf").copy_(gpu(s))
        self.q, self.q64 = rows(rng, B, N, H * Gq, D, dt, pad, 2.0)
        self.tk, self.tk64 = rows(rng, B, N, H, D, dt, pad)
        self.tv, self.tv64 = rows(rng, B, N, H, D, dt, pad, 0.5)
        parent = np.stack([np.arange(-1, N - 1) if chain else W.random_trie(rng, N, 64, 3)
                           for _ in range(B)])
        self.mask = np.zeros((B, N), np.uint64)
        for b in range(B):
            for i in range(N):
                up = self.mask[b, parent[b, i]] if i else np.uint64(0)
                self.mask[b, i] = up | np.uint64(1 << i)
        self.scale = float(D ** -0.5)

    def run(self, h, **kw):
        out, lse = G.tree_attention_fp4(h, self.q, self.tk, self.tv, self.cache, gpu(self.table),
                                        gpu(self.ctx), gpu(self.mask.view(np.int64)), self.scale,
                                        **kw)
        torch.cuda.synchronize()
        return out, lse

    def context(self, b):
        kv = [[S.read(c, f, self.layout, self.bs, self.table, b, p, ts)
               for p in range(int(self.ctx[b]))]
              for c, f, ts in zip(self.codes, self.sf, self.scales)]
        none = np.zeros((0, self.H, self.D))
        return [np.stack([x for x in r if x is not None]) if any(x is not None for x in r)
                else none for r in kv]

    def requests(self):
        return [(self.q64[b], self.tk64[b], self.tv64[b], *self.context(b), self.mask[b])
                for b in range(self.B)]

    def check(self, h):
        out, lse = self.run(h)
        check_attention(out, lse, self.requests(), self.scale, self.dt)
        return out, lse


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("N,Gq", [(1, 1), (1, 8), (5, 4), (3, 7), (64, 1), (17, 8), (33, 4)])
def test_attention(h, dt, D, N, Gq):
    rng = np.random.default_rng(D + 100 * N + Gq)
    layout, bs = (S.NHD, 16) if N % 2 else (S.HND, 32)
    Case(rng, 3, N, 2, Gq, D, dt, layout, bs, [0, 129, 300]).check(h)


@pytest.mark.parametrize("ctx", [0, 1, 15, 31, 32, 33, 127, 128, 129, 255, 257, 640])
def test_attention_context_lengths(h, ctx):
    rng = np.random.default_rng(ctx)
    Case(rng, 2, 4, 1, 2, 64, "bf16", S.HND, 16, [ctx, ctx // 2]).check(h)


@pytest.mark.parametrize("layout", [S.NHD, S.HND])
@pytest.mark.parametrize("bs", [1, 7, 16, 48, 200])
@pytest.mark.parametrize("pad", [0, 3])
def test_attention_pages_and_strides(h, layout, bs, pad):
    rng = np.random.default_rng(bs + 1000 * layout + pad)
    c = Case(rng, 2, 6, 3, 2, 128, "f16", layout, bs, [211, 150], pad=pad)
    out, lse = c.check(h)
    # an output that begins two bytes off
    ws = torch.empty(G.spec_tree_attention_workspace(h, 2, 6, 6, 3, 128), dtype=torch.uint8,
                     device=DEV)
    off = torch.zeros(out.numel() + 1, dtype=out.dtype, device=DEV)[1:].view(out.shape)
    G.spec_tree_attention_fp4(h, c.q, c.tk, c.tv, c.cache, gpu(c.table), gpu(c.ctx),
                              gpu(c.mask.view(np.int64)), c.scale, off, ws)
    torch.cuda.synchronize()
    assert torch.equal(off, out)


@pytest.mark.parametrize("N,Gq", [(1, 4), (6, 4), (40, 2)])
def test_attention_many_requests_and_splits(h, N, Gq):
    """More requests than lanes, of lengths from none to many tiles (items cut over CTAs), the
    same bits twice, and a longer batch than one whose parts share the workspace."""
    rng = np.random.default_rng(77 + N)
    ctx = [0, 1, 3000] + [int(x) for x in rng.integers(0, 700, 37)]
    c = Case(rng, 40, N, 2, Gq, 64, "bf16", S.NHD, 32, ctx)
    out, lse = c.check(h)
    again, lse2 = c.run(h)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_attention_one_long_request(h):
    """One item per head over 20000 positions: cut over many CTAs and joined."""
    rng = np.random.default_rng(78)
    c = Case(rng, 1, 1, 1, 2, 64, "f16", S.HND, 64, [20000])
    c.check(h)


@pytest.mark.parametrize("N,D", [(4, 64), (64, 128)])
def test_attention_rows_that_see_nothing(h, N, D):
    """Empty masks with and without a context, bits above N, one request without any."""
    rng = np.random.default_rng(79)
    c = Case(rng, 3, N, 2, 4, D, "bf16", S.NHD, 16, [0, 40, 0])
    c.mask[0, 1::2] = 0
    c.mask[1, :] = 0
    if N < 64:
        c.mask[2] |= np.uint64(1 << 63)
        c.mask[0] |= np.uint64((1 << 64) - (1 << N))
    out, lse = c.run(h)
    low = np.uint64((1 << N) - 1) if N < 64 else np.uint64(2 ** 64 - 1)
    c.mask &= low
    check_attention(out, lse, c.requests(), c.scale, "bf16")
    assert torch.all(out[0, 1::2] == 0) and torch.all(lse[0, 1::2] == -np.inf)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("N,Gq,D", [(6, 3, 64), (40, 4, 128), (20, 1, 256)])
def test_attention_unseen_nan_and_infinity(h, dt, N, Gq, D):
    """NaN and infinities in cache positions past the context, in unmapped pages, and in nodes
    that a row does not see change nothing; rows that see them follow the arithmetic."""
    rng = np.random.default_rng(80)
    c = Case(rng, 2, N, 2, Gq, D, dt, S.HND, 16, [37, 0])
    c.cache.k_sf.fill_(0x7F)
    c.cache.v_sf.fill_(0x7F)
    for b in range(2):                     # scales of the context alone are numbers
        for p in range(int(c.ctx[b])):
            blk, off = S.place(c.table, c.codes[0].shape[0], 16, b, p)
            c.cache.k_sf[blk, :, off] = gpu(c.sf[0][blk, :, off])
            c.cache.v_sf[blk, :, off] = gpu(c.sf[1][blk, :, off])
    # node 2: V infinite in one element, NaN in another; node 3: K NaN; seen by themselves only
    for i in range(N):
        c.mask[:, i] &= ~np.uint64(0b1100)
    c.mask[:, 2] |= np.uint64(0b0100)
    c.mask[:, 3] |= np.uint64(0b1000)
    c.tv[:, 2, :, 5] = float("inf")
    c.tv[:, 2, :, 6] = float("nan")
    c.tk[:, 3, 1, 0] = float("nan")
    out, lse = c.run(h)
    o = out.float().cpu().numpy()
    others = [i for i in range(N) if i not in (2, 3)]
    assert np.all(np.isfinite(o[:, others])) and torch.all(torch.isfinite(lse[:, others]))
    assert np.all(o[:, 2, :, 5] == np.inf) and np.all(np.isnan(o[:, 2, :, 6]))
    rest = [d for d in range(D) if d not in (5, 6)]
    assert np.all(np.isfinite(o[:, 2][..., rest]))
    assert np.all(np.isfinite(o[:, 3, :Gq])) and np.all(np.isnan(o[:, 3, Gq:]))
    req = []
    for b, (q, tk, tv, k, v, m) in enumerate(c.requests()):
        sel = others
        small = np.array([sum(1 << x for x, j in enumerate(sel) if int(m[i]) >> j & 1)
                          for i in sel], np.uint64)
        req.append((q[sel], tk[sel], tv[sel], k, v, small))
    check_attention(out[:, others], lse[:, others], req, c.scale, dt)


@pytest.mark.parametrize("N", [3, 64])
def test_attention_bad_pages_and_lengths(h, N):
    """Blocks outside the cache are not attended, lengths outside the table are clamped, and
    both are reported; the other requests are as ever."""
    rng = np.random.default_rng(81)
    c = Case(rng, 5, N, 1, 4, 128, "bf16", S.NHD, 16, [100, 100, 100, 100, 112])
    c.table[1, 2] = -2
    c.table[2, 6] = c.cache.num_blocks
    c.table[4, 1] = 2 ** 31 - 1
    c.ctx[3] = -5
    true = c.ctx.copy()
    c.ctx[4] = 10 ** 6
    st = torch.full((5,), 9, dtype=torch.int32, device=DEV)
    out = torch.empty_like(c.q)
    lse = torch.empty(out.shape[:3], device=DEV)
    ws = torch.empty(G.spec_tree_attention_workspace(h, 5, N, 4, 1, 128), dtype=torch.uint8,
                     device=DEV)
    G.spec_tree_attention_fp4(h, c.q, c.tk, c.tv, c.cache, gpu(c.table), gpu(c.ctx),
                              gpu(c.mask.view(np.int64)), c.scale, out, ws, lse, st)
    torch.cuda.synchronize()
    assert st.cpu().numpy().tolist() == [0, S.BAD_SLOT, S.BAD_SLOT, S.BAD_SLOT, S.BAD_SLOT]
    c.ctx = np.maximum(true, 0)
    check_attention(out, lse, c.requests(), c.scale, "bf16")


def test_attention_extreme_queries(h):
    """Rows of Q far from one in size (halves would overflow or vanish without their own
    scaling), rows of zeros, and scores far apart."""
    rng = np.random.default_rng(82)
    c = Case(rng, 1, 8, 1, 2, 128, "bf16", S.NHD, 16, [300])
    size = np.float64([1e-30, 1e-8, 1e-3, 1, 30, 0, 1e4, 1e-38])
    c.q.mul_(gpu(size.astype(np.float32)).view(1, 8, 1, 1).to(torch.bfloat16))
    c.q64 = c.q.double().cpu().numpy()
    out, lse = c.run(h)
    check_attention(out, lse, c.requests(), c.scale, "bf16")


@pytest.mark.parametrize("N", [2, 64])
def test_attention_in_a_graph_follows_its_inputs(h, N):
    """Captured once and replayed: lengths, tables, masks and rows are read when it runs; also
    on a stream of its own."""
    rng = np.random.default_rng(83)
    a = Case(rng, 4, N, 2, 4, 64, "bf16", S.NHD, 16, [50, 0, 200, 128])
    want, want_lse = a.run(h)
    dev = dict(table=gpu(a.table), ctx=gpu(a.ctx), mask=gpu(a.mask.view(np.int64)))
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    ws = torch.empty(G.spec_tree_attention_workspace(h, 4, N, 8, 2, 64), dtype=torch.uint8,
                     device=DEV)
    st = torch.zeros(4, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def call():
        G.spec_tree_attention_fp4(h, a.q, a.tk, a.tv, a.cache, dev["table"], dev["ctx"],
                                  dev["mask"], a.scale, out, ws, lse, st,
                                  stream=torch.cuda.current_stream())

    with torch.cuda.stream(s):
        call()
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    a.ctx = np.int32([10, 190, 0, 3])
    a.mask[:, -1] = 1
    dev["ctx"].copy_(gpu(a.ctx))
    dev["mask"].copy_(gpu(a.mask.view(np.int64)))
    for _ in range(2):
        out.fill_(7)
        g.replay()
    torch.cuda.synchronize()
    want, want_lse = a.run(h)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


# ---- refusals of the library (host checks: nothing is launched) ---------------------------------

def test_refusals(h):
    rng = np.random.default_rng(84)
    c = Case(rng, 2, 3, 2, 2, 64, "bf16", S.NHD, 16, [5, 6])
    ws = torch.empty(G.spec_tree_attention_workspace(h, 2, 3, 4, 2, 64), dtype=torch.uint8,
                     device=DEV)
    out = torch.empty_like(c.q)

    def attend(**kw):
        a = dict(q=c.q, k=c.tk, v=c.tv, cache=c.cache, block_table=gpu(c.table),
                 ctx_len=gpu(c.ctx), anc_mask=gpu(c.mask.view(np.int64)), scale=0.1, out=out,
                 workspace=ws)
        a.update(kw)
        G.spec_tree_attention_fp4(h, **a)

    attend()
    for kw in (dict(scale=float("nan")), dict(scale=0.0), dict(scale=-1.0),
               dict(workspace=ws[:-256]), dict(workspace=ws[1:])):
        with pytest.raises(G.SpecError) as e:
            attend(**kw)
        assert e.value.code == G.SPEC_ERR_ARG
    with pytest.raises(ValueError):        # strided heads
        attend(q=torch.zeros(2, 3, 4, 128, dtype=torch.bfloat16, device=DEV)[..., ::2])
    with pytest.raises(ValueError):        # tokens that lie unevenly
        attend(k=torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16, device=DEV)[:, :3])
    with pytest.raises(G.SpecError) as e:
        attend(q=c.q.float(), k=c.tk.float(), v=c.tv.float(), out=out.float())
    assert e.value.code == G.SPEC_ERR_ARG
    assert G.load().spec_tree_attention_workspace(h.ptr, 2, 3, 4, 2, 96, None) == \
        G.SPEC_ERR_UNSUPPORTED
    for B, N, Hq, H in ((65, 3, 4, 2), (2, 65, 4, 2), (2, 0, 4, 2), (2, 3, 5, 2), (2, 3, 4, 0)):
        with pytest.raises(G.SpecError) as e:
            G.spec_tree_attention_workspace(h, B, N, Hq, H, 64)
        assert e.value.code == G.SPEC_ERR_ARG
    odd = G.Fp4Cache.empty(4, 16, 2, 64, DEV)
    odd.k = torch.zeros(odd.k.numel() + 1, dtype=torch.uint8, device=DEV)[1:].view(odd.k.shape)
    pos = gpu(np.zeros(2, np.int32))
    table = gpu(np.zeros((2, 1), np.int32))
    for call in (lambda: attend(cache=odd),
                 lambda: G.spec_kv_commit_fp4(h, c.tk, c.tv, odd, table, pos),
                 lambda: G.kv_load_fp4(h, odd, table, pos, pos, 3)):
        with pytest.raises(G.SpecError) as e:
            call()
        assert e.value.code == G.SPEC_ERR_ARG
    with pytest.raises(G.SpecError):       # a path needs its lengths
        G.spec_kv_commit_fp4(h, c.tk, c.tv, c.cache, table, pos,
                             kv_commit=gpu(np.zeros((2, 3), np.int32)))
    f = gpu(np.ones(32, np.float32))
    for kw in (dict(eps=-1.0), dict(eps=float("inf")), dict(style=2),
               dict(inv_freq=gpu(np.ones(33, np.float32))),
               dict(q_weight=c.q.new_ones(64))):
        a = dict(q=c.q, k=c.tk, inv_freq=f, seq_pos=pos)
        a.update(kw)
        with pytest.raises(G.SpecError) as e:
            G.qk_norm_rope(h, **a)
        assert e.value.code == G.SPEC_ERR_ARG
    torch.cuda.synchronize()


def test_empty_batch(h):
    z = torch.zeros((0, 3, 2, 64), dtype=torch.bfloat16, device=DEV)
    c = G.Fp4Cache.empty(4, 16, 2, 64, DEV)
    i = torch.zeros(0, dtype=torch.int32, device=DEV)
    t = torch.zeros((0, 2), dtype=torch.int32, device=DEV)
    G.spec_kv_commit_fp4(h, z, z, c, t, i)
    assert G.kv_load_fp4(h, c, t, i, i, 5)[0].shape == (0, 5, 2, 64)
    assert G.tree_attention_fp4(h, z, z, z, c, t, i, torch.zeros((0, 3), dtype=torch.int64,
                                                                 device=DEV), 1.0)[0].numel() == 0
    assert G.qk_norm_rope(h, z, z, None, i)[0].numel() == 0


# ---- all of it together --------------------------------------------------------------------------

def test_example_decodes_and_keeps_the_accepted_path():
    """examples/tree_step_fp4.py: every committed position holds the 4-bit form of the K of its
    token at that position (the example's K depends on nothing else), and nodes are accepted."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "tree_step_fp4.py")
    spec = importlib.util.spec_from_file_location("tree_step_fp4_example", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    r = ex.decode(steps=5, batch=3, nodes=20, seed=3)
    n = r["length"].cpu().numpy()
    assert sum(map(sum, r["accepted"])) > 0
    assert [len(t) - 1 for t in r["tokens"]] == n.tolist()
    m, most = r["model"], int(n.max())
    with G.Handle(3, 20, 4096, 0) as hh:
        got, _ = G.kv_load_fp4(hh, r["cache"], r["table"], gpu(np.zeros(3, np.int32)), r["length"],
                               most, torch.float32)
        tok = torch.zeros((3, most), dtype=torch.int64, device=DEV)
        for b in range(3):
            tok[b, :n[b]] = torch.tensor(r["tokens"][b][:n[b]])
        rows_ = m.emb[tok] @ m.qkv.T
        k = rows_[..., m.Hq * m.D:(m.Hq + m.Hkv) * m.D].unflatten(2, (-1, m.D)).contiguous()
        ref = S.norm_rope(k.double().cpu().numpy(), np.ones(m.D), 1e-6, m.inv_freq.cpu().numpy(),
                          np.tile(np.arange(most), (3, 1)), False)
    for b in range(3):
        x, y = got[b, :n[b]].double().cpu().numpy(), ref[b, :n[b]]
        amax = np.abs(y).reshape(y.shape[:-1] + (-1, 16)).max(-1).repeat(16, -1)
        # half of the widest step (2 of 6) under a scale within 2^-4 of amax / 6, cut at 6 of it,
        # and the projection's and the rows' own bf16 roundings
        assert np.all(np.abs(x - y) <= amax * (1 / 6 * (1 + 2.0 ** -4) + 2.0 ** -4 + 2.0 ** -5))


# ---- schedules and paths of the attention kernels ----------------------------------------------

@pytest.mark.parametrize("H", [1, 3, 7, 16])
@pytest.mark.parametrize("N,Gq,D", [(2, 2, 64), (20, 3, 128), (64, 3, 64)])
def test_attention_head_counts(h, H, N, Gq, D):
    """Heads that divide the CTAs into columns and heads that do not, for both kernels."""
    rng = np.random.default_rng(1000 * H + N)
    Case(rng, 2, N, H, Gq, D, "f16", S.NHD, 16, [700, 130]).check(h)


@pytest.mark.parametrize("pad", [0, 3, 8])
@pytest.mark.parametrize("layout,bs", [(S.NHD, 1), (S.NHD, 48), (S.HND, 7), (S.HND, 200)])
@pytest.mark.parametrize("dt,N", [("bf16", 40), ("f16", 64)])
def test_attention_many_rows_pages_and_strides(h, layout, bs, pad, dt, N):
    rng = np.random.default_rng(bs + 1000 * layout + pad + N)
    Case(rng, 2, N, 2, 3, 128, dt, layout, bs, [211, 150], pad=pad).check(h)


@pytest.mark.parametrize("N,Gq,D,dt", [(6, 4, 128, "bf16"), (40, 2, 64, "bf16"),
                                       (40, 2, 128, "f16"), (64, 4, 128, "bf16"),
                                       (64, 4, 64, "f16")])
def test_attention_bits_do_not_change(h, N, Gq, D, dt):
    """Many runs of one batch whose items are cut in many places: the same bits each time, whole
    batches of requests without a context among them."""
    rng = np.random.default_rng(117)
    ctx = [0, 1, 3000, 0] + [int(x) for x in rng.integers(0, 700, 36)]
    c = Case(rng, 40, N, 2, Gq, D, dt, S.NHD, 32, ctx)
    first, first_lse = c.check(h)
    for _ in range(10):
        out, lse = c.run(h)
        assert torch.equal(out, first) and torch.equal(lse, first_lse)


@pytest.mark.parametrize("N,Gq,D", [(1, 1, 256), (3, 4, 64), (8, 4, 128)])
def test_attention_few_items_of_many_parts(h, N, Gq, D):
    """One request over many CTAs: the parts of an item are joined by several threads a value."""
    rng = np.random.default_rng(118)
    Case(rng, 1, N, 2, Gq, D, "bf16", S.HND, 32, [6000], chain=True).check(h)


def test_attention_all_rows_finite_with_negative_and_large_scores(h):
    """Scores that rise along the context, so that the running maximum is followed again and
    again, and scores that fall, so that it is not."""
    rng = np.random.default_rng(119)
    for N, Gq in ((2, 4), (40, 2), (64, 4)):
        c = Case(rng, 2, N, 1, Gq, 64, "f16", S.HND, 16, [900, 901])
        # a key direction shared by all queries, growing (request 0) or shrinking (request 1)
        x = rng.standard_normal(c.codes[0].shape).astype(np.float32) * 0.1
        for b in range(2):
            for p in range(int(c.ctx[b])):
                blk, off = S.place(c.table, x.shape[0], 16, b, p)
                x[blk, :, off] += (p if b == 0 else 900 - p) * 0.01
        c.codes[0], c.sf[0] = S.quantise(x, 0.75)
        c.cache.k.copy_(gpu(S.pack(c.codes[0])))
        c.cache.k_sf.copy_(gpu(c.sf[0]))
        c.q.fill_(1.0)
        c.q64 = c.q.double().cpu().numpy()
        c.check(h)
