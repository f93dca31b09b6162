"""New tokens into the paged cache against the float64 oracle (needs a GB300).

Tolerances as for the head norm and rotation (test_gpu_tree_step): one rounding to the output type
is half a step, before it float32 arithmetic within 2^-19 (|a| + |c|) for a pair. Values of V are
bit for bit what they were, or, in 8 bits, the nearest code of RN(x / scale).
"""
import numpy as np
import pytest
import torch

from oracle import kv_commit as KV
from oracle import paged_step as S
from speculative_decoding_tree_mask_gb300 import binding as G

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TDT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16,
       "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
# half a step relative to the value, and of the subnormals
HALF = {"e4m3": (2.0 ** -4, 2.0 ** -10, 448.0), "e5m2": (2.0 ** -3, 2.0 ** -17, 57344.0)}


@pytest.fixture(scope="module")
def h():
    G.load()
    with G.Handle(2048, 64, 1 << 10, 0) as handle:
        yield handle


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def rows(rng, T, H, D, dt, pad=0, std=1.0):
    x = torch.from_numpy((rng.standard_normal((T, H * D + 2 * pad)) * std).astype(np.float32))
    t = x.to(TDT[dt]).to(DEV)
    t = t[:, pad:pad + H * D].unflatten(1, (H, D)) if pad else t.view(T, H, D)
    return t, t.double().cpu().numpy()


def values(t, kind):
    """A cache's values in float64, over the tensor scale."""
    t = t.cpu()
    return S.fp8_values(t.view(torch.uint8).numpy(), kind == "e4m3") if kind in HALF else \
        t.double().numpy()


def turned(x, w, eps, f, where, pairs):
    """(result, size of what each element was made from) of rows x [T, H, D]."""
    w64 = None if w is None else w.double().cpu().numpy()
    ref = S.norm_rope(x, w64, eps, f, where, pairs)
    size = np.abs(S.norm_rope(x, w64, eps, f[:0], where, pairs))
    a = np.arange(len(f)) * (2 if pairs else 1)
    c = a + (1 if pairs else len(f))
    size[..., a] = size[..., c] = size[..., a] + size[..., c]
    return ref, size


@pytest.mark.parametrize("dt,kind", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"),
                                     ("bf16", "e4m3"), ("f16", "e5m2"), ("f32", "e4m3")])
@pytest.mark.parametrize("D,rot,pairs,norm,pad,layout,bs", [
    (128, 128, False, True, 0, S.NHD, 16), (64, 64, True, False, 8, S.HND, 8),
    (80, 42, False, True, 16, S.NHD, 5), (256, 90, False, False, 0, S.HND, 48),
    (16, 16, True, True, 3, S.NHD, 1), (128, 0, False, True, 0, S.HND, 64),
    (96, 96, False, False, 4, S.NHD, 32)])
def test_append(h, dt, kind, D, rot, pairs, norm, pad, layout, bs):
    rng = np.random.default_rng(D + rot + bs)
    counts, pos = [1, 0, 7, 70, 1], [0, 3, bs - 1, 2 * bs + 1, 50]
    B, T, Hq, H = 5, sum(counts), 6, 3
    scale = 0.25 if kind in HALF else 1.0
    q, q64 = rows(rng, T, Hq, D, dt, pad, 2.0)
    k, k64 = rows(rng, T, H, D, dt, pad)
    v, v64 = rows(rng, T, H, D, dt, pad)
    q0 = q.clone()
    f = (10000.0 ** -(np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    w = [torch.from_numpy(rng.uniform(0.5, 2, D).astype(np.float32)).to(TDT[dt]).to(DEV)
         if norm else None for _ in range(2)]
    width = max((p + n + bs - 1) // bs for p, n in zip(pos, counts))
    nb = B * width + 2
    table = rng.permutation(nb)[:B * width].reshape(B, width).astype(np.int32)
    shape = (nb, bs, H, D) if layout == S.NHD else (nb, H, bs, D)
    both = torch.zeros((nb, 2) + shape[1:], device=DEV).to(TDT[kind])      # interleaved blocks
    sc = [torch.tensor([scale], device=DEV) if kind in HALF else None] * 2
    cache = G.KvCache(both[:, 0], both[:, 1], layout, *sc)
    start = np.cumsum([0] + counts).astype(np.int32)
    st = torch.full((B,), 9, dtype=torch.int32, device=DEV)
    args = (cache, gpu(table), gpu(np.array(pos, np.int32)), gpu(start))
    style = G.SPEC_ROPE_PAIRS if pairs else G.SPEC_ROPE_HALVES
    inv = gpu(f) if rot else None
    qo = G.kv_append(h, q, k, v, *args, inv, *w, 1e-5, style, status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [0] * B and torch.equal(q, q0)
    where = np.concatenate([p + np.arange(n) for p, n in zip(pos, counts)])
    ref, size = turned(q64, w[0], 1e-5, f, where, pairs)
    tol = torch.finfo(TDT[dt]).eps / 2 * np.abs(ref) + 2.0 ** -19 * size
    tol += 2.0 ** -25 if dt == "f16" else 0.0
    assert np.all(np.abs(qo.double().cpu().numpy() - ref) <= tol)
    ref, size = turned(k64, w[1], 1e-5, f, where, pairs)
    got_k, got_v = values(both[:, 0], kind), values(both[:, 1], kind)
    touched = np.zeros(shape, bool)
    row = 0
    for b, n in enumerate(counts):
        for i in range(n):
            blk, off = table[b, (pos[b] + i) // bs], (pos[b] + i) % bs
            at = (blk, off) if layout == S.NHD else (blk, slice(None), off)
            touched[at] = True
            if kind in HALF:
                rel, sub, most = HALF[kind]
                x = np.clip(ref[row] / scale, -most, most)
                t = rel * np.abs(x) + sub + 2.0 ** -19 * size[row] / scale
                assert np.all(np.abs(got_k[at] - x) <= t)
                code = KV.fp8_encode((v64[row].astype(np.float32) / np.float32(scale)).astype(
                    np.float32), KV.FP8_E4M3 if kind == "e4m3" else KV.FP8_E5M2)
                assert np.array_equal(got_v[at].ravel(), S.fp8_values(code, kind == "e4m3"))
            else:
                t = torch.finfo(TDT[dt]).eps / 2 * np.abs(ref[row]) + 2.0 ** -19 * size[row]
                t += 2.0 ** -25 if dt == "f16" else 0.0
                assert np.all(np.abs(got_k[at] - ref[row]) <= t)
                assert np.array_equal(got_v[at], v64[row])
            row += 1
    assert np.all(got_k[~touched] == 0) and np.all(got_v[~touched] == 0)
    # in place, and the keys and values alone
    one, two = both.clone(), torch.zeros_like(both)
    cache = G.KvCache(two[:, 0], two[:, 1], layout, *sc)
    G.spec_kv_append(h, q, k, v, cache, *args[1:3], q, args[3], inv, *w, 1e-5, style)
    assert torch.equal(q, qo) and torch.equal(one.view(torch.uint8), two.view(torch.uint8))
    two.view(torch.uint8).zero_()
    assert G.kv_append(h, None, k, v, cache, *args[1:], inv, None, w[1], 1e-5, style) is None
    assert torch.equal(one.view(torch.uint8), two.view(torch.uint8))


def test_same_as_head_norm_and_rotation(h):
    """A prompt's rows are what spec_qk_norm_rope makes of them, bit for bit."""
    rng = np.random.default_rng(3)
    B, N, Hq, H, D = 3, 40, 8, 2, 128
    q, _ = rows(rng, B * N, Hq, D, "bf16")
    k, _ = rows(rng, B * N, H, D, "bf16")
    w = torch.rand(D, device=DEV).to(torch.bfloat16)
    f = (1e6 ** (-torch.arange(64, device=DEV) / 64)).float()
    pos = gpu(np.array([0, 5, 1000], np.int32))
    qo, ko = G.qk_norm_rope(h, q.view(B, N, Hq, D), k.view(B, N, H, D), f, pos, None, w, w)
    cache = G.KvCache.empty(B * 70, 16, H, D, torch.bfloat16, DEV)
    table = gpu(np.arange(B * 70, dtype=np.int32).reshape(B, 70))
    got = G.kv_append(h, q, k, k, cache, table, pos, None, f, w, w)
    assert torch.equal(got.view(B, N, Hq, D), qo)
    flat = cache.k.view(B, 70 * 16, H, D)
    for b, p in enumerate([0, 5, 1000]):
        assert torch.equal(flat[b, p:p + N], ko[b])


def test_places_that_are_not_there(h):
    """Blocks outside the cache and positions outside the table are skipped and reported, queries
    written all the same; rows of no request stay."""
    rng = np.random.default_rng(4)
    counts, pos = [3, 4, 2, 5, 1], [0, -2, 63, 14, 2 ** 31 - 1]
    start = np.array([0, 3, 7, 9, 14, 15], np.int32)
    T, B = 18, 5
    q, _ = rows(rng, T, 2, 64, "f16")
    k, k64 = rows(rng, T, 1, 64, "f16")
    table = np.arange(B * 4, dtype=np.int32).reshape(B, 4)
    table[0, 0], table[3, 1] = -1, 99
    cache = G.KvCache.empty(B * 4, 16, 1, 64, torch.float16, DEV)
    st = torch.full((B,), 9, dtype=torch.int32, device=DEV)
    qo = torch.full_like(q, 7.0)
    call = (q, k, k, cache, gpu(table), gpu(np.array(pos, np.int32)), qo)
    G.spec_kv_append(h, *call, gpu(start), status=st)
    assert st.tolist() == [S.BAD_SLOT] * 5
    assert torch.equal(qo[:15], q[:15]) and (qo[15:] == 7).all()
    want = np.zeros((B * 4 * 16, 64))
    row = 0
    for b, n in enumerate(counts):
        for i in range(n):
            p = pos[b] + i
            if 0 <= p < 64 and 0 <= table[b, p // 16] < B * 4:
                want[table[b, p // 16] * 16 + p % 16] = k64[row, 0]
            row += 1
    assert np.array_equal(cache.k.view(-1, 64).double().cpu().numpy(), want)
    qo.fill_(7.0)
    G.spec_kv_append(h, *call, gpu(np.array([0, 3, 2, 9, 14, 19], np.int32)), status=st)
    assert st.tolist() == [S.BAD_SLOT, S.BAD_RANGE, S.BAD_SLOT, S.BAD_SLOT, S.BAD_RANGE]
    assert (qo[14:] == 7).all()


@pytest.mark.parametrize("B", [1, 33, 1025, 2048])
def test_rows_find_their_request(h, B):
    """Many requests of no, one and a few rows."""
    rng = np.random.default_rng(B)
    counts = rng.choice([0, 0, 1, 1, 2, 5], B)
    counts[-1] = 1
    start = np.cumsum([0] + list(counts)).astype(np.int32)
    T = int(start[-1])
    k, _ = rows(rng, T, 1, 64, "bf16")
    cache = G.KvCache.empty(B, 8, 1, 64, torch.bfloat16, DEV)
    G.kv_append(h, None, k, k, cache, gpu(np.arange(B, dtype=np.int32)[:, None]),
                gpu(np.full(B, 2, np.int32)), gpu(start))
    owner = np.repeat(np.arange(B), counts)
    place = np.arange(T) - start[owner]
    assert torch.equal(cache.k[gpu(owner), gpu(place + 2)], k)
    assert float(cache.k.abs().sum(dtype=torch.float64)) == float(k.abs().sum(dtype=torch.float64))


@pytest.mark.parametrize("kw", [dict(rot=130), dict(rot=3), dict(eps=-1.0), dict(style=2),
                                dict(w="q"), dict(T=5), dict(D=12), dict(B=2049)])
def test_library_refusals(h, kw):
    B, D = kw.get("B", 2), kw.get("D", 128)
    T = kw.get("T", 2 * B)
    x = torch.zeros((T, 2, D), dtype=torch.bfloat16, device=DEV)
    cache = G.KvCache.empty(4, 16, 2, D, torch.bfloat16, DEV)
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(G.SpecError):
        G.spec_kv_append(h, x, x, x, cache, torch.zeros((B, 4), dtype=torch.int32, device=DEV),
                         torch.zeros(B, dtype=torch.int32, device=DEV), x, None,
                         torch.zeros(kw.get("rot", 64) // 2 + kw.get("rot", 64) % 2 * 64, device=DEV),
                         w if kw.get("w") else None, None, kw.get("eps", 1e-6), kw.get("style", 0))
    torch.cuda.synchronize()
