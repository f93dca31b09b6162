"""Work cases of the tree step over a 4-bit cache: what one pass of each operator computes, in
plain torch operations and through the library's entry points.

Operators (formulas in ``include/spec_verify.h``):
  rope    norm of every query and key head and the rotation by the tree position, in one pass;
  commit  K/V rows quantised into the paged 4-bit cache as they are written, then the written
          slots read back (a cache's codes are returned as the values they stand for);
  load    a stretch of the paged 4-bit cache read back into dense rows;
  attend  attention of a draft tree's nodes over a paged 4-bit context and the tree itself.

The 4-bit format: 16 consecutive elements of a head share one e4m3 scale, elements are e2m1
(two per byte, the even element in the low nibble), and one float32 scale covers a tensor.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LAYOUTS = {"NHD": 0, "HND": 1}
DEV = "cuda"
EPS = 1e-6


# ---- the cases -----------------------------------------------------------------------------

def listed():
    return [
        # a chain of five tokens from two small requests in float32: the smallest call
        dict(name="rope_chain_small", op="rope", B=2, N=5, Hq=4, Hkv=2, D=64, dtype="f32",
             rot=64, pairs=True, norm=True, strided=False, pos=1000),
        # a 32-node trie of eight requests, queries and keys still inside the fused projection
        dict(name="rope_trie", op="rope", B=8, N=32, Hq=32, Hkv=8, D=128, dtype="bf16",
             rot=128, pairs=False, norm=True, strided=True, pos=32768),
        # the full batch of large trees, far positions, a quarter of each head not rotated
        dict(name="rope_large_tree", op="rope", B=256, N=64, Hq=32, Hkv=8, D=128, dtype="bf16",
             rot=96, pairs=False, norm=True, strided=False, pos=1000000),
        # the accepted path of 64 short chains into the cache, after their verification
        dict(name="commit_chain", op="commit", B=64, N=6, Hkv=8, D=128, dtype="bf16",
             layout="NHD", bs=16, path=True, amax=5, strided=True),
        # the accepted paths of the full batch of large trees, 32 heads
        dict(name="commit_large_tree", op="commit", B=256, N=64, Hkv=32, D=128, dtype="bf16",
             layout="NHD", bs=16, path=True, amax=14, strided=False),
        # a prompt's K/V of a few requests written in one go, odd head size, HND pages
        dict(name="commit_prompt", op="commit", B=4, N=4097, Hkv=8, D=80, dtype="f16",
             layout="HND", bs=32, path=False, amax=0, strided=False),
        # a short context read back for a request that moves elsewhere
        dict(name="load_short", op="load", B=2, N=333, Hkv=4, D=64, dtype="f32", layout="HND",
             bs=16),
        # long contexts of a whole batch read back
        dict(name="load_long", op="load", B=16, N=16384, Hkv=8, D=128, dtype="bf16",
             layout="NHD", bs=16),
        # the chain of five over a short context: the smallest attention call
        dict(name="attend_chain_small", op="attend", B=2, N=5, Hq=8, Hkv=2, D=64, dtype="f16",
             layout="NHD", bs=16, ctx=1000, chain=True, strided=False),
        # one token of one request over a very long context (decoding without a draft)
        dict(name="attend_token_long", op="attend", B=1, N=1, Hq=32, Hkv=8, D=128,
             dtype="bf16", layout="HND", bs=32, ctx=262000, chain=True, strided=False),
        # 64 requests with chains of six, contexts of all lengths up to 12000
        dict(name="attend_chain", op="attend", B=64, N=6, Hq=32, Hkv=8, D=128, dtype="bf16",
             layout="NHD", bs=16, ctx=12000, chain=True, strided=True),
        # 64-node trees of 32 requests over contexts up to 8192: bound by the products
        dict(name="attend_large_tree", op="attend", B=32, N=64, Hq=32, Hkv=8, D=128,
             dtype="bf16", layout="HND", bs=16, ctx=8192, chain=False, strided=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "commit", "load", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    layout, bs = rng.choice(["NHD", "HND"]), rng.choice([8, 16, 32, 48, 64])
    hkv = rng.choice([1, 2, 4, 5, 8])
    if op == "rope":
        D = rng.choice([64, 80, 128, 256])
        B = _log(rng, 1, 256)
        N = min(_log(rng, 1, 2048), max(1, 16384 // B))
        return dict(op=op, B=B, N=N, Hq=hkv * rng.choice([1, 3, 4, 8]), Hkv=hkv, D=D,
                    dtype=dtype, rot=2 * rng.randint(D // 8, D // 2),
                    pairs=rng.random() < 0.3, norm=rng.random() < 0.8,
                    strided=rng.random() < 0.5, pos=_log(rng, 64, 1000000))
    if op == "commit":
        path = rng.random() < 0.6
        B = _log(rng, 1, 256) if path else _log(rng, 1, 16)
        N = rng.randint(1, 64) if path else _log(rng, 1, 4097)
        return dict(op=op, B=B, N=N, Hkv=rng.choice([1, 3, 8, 32]) if path else hkv,
                    D=rng.choice([64, 80, 128, 256]), dtype=dtype, layout=layout, bs=bs,
                    path=path, amax=rng.randint(0, min(N - 1, 14)) if path else 0,
                    strided=rng.random() < 0.5)
    if op == "load":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, N=_log(rng, 1, 200000 // B), Hkv=hkv,
                    D=rng.choice([64, 80, 128, 256]), dtype=dtype, layout=layout, bs=bs)
    D = rng.choice([64, 128, 128, 256])
    G = rng.choice([1, 2, 4, 7, 8])
    B = _log(rng, 1, 128)
    N = rng.choice([1, 2, rng.randint(3, 16), rng.randint(17, 64), 64])
    ctx = _log(rng, 1, 200000)
    ctx = max(1, min(ctx, 2000000 * 128 // (B * hkv * D), 500000000 // (B * hkv * G * N)))
    return dict(op=op, B=B, N=N, Hq=hkv * G, Hkv=hkv, D=D,
                dtype="bf16" if dtype == "f32" else dtype, layout=layout, bs=bs, ctx=ctx,
                chain=rng.random() < 0.4, strided=rng.random() < 0.5)


def _lengths(c):
    """Context lengths (attend), read-back lengths (load) of a batch: the first request has the
    longest, the others spread over a quarter to all of it, every thirteenth has none."""
    most = c["ctx"] if c["op"] == "attend" else c["N"]
    out = []
    for b in range(c["B"]):
        f = 1.0 if b == 0 else 0.25 + 0.75 * math.modf(b * 0.6180339887498949)[0]
        out.append(0 if b % 13 == 12 else max(1, int(most * f)))
    return out


def _accepted(c):
    """Tokens written for each request by a commit (accept_len + 1)."""
    return [(3 + 7 * b) % (c["amax"] + 1) + 1 if c["path"] else c["N"] for b in range(c["B"])]


def work(case):
    c, op = case, case["op"]
    e = 4 if c["dtype"] == "f32" else 2
    if op == "rope":
        rows = c["B"] * c["N"] * (c["Hq"] + c["Hkv"])
        flops = rows * c["D"] * (4 * c["norm"]) + rows * c["rot"] * 3
        return {"bytes": 2 * rows * c["D"] * e + 4 * c["B"] * (c["N"] + 1), "flops": flops}
    four = c["Hkv"] * (c["D"] // 2 + c["D"] // 16) * 2          # 4-bit K and V of a token
    wide = c["Hkv"] * c["D"] * e * 2
    if op == "commit":
        n = sum(_accepted(c))
        return {"bytes": n * (2 * wide + 2 * four), "flops": n * c["Hkv"] * c["D"] * 2 * 4}
    if op == "load":
        n = sum(_lengths(c))
        return {"bytes": n * four + c["B"] * c["N"] * wide, "flops": n * c["Hkv"] * c["D"] * 2}
    n = sum(_lengths(c))
    rows = c["B"] * c["N"]
    io = rows * (2 * c["Hq"] * c["D"] * e + wide + 4 * c["Hq"] + 8)
    return {"bytes": n * four + io,
            "flops": 4 * c["N"] * c["Hq"] * c["D"] * (n + c["B"] * (c["N"] + 1) // 2)}


# ---- inputs --------------------------------------------------------------------------------

def _rows(g, B, N, H, D, dtype, strided, std=1.0):
    """[B, N, H, D] rows: contiguous, or the middle columns of a wider projection output."""
    wide = H * D + (2 * D if strided else 0)
    x = torch.randn((B, N, wide), generator=g, device=DEV) * std
    x = x.to(DTYPES[dtype])
    return x[:, :, D:D + H * D].unflatten(2, (H, D)) if strided else x.view(B, N, H, D)


def _cache(c, g, table_len, tokens):
    """A paged 4-bit cache with K/V in all its pages, and a block table in random order."""
    B, H, D, bs = c["B"], c["Hkv"], c["D"], c["bs"]
    nb = B * table_len + 1
    shape = (nb, bs, H) if c["layout"] == "NHD" else (nb, H, bs)
    s = dict(k=torch.empty(shape + (D // 2,), dtype=torch.uint8, device=DEV),
             k_sf=torch.empty(shape + (D // 16,), dtype=torch.uint8, device=DEV))
    s["v"], s["v_sf"] = torch.empty_like(s["k"]), torch.empty_like(s["k_sf"])
    s["k_scale"] = torch.tensor([0.75], device=DEV)
    s["v_scale"] = torch.tensor([0.0625], device=DEV)
    step = max(1, (1 << 26) // (bs * H * D))
    for at in range(0, nb if tokens else 0, step):
        n = min(step, nb - at)
        for key, std in (("k", 1.0), ("v", 0.5)):
            # heads have channels of unequal size, as keys have
            x = torch.randn((n,) + shape[1:] + (D,), generator=g, device=DEV) * std
            x *= 0.5 + 2.0 * torch.rand((D,), generator=g, device=DEV) ** 4
            s[key][at:at + n], s[key + "_sf"][at:at + n] = _quantise(x, s[key + "_scale"])
    if not tokens:
        for key in ("k", "v", "k_sf", "v_sf"):
            s[key].zero_()
    pages = torch.randperm(nb, generator=g, device=DEV)
    s["table"], s["spare"] = pages[1:].reshape(B, table_len).int().contiguous(), pages[0]
    return s


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) % (1 << 62))
    rng = np.random.default_rng(int(seed) % (1 << 62))
    B, N, D, op = c["B"], c["N"], c["D"], c["op"]
    s = {"case": c}
    if op in ("rope", "attend"):
        chain = c.get("chain", N > 64)
        parent = np.full((B, N), -1, np.int64)
        for i in range(1, N):
            parent[:, i] = i - 1 if chain else rng.integers(max(0, i - 12), i, B)
        depth, mask, each = np.zeros((B, N), np.int32), np.zeros((B, N), np.uint64), np.arange(B)
        for i in range(N):
            up = parent[:, i]
            depth[:, i] = depth[each, up] + 1 if i else 0
            if N <= 64:
                mask[:, i] = (mask[each, up] if i else 0) | np.uint64(1 << i)
        s["depth"] = torch.from_numpy(depth).to(DEV)
        s["mask"] = torch.from_numpy(mask.view(np.int64)).to(DEV)
    if op == "rope":
        s["q"] = _rows(g, B, N, c["Hq"], D, c["dtype"], c["strided"])
        s["k"] = _rows(g, B, N, c["Hkv"], D, c["dtype"], c["strided"])
        s["qw"] = s["kw"] = None
        if c["norm"]:
            s["qw"], s["kw"] = ((torch.rand(D, generator=g, device=DEV) + 0.5).to(
                DTYPES[c["dtype"]]) for _ in range(2))
        s["inv_freq"] = (1e6 ** (-torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64) /
                                 (c["rot"] // 2))).float()
        s["seq_pos"] = torch.randint(0, c["pos"], (B,), generator=g, device=DEV).int()
    elif op == "commit":
        table_len = (N + c["bs"] - 1) // c["bs"] + 2
        s.update(_cache(c, g, table_len, False))
        s["src_k"] = _rows(g, B, N, c["Hkv"], D, c["dtype"], c["strided"])
        s["src_v"] = _rows(g, B, N, c["Hkv"], D, c["dtype"], c["strided"], 0.5)
        s["seq_pos"] = torch.randint(0, c["bs"], (B,), generator=g, device=DEV).int()
        cnt = _accepted(c)
        s["count"] = torch.tensor(cnt, dtype=torch.int32, device=DEV)
        s["most"] = max(cnt)
        s["kv_commit"] = s["accept_len"] = None
        if c["path"]:
            kv = np.full((B, N), -1, np.int32)
            for b in range(B):
                kv[b, 1:cnt[b]] = 1 + np.sort(rng.permutation(N - 1)[:cnt[b] - 1])
            kv[:, 0] = 0
            s["kv_commit"] = torch.from_numpy(kv).to(DEV)
            s["accept_len"] = s["count"] - 1
    elif op == "load":
        s.update(_cache(c, g, (N + c["bs"] - 1) // c["bs"] + 1, True))
        s["start"] = torch.randint(0, c["bs"], (B,), generator=g, device=DEV).int()
        s["count"] = torch.tensor(_lengths(c), dtype=torch.int32, device=DEV)
    else:
        s.update(_cache(c, g, (c["ctx"] + N + c["bs"] - 1) // c["bs"], True))
        s["q"] = _rows(g, B, N, c["Hq"], D, c["dtype"], c["strided"], 1.5)
        s["tk"] = _rows(g, B, N, c["Hkv"], D, c["dtype"], c["strided"])
        s["tv"] = _rows(g, B, N, c["Hkv"], D, c["dtype"], c["strided"], 0.5)
        s["ctx_len"] = torch.tensor(_lengths(c), dtype=torch.int32, device=DEV)
    return s


# ---- the operators in plain torch operations -------------------------------------------------

def _quantise(x, scale):
    """float32 [..., D] -> (codes uint8 [..., D/2], block scales uint8 [..., D/16])."""
    blocks = x.float().unflatten(-1, (-1, 16))
    inv = 1.0 / scale
    amax = blocks.abs().amax(-1, keepdim=True)
    sixth = inv * torch.full_like(inv, 1.0 / 6.0)
    sf = (amax * sixth).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = sf.float()
    mul = torch.where(f > 0, (1.0 / f) * inv, torch.zeros_like(f))
    y = blocks * mul
    a = y.abs()
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) +
            (a > 5.0) + (y < 0).byte() * 8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), sf.view(torch.uint8).squeeze(-1)


def _values(codes, sf, scale):
    """codes [..., D/2] and block scales [..., D/16] -> float32 [..., D]."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    mag = (n & 7).float()
    mag = torch.where(mag < 4, mag * 0.5, torch.where(mag < 6, mag - 2, 2 * mag - 8))
    v = torch.where(n >= 8, -mag, mag).unflatten(-1, (-1, 16))
    return (v * sf.view(torch.float8_e4m3fn).float().unsqueeze(-1) * scale).flatten(-2)


def _slots(s, pos):
    """(block, offset) index pairs of positions [B, L] through the block table."""
    bs = s["case"]["bs"]
    blk = torch.gather(s["table"], 1, (pos // bs).clamp(0, s["table"].shape[1] - 1)).long()
    return blk, pos % bs


def _at(s, t, blk, off):
    return t[blk, off] if s["case"]["layout"] == "NHD" else t[blk, :, off]


def _read(s, key, pos):
    blk, off = _slots(s, pos)
    return _values(_at(s, s[key], blk, off), _at(s, s[key + "_sf"], blk, off), s[key + "_scale"])


def _plain_rope(s):
    c = s["case"]
    half = c["rot"] // 2
    pos = s["seq_pos"].double().unsqueeze(1) + s["depth"]
    ang = (pos.unsqueeze(-1) * s["inv_freq"].double()).unsqueeze(2)
    cos, sin = ang.cos().float(), ang.sin().float()

    def one(x, w):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
        r, rest = y[..., :c["rot"]], y[..., c["rot"]:]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["pairs"] else (r[..., :half], r[..., half:])
        a, b = a * cos - b * sin, b * cos + a * sin
        r = torch.stack((a, b), -1).flatten(-2) if c["pairs"] else torch.cat((a, b), -1)
        return torch.cat((r, rest), -1).to(x.dtype)

    return one(s["q"], s["qw"]), one(s["k"], s["kw"])


def _plain_commit(s):
    c = s["case"]
    j = torch.arange(s["most"], device=DEV).unsqueeze(0).expand(c["B"], -1)
    live = j < s["count"].unsqueeze(1)
    node = s["kv_commit"][:, :s["most"]].long().clamp(min=0) if c["path"] else j
    blk, off = _slots(s, s["seq_pos"].long().unsqueeze(1) + j)
    blk = torch.where(live, blk, s["spare"])            # nobody's page takes what is not kept
    for key in ("k", "v"):
        src = s["src_" + key]
        codes, sf = _quantise(src[torch.arange(c["B"], device=DEV).unsqueeze(1), node],
                              s[key + "_scale"])
        for name, val in ((key, codes), (key + "_sf", sf)):
            if c["layout"] == "NHD":
                s[name][blk, off] = val
            else:
                s[name][blk, :, off] = val
    return _plain_load(s, s["seq_pos"], s["most"])


def _plain_load(s, start, n):
    i = torch.arange(n, device=DEV).unsqueeze(0)
    live = (i < s["count"].unsqueeze(1)).unsqueeze(-1).unsqueeze(-1)
    pos = start.long().unsqueeze(1) + i
    return tuple(torch.where(live, _read(s, key, pos), 0.0).to(DTYPES[s["case"]["dtype"]])
                 for key in ("k", "v"))


def _plain_attend(s):
    c = s["case"]
    B, N, H, G, D = c["B"], c["N"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    pos = torch.arange(c["ctx"], device=DEV).unsqueeze(0).expand(B, -1)
    k = torch.cat((_read(s, "k", pos), s["tk"].float()), 1).permute(0, 2, 3, 1)   # [B,H,D,L]
    q = s["q"].float().unflatten(2, (H, G)).permute(0, 2, 1, 3, 4).reshape(B, H, N * G, D)
    z = torch.matmul(q * D ** -0.5, k).unflatten(2, (N, G))                       # [B,H,N,G,L]
    del k
    seen = (pos < s["ctx_len"].unsqueeze(1)).unsqueeze(1).expand(-1, N, -1)
    tree = (s["mask"].unsqueeze(-1) >> torch.arange(N, device=DEV)) & 1
    seen = torch.cat((seen, tree.bool()), -1).unsqueeze(2).unsqueeze(1)           # [B,1,N,1,L]
    z = torch.where(seen, z, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(z - m), 0.0)
    del z
    total = p.sum(-1, keepdim=True)
    v = torch.cat((_read(s, "v", pos), s["tv"].float()), 1).permute(0, 2, 1, 3)   # [B,H,L,D]
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (N, G))
    o = torch.where(total > 0, o / total, 0.0)
    lse = torch.where(total > 0, m + total.log(), -math.inf).squeeze(-1)
    return (o.permute(0, 2, 1, 3, 4).reshape(B, N, c["Hq"], D).to(DTYPES[c["dtype"]]),
            lse.permute(0, 2, 1, 3).reshape(B, N, c["Hq"]).contiguous())


# ---- one pass ------------------------------------------------------------------------------

_kept = {}


def _handle():
    """The library handle that a program keeps for its process."""
    if "h" not in _kept:
        from speculative_decoding_tree_mask_gb300 import binding as G
        _kept["G"], _kept["h"] = G, G.Handle(256, 64, 4096, torch.cuda.current_device())
    return _kept["G"], _kept["h"]


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "rope":
            return _plain_rope(s)
        if op == "commit":
            return _plain_commit(s)
        return _plain_load(s, s["start"], c["N"]) if op == "load" else _plain_attend(s)
    G, h = _handle()
    if op == "rope":
        return G.qk_norm_rope(h, s["q"], s["k"], s["inv_freq"], s["seq_pos"], s["depth"],
                              q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                              style=G.SPEC_ROPE_PAIRS if c["pairs"] else G.SPEC_ROPE_HALVES)
    cache = G.Fp4Cache(s["k"], s["v"], s["k_sf"], s["v_sf"], LAYOUTS[c["layout"]],
                       s["k_scale"], s["v_scale"])
    if op == "commit":
        G.spec_kv_commit_fp4(h, s["src_k"], s["src_v"], cache, s["table"], s["seq_pos"],
                             kv_commit=s["kv_commit"], accept_len=s["accept_len"])
        return G.kv_load_fp4(h, cache, s["table"], s["seq_pos"], s["count"], s["most"],
                             DTYPES[c["dtype"]])
    if op == "load":
        return G.kv_load_fp4(h, cache, s["table"], s["start"], s["count"], c["N"],
                             DTYPES[c["dtype"]])
    return G.tree_attention_fp4(h, s["q"], s["tk"], s["tv"], cache, s["table"], s["ctx_len"],
                                s["mask"], scale=c["D"] ** -0.5)


# ---- the definitions in 64 bits --------------------------------------------------------------

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _e4m3_table():
    code = np.arange(128)
    e, m = code >> 3, code & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v[127] = np.nan
    return np.concatenate((v, -v))


def _exact_read(s, key, b, lo, hi):
    """The float64 values of positions lo..hi-1 of request b, [n, H, D]."""
    bs, D = s["case"]["bs"], s["case"]["D"]
    e2m1 = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=DEV)
    e4m3 = torch.from_numpy(_e4m3_table()).to(DEV)
    pos = torch.arange(lo, hi, device=DEV)
    page = s["table"][b].long()[pos // bs]
    codes, sf = _at(s, s[key], page, pos % bs).long(), _at(s, s[key + "_sf"], page, pos % bs)
    v = torch.empty(codes.shape[:-1] + (D,), dtype=torch.float64, device=DEV)
    v[..., 0::2], v[..., 1::2] = e2m1[codes % 16], e2m1[codes // 16]
    return v * e4m3[sf.long()].repeat_interleave(16, -1) * s[key + "_scale"].double()


def _exact_quantised(x, scale):
    """What x [n, H, D] stands for once stored: the block scale is the e4m3 nearest to
    amax * r6 and a value the e2m1 nearest to x * r (ties to the even code), the factors
    rounded to float32 as the format's definition says."""
    f32 = np.float32
    x = x.double().cpu().numpy().reshape(-1, 16)
    inv = f32(1) / f32(float(scale))
    amax = np.abs(x).max(-1)
    want = np.minimum((amax * np.float64(inv * f32(1.0 / 6.0))).astype(f32).astype(np.float64), 448)
    grid = _e4m3_table()[:127]
    hi = np.searchsorted(grid, want).clip(1, 126)
    lo = hi - 1
    near = want - grid[lo], grid[hi] - want
    pick = np.where((near[0] < near[1]) | ((near[0] == near[1]) & (lo % 2 == 0)), lo, hi)
    sf = grid[pick]
    with np.errstate(divide="ignore"):
        r = np.where(sf > 0, (f32(1) / sf.astype(f32)).astype(f32) * inv, f32(0)).astype(f32)
    y = (x * r.astype(np.float64)[:, None]).astype(f32).astype(np.float64)
    a, grid = np.abs(y).clip(max=6.0), np.array(E2M1)
    hi = np.searchsorted(grid, a).clip(1, 7)
    lo = hi - 1
    near = a - grid[lo], grid[hi] - a
    pick = np.where((near[0] < near[1]) | ((near[0] == near[1]) & (lo % 2 == 0)), lo, hi)
    return np.where(y < 0, -grid[pick], grid[pick]) * sf[:, None] * float(scale)


def _exact_rope(s):
    c = s["case"]
    pos = s["seq_pos"].cpu().numpy().astype(np.float64)[:, None] + s["depth"].cpu().numpy()
    turn = pos[..., None] * s["inv_freq"].cpu().numpy().astype(np.float64)
    turn = torch.from_numpy(np.exp(1j * turn)).to(DEV).unsqueeze(2)
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt(torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / c["D"] +
                               EPS) * w.double()
        n, half = c["rot"], c["rot"] // 2
        first = torch.arange(0, n, 2) if c["pairs"] else torch.arange(half)
        second = first + (1 if c["pairs"] else half)
        z = torch.complex(y[..., first], y[..., second]) * turn
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    return tuple(out)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op, B, N, D = c["op"], c["B"], c["N"], c["D"]
    if op == "rope":
        return _exact_rope(s)
    H = c["Hkv"]
    if op == "commit":
        cnt = _accepted(c)
        out = [np.zeros((B, s["most"], H, D)) for _ in range(2)]
        kv = s["kv_commit"].cpu() if c["path"] else None
        for b in range(B):
            node = kv[b, :cnt[b]].long() if c["path"] else torch.arange(cnt[b])
            for o, key in zip(out, ("k", "v")):
                x = s["src_" + key][b, node.to(DEV)]
                o[b, :cnt[b]] = _exact_quantised(x, s[key + "_scale"]).reshape(cnt[b], H, D)
        return tuple(out)
    if op == "load":
        out = [torch.zeros((B, N, H, D), dtype=torch.float64, device=DEV) for _ in range(2)]
        lo = s["start"].tolist()
        for b, n in enumerate(_lengths(c)):
            for o, key in zip(out, ("k", "v")):
                o[b, :n] = _exact_read(s, key, b, lo[b], lo[b] + n)
        return tuple(out)
    G = c["Hq"] // H
    out = torch.zeros((B, N, c["Hq"], D), dtype=torch.float64, device=DEV)
    lse = torch.full((B, N, c["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    bits = torch.arange(N, device=DEV)
    for b, n in enumerate(_lengths(c)):
        k = torch.cat((_exact_read(s, "k", b, 0, n), s["tk"][b].double()))
        v = torch.cat((_exact_read(s, "v", b, 0, n), s["tv"][b].double()))
        tree = ((s["mask"][b].unsqueeze(1) >> bits) & 1).bool()
        hide = torch.zeros((N, n + N), dtype=torch.float64, device=DEV)
        hide[:, n:].masked_fill_(~tree, -math.inf)
        for h in range(H):
            q = s["q"][b, :, h * G:(h + 1) * G].double()
            z = torch.einsum("ngd,ld->ngl", q, k[:, h]) / math.sqrt(D) + hide.unsqueeze(1)
            lse[b, :, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
            out[b, :, h * G:(h + 1) * G] = torch.einsum("ngl,ld->ngd", torch.softmax(z, -1),
                                                        v[:, h])
    return out, lse
