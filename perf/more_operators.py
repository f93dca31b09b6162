"""Work cases of the paged step over a 16-bit or 8-bit cache and of the scores of what it answers:
what one pass of each operator computes, in plain torch operations and through the library's entry
points.

Operators (formulas in ``include/spec_verify.h``):
  append    queries and keys of new tokens normalised and rotated, keys and values written into
            the paged cache on the way;
  attend    attention of each request's new tokens (one, a draft chain, a prompt's chunk) over its
            paged cache, causal, with a sliding window and first tokens that stay visible if asked;
  logprobs  log probabilities of given tokens, entropy and the likeliest tokens of logits rows.

The new tokens of a batch are rows [T, heads, D]; rows row_start[b] .. row_start[b + 1] - 1 are
request b's, at positions seq_pos[b] and on.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
          "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LAYOUTS = {"NHD": 0, "HND": 1}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1, "e5m2": 1}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
DEV = "cuda"
EPS = 1e-6


# ---- the cases -----------------------------------------------------------------------------

def listed():
    return [
        # one decoding step of 16 requests: the smallest call
        dict(name="append_token", op="append", B=16, N=1, chunks=0, Hq=32, Hkv=8, D=128,
             dtype="bf16", cache="bf16", layout="NHD", bs=16, rot=128, pairs=False, norm=False,
             strided=True, pos=32768),
        # a few prompts of all lengths, head norms, the fused projection's columns
        dict(name="append_prompt", op="append", B=6, N=8192, chunks=6, Hq=32, Hkv=8, D=128,
             dtype="bf16", cache="bf16", layout="HND", bs=32, rot=128, pairs=False, norm=True,
             strided=True, pos=4096),
        # chunks of prompts between decoding requests, into an 8-bit cache; odd head size
        dict(name="append_mixed_8bit", op="append", B=64, N=1024, chunks=3, Hq=20, Hkv=5, D=80,
             dtype="f16", cache="e4m3", layout="NHD", bs=16, rot=64, pairs=True, norm=False,
             strided=False, pos=100000),
        # draft chains of five of four requests over short contexts: the smallest attention call
        dict(name="attend_chain_small", op="attend", B=4, N=5, chunks=4, Hq=8, Hkv=2, D=64,
             dtype="f16", cache="f16", layout="NHD", bs=16, ctx=700, window=0, sinks=0,
             strided=False),
        # a decoding step of 128 requests, contexts of all lengths up to 8192
        dict(name="attend_token", op="attend", B=128, N=1, chunks=0, Hq=32, Hkv=8, D=128,
             dtype="bf16", cache="bf16", layout="NHD", bs=16, ctx=8192, window=0, sinks=0,
             strided=True),
        # one token of one request over a very long 8-bit cache
        dict(name="attend_token_long_8bit", op="attend", B=1, N=1, chunks=0, Hq=64, Hkv=8, D=128,
             dtype="bf16", cache="e4m3", layout="HND", bs=64, ctx=500000, window=0, sinks=0,
             strided=False),
        # two prompts from their first token on: bound by the products
        dict(name="attend_prompt", op="attend", B=2, N=8192, chunks=2, Hq=32, Hkv=8, D=128,
             dtype="bf16", cache="bf16", layout="NHD", bs=16, ctx=0, window=0, sinks=0,
             strided=True),
        # a chunk of a long prompt, window of 4096 positions, four first tokens kept
        dict(name="attend_window", op="attend", B=2, N=2000, chunks=2, Hq=32, Hkv=4, D=128,
             dtype="f16", cache="f16", layout="HND", bs=32, ctx=50000, window=4096, sinks=4,
             strided=False),
        # prompt chunks of two requests in a batch of decoding ones
        dict(name="attend_mixed", op="attend", B=24, N=512, chunks=2, Hq=32, Hkv=8, D=64,
             dtype="bf16", cache="bf16", layout="HND", bs=16, ctx=12000, window=0, sinks=0,
             strided=False),
        # the answer's tokens of eight small requests, float32 rows of an odd vocabulary
        dict(name="logprobs_small", op="logprobs", B=8, N=6, P=4, V=50257, dtype="f32", C=1, K=5,
             temp=0.7, path=True),
        # the accepted paths of the full batch of large trees
        dict(name="logprobs_path", op="logprobs", B=256, N=64, P=12, V=152064, dtype="bf16", C=1,
             K=20, temp=1.0, path=True),
        # every token of a prompt
        dict(name="logprobs_prompt", op="logprobs", B=1, N=4096, P=4096, V=152064, dtype="bf16",
             C=1, K=8, temp=1.0, path=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "logprobs"])
    if op == "logprobs":
        V = _log(rng, 1000, 200000)
        path = rng.random() < 0.5
        if path:
            B, N = _log(rng, 1, 256), rng.randint(1, 64)
            N = max(1, min(N, 2500000000 // (B * V)))
            P = rng.randint(1, N)
        else:
            B = _log(rng, 1, 16)
            N = P = max(1, min(_log(rng, 1, 8192), 600000000 // (B * V)))
        return dict(op=op, B=B, N=N, P=P, V=V, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    C=rng.choice([1, 1, 1, 4, 17]), K=rng.choice([0, 1, 5, 8, 20, 32]),
                    temp=rng.choice([1.0, 1.0, 0.6, 1.7]), path=path)
    layout, bs = rng.choice(["NHD", "HND"]), rng.choice([8, 16, 16, 32, 48, 64, 128])
    hkv = rng.choice([1, 2, 4, 5, 8])
    strided = rng.random() < 0.5
    if op == "append":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        D = rng.choice([64, 80, 128, 128, 256])
        B = _log(rng, 1, 256)
        G = rng.choice([1, 3, 4, 8])
        N = max(1, min(_log(rng, 1, 8192), 150000000 // (B * hkv * (G + 2) * D)))
        chunks = rng.choice([B, B, rng.randint(0, B)])
        return dict(op=op, B=B, N=N, chunks=chunks, Hq=hkv * G, Hkv=hkv, D=D,
                    dtype=dtype, cache=rng.choice([dtype, dtype, "e4m3", "e5m2"]), layout=layout,
                    bs=bs, rot=2 * rng.randint(D // 8, D // 2), pairs=rng.random() < 0.3,
                    norm=rng.random() < 0.5, strided=strided, pos=_log(rng, 64, 1000000))
    dtype = rng.choice(["bf16", "bf16", "f16"])
    D = rng.choice([64, 80, 96, 128, 128, 128, 256])
    G = rng.choice([1, 2, 4, 4, 5, 7, 8])
    kind = rng.choice(["token", "chain", "prompt", "chunk", "mixed"])
    B = _log(rng, 1, 128) if kind in ("token", "chain", "mixed") else rng.randint(1, 4)
    N = {"token": 1, "chain": rng.randint(2, 16), "prompt": _log(rng, 20, 8192),
         "chunk": _log(rng, 20, 2048), "mixed": _log(rng, 20, 1024)}[kind]
    chunks = rng.randint(1, min(4, B)) if kind == "mixed" else B
    ctx = 0 if kind == "prompt" else _log(rng, 1, 300000 if kind == "token" else 100000)
    # what the plain form holds at once: scores of all pairs, and K and V in 32 bits
    N = max(1, min(N, int((2000000000 // (B * hkv * G)) ** 0.5)))
    ctx = max(0, min(ctx, 2000000000 // (B * hkv * G * N) - N, 1500000000 // (B * hkv * D)))
    window = rng.choice([0, 0, 0, _log(rng, 1, 8192)])
    return dict(op=op, B=B, N=N, chunks=chunks, Hq=hkv * G, Hkv=hkv, D=D, dtype=dtype,
                cache=rng.choice([dtype, dtype, dtype, "e4m3", "e5m2"]), layout=layout, bs=bs,
                ctx=ctx, window=window, sinks=rng.choice([0, 1, 4, 130]) if window else 0,
                strided=strided)


def _spread(most, b):
    """Request b's share of the largest size: all of it for the first, a quarter to all later."""
    f = 1.0 if b == 0 else 0.25 + 0.75 * math.modf(b * 0.6180339887498949)[0]
    return int(most * f)


def _counts(c):
    """New tokens of each request: about N for `chunks` of them, one for the others; every
    thirteenth has none."""
    every = max(1, c["B"] // c["chunks"]) if c["chunks"] else 0
    out, left = [], c["chunks"]
    for b in range(c["B"]):
        chunk = left > 0 and b % every == 0
        left -= chunk
        out.append(0 if b % 13 == 12 else max(1, _spread(c["N"], b)) if chunk else 1)
    return out


def _earlier(c):
    """Positions of each request before its new tokens (attend)."""
    return [_spread(c["ctx"], b) for b in range(c["B"])]


def _live(c):
    """Slots of each request that a logprobs call scores: all P, or an accepted path and bonus."""
    return [1 + (3 + 5 * b) % c["P"] if c["path"] else c["P"] for b in range(c["B"])]


def _seen(c, p, n):
    """(keys that any of n tokens from position p on sees, pairs of a token and a key it sees)."""
    w, s = c["window"], c["sinks"]
    if not w:
        return p + n, n * p + n * (n + 1) // 2
    t = np.arange(p, p + n, dtype=np.int64)
    first = np.maximum(t - w + 1, 0)
    pairs = int((t - first + 1 + np.minimum(first, s)).sum())
    return (int(p + n - first[0] + min(first[0], s)), pairs) if n else (0, 0)


def work(case):
    c = case
    e = BYTES[c["dtype"]]
    if c["op"] == "logprobs":
        rows = sum(_live(c))
        out = c["B"] * c["P"] * (4 + 8 * c["C"] + 8 * c["K"])
        return {"bytes": rows * c["V"] * e + out, "flops": rows * c["V"] * 6}
    ce, n = BYTES[c["cache"]], _counts(c)
    wide, kv = c["Hq"] * c["D"], 2 * c["Hkv"] * c["D"]
    if c["op"] == "append":
        return {"bytes": sum(n) * (2 * wide * e + kv * (e + ce)),
                "flops": sum(n) * (wide + kv // 2) * (3 + 4 * c["norm"])}
    seen = [_seen(c, p, k) for p, k in zip(_earlier(c), n)]
    return {"bytes": sum(s[0] for s in seen) * kv * ce + sum(n) * (2 * wide * e + 4 * c["Hq"]),
            "flops": 4 * wide * sum(s[1] for s in seen)}


# ---- inputs --------------------------------------------------------------------------------

def _rows(g, T, H, D, dtype, strided, std=1.0):
    """[T, H, D] rows: contiguous, or the middle columns of a wider projection output."""
    wide = H * D + (2 * D if strided else 0)
    x = (torch.randn((T, wide), generator=g, device=DEV) * std).to(DTYPES[dtype])
    return x[:, D:D + H * D].unflatten(1, (H, D)) if strided else x.view(T, H, D)


def _cache(c, g, last, filled):
    """A paged cache for positions below last[b], and a block table in random order. Without
    `filled` it holds zeros."""
    H, D, bs, kind = c["Hkv"], c["D"], c["bs"], c["cache"]
    pages = [(n + bs - 1) // bs for n in last]
    nb = sum(pages) + 1
    shape = (nb, bs, H, D) if c["layout"] == "NHD" else (nb, H, bs, D)
    s = {key: torch.zeros(shape, dtype=DTYPES[kind], device=DEV) for key in ("k", "v")}
    s["k_scale"] = s["v_scale"] = None
    if BYTES[kind] == 1:
        s["k_scale"] = torch.tensor([0.0625], device=DEV)
        s["v_scale"] = torch.tensor([0.015625], device=DEV)
    step = max(1, (1 << 26) // (bs * H * D))
    for at in range(0, nb if filled else 0, step):
        for key, std in (("k", 1.0), ("v", 0.5)):
            # heads have channels of unequal size, as keys have
            to = s[key][at:at + step]
            x = torch.randn(to.shape, generator=g, device=DEV) * std
            x *= 0.5 + 2.0 * torch.rand((D,), generator=g, device=DEV) ** 4
            to.view(torch.uint8).copy_(_stored(x, s[key + "_scale"], kind).view(torch.uint8))
    order = torch.randperm(nb, generator=g, device=DEV).int().cpu().numpy()
    table, at = np.zeros((len(last), max(1, max(pages))), np.int32), 1
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"], s["spare"] = torch.from_numpy(table).to(DEV), int(order[0])
    return s


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) % (1 << 62))
    rng = np.random.default_rng(int(seed) % (1 << 62))
    s = {"case": c}
    B, dtype = c["B"], c["dtype"]
    if c["op"] == "logprobs":
        N, P, V = c["N"], c["P"], c["V"]
        s["logits"] = torch.empty((B, N, V), dtype=DTYPES[dtype], device=DEV)
        rows = s["logits"].view(B * N, V)
        step = max(1, (1 << 26) // V)
        for at in range(0, B * N, step):
            rows[at:at + step] = 2.5 * torch.randn(rows[at:at + step].shape, generator=g,
                                                   device=DEV)
        tokens = rng.integers(0, V, (B, P, c["C"]))
        node = np.tile(np.arange(P), (B, 1))
        if c["path"]:
            for b, n in enumerate(_live(c)):
                node[b, 1:n] = 1 + np.sort(rng.permutation(N - 1)[:n - 1])
                node[b, n:] = -1
                tokens[b, n:] = -1
        s["node"] = torch.from_numpy(node.astype(np.int32)).to(DEV) if c["path"] else None
        tokens = torch.from_numpy(tokens.astype(np.int32)).to(DEV)
        # the model likes most of what it answered
        at = torch.from_numpy((np.arange(B)[:, None] * N + node)[node >= 0]).to(DEV)
        liked = tokens[..., 0][torch.from_numpy(node >= 0).to(DEV)].long()
        rows[at, liked] = (8 + 6 * torch.rand(at.shape, generator=g, device=DEV)).to(rows.dtype)
        s["tokens"] = tokens.squeeze(-1) if c["C"] == 1 else tokens
        return s
    counts = _counts(c)
    T, Hq, Hkv, D = sum(counts), c["Hq"], c["Hkv"], c["D"]
    s["T"], s["most"] = T, max(counts)
    s["row_start"] = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device=DEV)
    s["q"] = _rows(g, T, Hq, D, dtype, c["strided"], 1.5)
    if c["op"] == "append":
        s["pos"] = rng.integers(0, c["bs"], B)
        s.update(_cache(c, g, [c["bs"] - 1 + n for n in counts], False))
        s["new_k"] = _rows(g, T, Hkv, D, dtype, c["strided"])
        s["new_v"] = _rows(g, T, Hkv, D, dtype, c["strided"], 0.5)
        s["qw"] = s["kw"] = None
        if c["norm"]:
            s["qw"], s["kw"] = ((torch.rand(D, generator=g, device=DEV) + 0.5).to(DTYPES[dtype])
                                for _ in range(2))
        # pages before the new tokens' are another request's business: positions begin a
        # multiple of the page size further on, and the table does too
        far = rng.integers(0, c["pos"] // c["bs"] + 1, B)
        width = int(far.max()) + s["table"].shape[1]
        table = np.zeros((B, width), np.int32)
        for b in range(B):
            table[b, far[b]:far[b] + s["table"].shape[1]] = s["table"][b].cpu().numpy()
        s["table"] = torch.from_numpy(table).to(DEV)
        s["pos"] = s["pos"] + far * c["bs"]
        s["inv_freq"] = (1e6 ** (-torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64) /
                                 (c["rot"] // 2))).float()
    else:
        s["pos"] = np.array(_earlier(c))
        s.update(_cache(c, g, [int(p) + n for p, n in zip(s["pos"], counts)], True))
    s["seq_pos"] = torch.from_numpy(s["pos"].astype(np.int32)).to(DEV)
    owner = np.repeat(np.arange(B), counts)
    start = np.cumsum([0] + counts)[:-1]
    s["owner"] = torch.from_numpy(owner).to(DEV)
    s["place"] = torch.from_numpy(np.arange(T) - start[owner]).to(DEV)
    return s


# ---- the operators in plain torch operations -------------------------------------------------

def _stored(x, scale, kind):
    """float32 values as the cache holds them."""
    if BYTES[kind] > 1:
        return x.to(DTYPES[kind])
    return (x / scale).clamp(-LARGEST[kind], LARGEST[kind]).to(DTYPES[kind])


def _plain_append(s):
    c = s["case"]
    half = c["rot"] // 2
    pos = s["seq_pos"].long()[s["owner"]] + s["place"]
    ang = (pos.double().unsqueeze(-1) * s["inv_freq"].double()).unsqueeze(1)
    cos, sin = ang.cos().float(), ang.sin().float()

    def turned(x, w):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
        r, rest = y[..., :c["rot"]], y[..., c["rot"]:]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["pairs"] else (r[..., :half], r[..., half:])
        a, b = a * cos - b * sin, b * cos + a * sin
        r = torch.stack((a, b), -1).flatten(-2) if c["pairs"] else torch.cat((a, b), -1)
        return torch.cat((r, rest), -1)

    page = s["table"].long()[s["owner"], pos // c["bs"]]
    slot = pos % c["bs"]
    for key, x in (("k", turned(s["new_k"], s["kw"])), ("v", s["new_v"].float())):
        x = _stored(x, s[key + "_scale"], c["cache"])
        to = s[key]
        if BYTES[c["cache"]] == 1:
            x, to = x.view(torch.uint8), to.view(torch.uint8)
        if c["layout"] == "NHD":
            to[page, slot] = x
        else:
            to[page, :, slot] = x
    return turned(s["q"], s["qw"]).to(s["q"].dtype), s["k"], s["v"]


def _read(s, key, pos):
    """Positions [B, L] of the cache in 32 bits, [B, L, H, D]."""
    c = s["case"]
    page = torch.gather(s["table"].long(), 1, (pos // c["bs"]).clamp(max=s["table"].shape[1] - 1))
    slot, t = pos % c["bs"], s[key]
    small = BYTES[c["cache"]] == 1
    if small:
        t = t.view(torch.uint8)
    x = t[page, slot] if c["layout"] == "NHD" else t[page, :, slot]
    return x.view(s[key].dtype).float() * s[key + "_scale"] if small else x.float()


def _plain_attend(s):
    c = s["case"]
    B, N, H, G, D = c["B"], s["most"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    L = int(s["pos"].max()) + N
    key = torch.arange(L, device=DEV)
    n = (s["row_start"][1:] - s["row_start"][:-1]).unsqueeze(1)
    live = torch.arange(N, device=DEV).unsqueeze(0) < n                             # [B, N]
    at = s["seq_pos"].unsqueeze(1) + torch.arange(N, device=DEV)                    # [B, N]
    seen = (key <= at.unsqueeze(-1)) & live.unsqueeze(-1)                           # [B, N, L]
    if c["window"]:
        seen &= (key > at.unsqueeze(-1) - c["window"]) | (key < c["sinks"])
    seen = seen.unsqueeze(2).unsqueeze(1)                                           # [B, 1, N, 1, L]
    q = torch.zeros((B, N, c["Hq"], D), device=DEV)
    q[s["owner"], s["place"]] = s["q"].float() * D ** -0.5
    q = q.unflatten(2, (H, G)).permute(0, 2, 1, 3, 4).reshape(B, H, N * G, D)
    k = _read(s, "k", key.unsqueeze(0).expand(B, -1)).permute(0, 2, 3, 1)           # [B, H, D, L]
    z = torch.matmul(q, k).unflatten(2, (N, G))                                     # [B, H, N, G, L]
    del k
    z.masked_fill_(~seen, -math.inf)
    m = z.amax(-1, keepdim=True).clamp(min=-3.0e38)
    z = z.sub_(m).exp_()
    total = z.sum(-1, keepdim=True)
    v = _read(s, "v", key.unsqueeze(0).expand(B, -1)).permute(0, 2, 1, 3)           # [B, H, L, D]
    o = torch.matmul(z.flatten(2, 3), v).unflatten(2, (N, G))
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4)
    lse = torch.where(total > 0, m + total.log(), -math.inf).squeeze(-1).permute(0, 2, 1, 3)
    at = s["owner"], s["place"]
    return (o.reshape(B, N, c["Hq"], D)[at].to(DTYPES[c["dtype"]]),
            lse.reshape(B, N, c["Hq"])[at].contiguous())


def _plain_logprobs(s):
    c = s["case"]
    B, P, V, K = c["B"], c["P"], c["V"], c["K"]
    node = s["node"].long() if c["path"] else torch.arange(P, device=DEV).expand(B, -1)
    live = (node >= 0).flatten()
    at = (torch.arange(B, device=DEV).unsqueeze(1) * c["N"] + node).flatten()[live]
    x = s["logits"].view(-1, V)[at].float()
    z = x / c["temp"]
    z = z - z.amax(-1, keepdim=True)
    e = z.exp()
    total = e.sum(-1, keepdim=True)
    log_total = total.log()
    entropy = torch.zeros(B * P, device=DEV)
    entropy[live] = (log_total - (e * z).sum(-1, keepdim=True) / total).squeeze(-1)
    tokens = s["tokens"].view(B * P, c["C"])[live].long()
    logprob = torch.zeros((B * P, c["C"]), device=DEV)
    logprob[live] = torch.where(tokens >= 0, z.gather(1, tokens.clamp(min=0)) - log_total, 0.0)
    out = dict(logprob=logprob.view(s["tokens"].shape), entropy=entropy.view(B, P))
    del e
    if K:
        # one number orders them: the value, then the lower index
        bits = (x + 0.0).view(torch.int32).long()
        bits = torch.where(bits < 0, bits ^ 0x7fffffff, bits)
        order = bits * 4294967296 + (4294967295 - torch.arange(V, device=DEV))
        ids = 4294967295 - (order.topk(K, -1).values & 4294967295)
        top_ids = torch.full((B * P, K), -1, dtype=torch.int32, device=DEV)
        top = torch.full((B * P, K), -math.inf, device=DEV)
        top_ids[live] = ids.int()
        top[live] = z.gather(1, ids) - log_total
        out.update(top_ids=top_ids.view(B, P, K), top_logprobs=top.view(B, P, K))
    return out


# ---- one pass ------------------------------------------------------------------------------

_kept = {}


def _handle():
    """The library handle that a program keeps for its process."""
    if "h" not in _kept:
        from speculative_decoding_tree_mask_gb300 import binding as G
        _kept["G"], _kept["h"] = G, G.Handle(256, 64, 1 << 18, torch.cuda.current_device())
    return _kept["G"], _kept["h"]


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend,
                "logprobs": _plain_logprobs}[op](s)
    G, h = _handle()
    if op == "logprobs":
        out = G.token_logprobs(h, s["logits"], s["tokens"], node=s["node"],
                               temperature=c["temp"], top=c["K"])
        return {k: out[k] for k in ("logprob", "entropy") +
                (("top_ids", "top_logprobs") if c["K"] else ())}
    cache = G.KvCache(s["k"], s["v"], LAYOUTS[c["layout"]], s["k_scale"], s["v_scale"])
    if op == "append":
        q = G.kv_append(h, s["q"], s["new_k"], s["new_v"], cache, s["table"], s["seq_pos"],
                        s["row_start"], inv_freq=s["inv_freq"], q_weight=s["qw"],
                        k_weight=s["kw"], eps=EPS,
                        style=G.SPEC_ROPE_PAIRS if c["pairs"] else G.SPEC_ROPE_HALVES)
        return q, s["k"], s["v"]
    return G.paged_attention(h, s["q"], cache, s["table"], s["seq_pos"], c["D"] ** -0.5,
                             s["row_start"], max_new=s["most"], window=c["window"],
                             sinks=c["sinks"])


# ---- the definitions in 64 bits --------------------------------------------------------------

def _grid(kind):
    """The values of an 8-bit type's codes 0 .. 127 that are numbers, in order."""
    code = np.arange(128)
    bits, bias = (3, 7) if kind == "e4m3" else (2, 15)
    e, m = code >> bits, (code & ((1 << bits) - 1)) / 2.0 ** bits
    v = np.where(e == 0, m * 2.0 ** (1 - bias), (1 + m) * 2.0 ** (e.astype(np.float64) - bias))
    return v[:127] if kind == "e4m3" else v[:124]


def _exact_stored(x, scale, kind):
    """What float64 x stands for in the cache, over the tensor scale."""
    if BYTES[kind] > 1:
        return x
    x = x / scale.double()
    grid = torch.from_numpy(_grid(kind)).to(DEV)
    a = x.abs().clamp(max=float(grid[-1]))
    hi = torch.searchsorted(grid, a).clamp(1, len(grid) - 1)
    lo = hi - 1
    d0, d1 = a - grid[lo], grid[hi] - a
    pick = torch.where((d0 < d1) | ((d0 == d1) & (lo % 2 == 0)), lo, hi)
    return torch.copysign(grid[pick], x)


def _exact_append(s):
    c = s["case"]
    counts = _counts(c)
    pos = np.concatenate([s["pos"][b] + np.arange(n) for b, n in enumerate(counts)])
    turn = pos.astype(np.float64)[:, None] * s["inv_freq"].cpu().numpy().astype(np.float64)
    turn = torch.from_numpy(np.exp(1j * turn)).to(DEV).unsqueeze(1)
    n, half = c["rot"], c["rot"] // 2
    first = torch.arange(0, n, 2) if c["pairs"] else torch.arange(half)
    second = first + (1 if c["pairs"] else half)
    out = []
    for x, w in ((s["q"], s["qw"]), (s["new_k"], s["kw"])):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt(torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / c["D"] +
                               EPS) * w.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    table = s["table"].cpu().numpy()
    owner = np.repeat(np.arange(c["B"]), counts)
    page = torch.from_numpy(table[owner, pos // c["bs"]].astype(np.int64)).to(DEV)
    slot = torch.from_numpy(pos % c["bs"]).to(DEV)
    caches = []
    for key, x in (("k", out[1]), ("v", s["new_v"].double())):
        to = s[key].double()
        x = _exact_stored(x, s[key + "_scale"], c["cache"])
        flat = to if c["layout"] == "NHD" else to.transpose(1, 2)
        flat[page, slot] = x
        caches.append(to)
    return out[0], caches[0], caches[1]


def _exact_read(s, name, page, slot, head):
    """Positions of one head in float64."""
    t, scale = s[name], s[name + "_scale"]
    bits = t.view(torch.uint8 if t.element_size() == 1 else torch.int16)
    x = bits[page, slot, head] if s["case"]["layout"] == "NHD" else bits[page, head, slot]
    x = x.view(t.dtype).double()
    return x if scale is None else x * scale.double()


def _exact_attend(s):
    c = s["case"]
    G, D, bs = c["Hq"] // c["Hkv"], c["D"], c["bs"]
    out = torch.zeros((s["T"], c["Hq"], D), dtype=torch.float64, device=DEV)
    lse = torch.full((s["T"], c["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    row = 0
    for b, n in enumerate(_counts(c)):
        if n == 0:
            continue
        p = int(s["pos"][b])
        key = torch.arange(p + n, device=DEV)
        page, slot = s["table"][b].long()[key // bs], key % bs
        for h in range(c["Hkv"]):
            k, v = (_exact_read(s, key_, page, slot, h) for key_ in ("k", "v"))
            for at in range(0, n, 1024):
                t = torch.arange(p + at, p + min(n, at + 1024), device=DEV).unsqueeze(1)
                hide = key > t
                if c["window"]:
                    hide = hide | ((t - key >= c["window"]) & (key >= c["sinks"]))
                rows = slice(row + at, row + min(n, at + 1024))
                q = s["q"][rows, h * G:(h + 1) * G].double()
                z = torch.einsum("ngd,ld->ngl", q, k) / math.sqrt(D)
                z = z.masked_fill(hide.unsqueeze(1), -math.inf)
                lse[rows, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                out[rows, h * G:(h + 1) * G] = torch.einsum("ngl,ld->ngd",
                                                            torch.softmax(z, -1), v)
        row += n
    return out, lse


def _exact_logprobs(s):
    c = s["case"]
    B, P, K = c["B"], c["P"], c["K"]
    f64 = dict(dtype=torch.float64, device=DEV)
    logprob = torch.zeros(s["tokens"].shape, **f64)
    entropy = torch.zeros((B, P), **f64)
    top_ids = torch.full((B, P, K), -1, dtype=torch.int32, device=DEV)
    top = torch.full((B, P, K), -math.inf, **f64)
    live = _live(c)
    for b in range(B):
        for at in range(0, live[b], 256):
            slots = slice(at, min(live[b], at + 256))
            nodes = s["node"][b, slots].long() if c["path"] else torch.arange(
                slots.start, slots.stop, device=DEV)
            x = s["logits"][b, nodes].double()
            lp = torch.log_softmax(x / c["temp"], -1)
            entropy[b, slots] = -(lp.exp() * lp).sum(-1)
            tok = s["tokens"][b, slots].long()
            got = lp.gather(1, tok if tok.dim() == 2 else tok.unsqueeze(1))
            logprob[b, slots] = got if tok.dim() == 2 else got.squeeze(1)
            if K:
                value, index = x.sort(dim=-1, descending=True, stable=True)
                top_ids[b, slots] = index[:, :K].int()
                top[b, slots] = lp.gather(1, index[:, :K])
    out = dict(logprob=logprob, entropy=entropy)
    if K:
        out.update(top_ids=top_ids, top_logprobs=top)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend,
            "logprobs": _exact_logprobs}[case["op"]](s)
