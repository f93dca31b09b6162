"""ctypes binding of ``libspecverify.so`` (C ABI in ``include/spec_verify.h``).

Argument marshalling only: every step runs in the library's CUDA kernels. Tensors are torch
CUDA tensors (torch provides device memory and streams); the functions keep the C names.
Loading fails loudly when the library has not been built.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(HERE, "libspecverify.so")
DEBUG_LIBRARY = os.path.join(HERE, "libspecverify_debug.so")   # checked flavour (SPEC_DEBUG)

SPEC_OK, SPEC_ERR_ARG, SPEC_ERR_UNSUPPORTED, SPEC_ERR_CUDA, SPEC_ERR_WORKSPACE = 0, -1, -2, -3, -4
SPEC_F32, SPEC_BF16 = 0, 1
SPEC_DRAFT_POINT, SPEC_DRAFT_PROBS_F32, SPEC_DRAFT_LOGITS = 0, 1, 2
SPEC_REQ_OK, SPEC_REQ_BAD_PARENT, SPEC_REQ_BAD_TOKEN, SPEC_REQ_BAD_ROW, SPEC_REQ_BAD_UNIFORM = \
    0, 1, 2, 3, 4
SPEC_ROW_NAN, SPEC_ROW_POSINF, SPEC_ROW_ALL_NEGINF = 1, 2, 4
KERNEL_CLASSES = ("tree_mask", "row_stats", "draft_stats", "walk_greedy", "walk_sample",
                  "lazy_greedy", "lazy_sample", "kv_commit", "budget", "qk_rope",
                  "kv_commit_fp4", "kv_load_fp4", "tree_attn")
SPEC_F16 = 2
SPEC_REQ_BAD_SLOT = 5
SPEC_REQ_BAD_BUDGET = 6
SPEC_REQ_INTERNAL = 7   # debug builds: a kernel's own consistency check failed
DBG_INDEX, DBG_ARRIVAL, DBG_WALK = 1, 2, 4
SPEC_KV_NHD, SPEC_KV_HND = 0, 1
SPEC_CACHE_SAME, SPEC_CACHE_FP8_E4M3, SPEC_CACHE_FP8_E5M2 = 0, 1, 2
SPEC_SCALE_TENSOR, SPEC_SCALE_PER_TOKEN = 0, 1
SPEC_ROPE_HALVES, SPEC_ROPE_PAIRS = 0, 1


class Fp4CacheStruct(ctypes.Structure):
    """spec_fp4_cache: the 4-bit paged cache as the library takes it (see Fp4Cache)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_sf", ctypes.c_void_p),
                ("v_sf", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_blocks", ctypes.c_int64),
                ("layout", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("H", ctypes.c_int32), ("D", ctypes.c_int32),
                ("block_table", ctypes.c_void_p), ("max_blocks", ctypes.c_int32)]


class BudgetParams(ctypes.Structure):
    """spec_budget_params: target ratio, moving-average weight, dead band, limits, step."""
    _fields_ = [("target", ctypes.c_double), ("alpha", ctypes.c_double),
                ("band", ctypes.c_double), ("n_min", ctypes.c_int32),
                ("n_max", ctypes.c_int32), ("step", ctypes.c_int32)]


_lock = threading.Lock()
_lib = None


class SpecError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {error_string(code)} ({code})")


def load() -> ctypes.CDLL:
    """Open the CUDA library (raises if it is missing)."""
    global _lib
    lib = _lib
    if lib is not None:
        return lib
    with _lock:
        if _lib is None:
            _lib = _open(LIBRARY)
        return _lib


@contextlib.contextmanager
def use_library(path: str):
    """Route every call of this module through another build of the library (for example the
    debug flavour, DEBUG_LIBRARY) inside the `with` block. Handles are tied to the build that
    created them: make them inside the block."""
    global _lib
    lib = _open(path)
    with _lock:
        prev = _lib
        _lib = lib
    try:
        yield lib
    finally:
        with _lock:
            _lib = prev


def _open(path: str) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it first "
            "(python -m speculative_decoding_tree_mask_gb300.build)")
    lib = ctypes.CDLL(path)
    P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    lib.spec_verify_init.argtypes = [ctypes.POINTER(P), i32, i32, i64, i32]
    lib.spec_verify_destroy.argtypes = [P]
    lib.spec_build_tree_mask.argtypes = [P, P, i32, i32, P, P, P, P]
    lib.spec_verify_greedy.argtypes = [P, P, i32, i32, i32, i64, P, P, P, P, P, P, P, P]
    lib.spec_verify_sample.argtypes = [P, P, i32, i32, i32, i64, P, P, P, i32, i32, f32,
                                       P, P, P, P, P, P, P]
    lib.spec_row_stats.argtypes = [P, P, i32, i32, i32, i64, f32, P, P, P, P, P, P, P, P]
    lib.spec_verify_greedy_lazy.argtypes = lib.spec_verify_greedy.argtypes
    lib.spec_kv_commit.argtypes = [P, P, P, i32, i32, i32, i32, i32, P, P, P, P, i32,
                                   i32, i32, i64, P, i32, P, P, P, i32, P, P]
    lib.spec_verify_sample_lazy.argtypes = lib.spec_verify_sample.argtypes
    lib.spec_set_node_budget.argtypes = [P, P]
    lib.spec_budget_update.argtypes = [P, ctypes.POINTER(BudgetParams), P, P, P, i32,
                                       i32, P, P, P]
    C = ctypes.POINTER(Fp4CacheStruct)
    lib.spec_qk_norm_rope.argtypes = [P, P, i64, P, i64, i32, i32, i32, i32, i32, i32, P, P, f32,
                                      P, i32, i32, P, P, P, i64, P, i64, P]
    lib.spec_kv_commit_fp4.argtypes = [P, P, i64, P, i64, i32, i32, i32, C, P, P, P, P, P]
    lib.spec_kv_load_fp4.argtypes = [P, C, i32, P, P, i64, P, P, i32, P, P]
    lib.spec_tree_attention_workspace.argtypes = [P, i32, i32, i32, i32, i32,
                                                  ctypes.POINTER(i64)]
    lib.spec_tree_attention_fp4.argtypes = [P, P, i64, P, i64, P, i64, i32, i32, i32, i32, C, P,
                                            P, f32, P, P, P, P, i64, P]
    lib.spec_profile_begin.argtypes = [P]
    lib.spec_profile_end.argtypes = [P, P, P]
    lib.spec_error_string.argtypes = [i32]
    lib.spec_error_string.restype = ctypes.c_char_p
    lib.spec_debug_build.argtypes = []
    lib.spec_debug_inject_arrival.argtypes = [P, i32, i32]
    lib.spec_debug_inject_lost_wait.argtypes = [P]
    lib.spec_debug_words.argtypes = [P, P, i32, P]
    return lib


def error_string(code: int) -> str:
    return load().spec_error_string(int(code)).decode()


def _check(rc: int, where: str):
    if rc != SPEC_OK:
        raise SpecError(rc, where)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to the library must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _ptr_dev_or_pinned(t):
    """Logits of the lazy calls: a CUDA tensor, or a page-locked host tensor (the library
    checks that the device maps it at the same address)."""
    if t is None:
        return None
    if not t.is_cuda and not t.is_pinned():
        raise ValueError("logits must be a CUDA tensor or a pinned host tensor")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _hdev(h) -> str:
    return f"cuda:{h.device}"


def _same_device(tensors, device, where):
    """Every CUDA tensor of a call must live on `device` (the handle's GPU, or for the
    handle-free call the logits' GPU): the kernels run there and take raw addresses."""
    dev = torch.device(device)
    for t in tensors:
        if t is not None and t.is_cuda and t.device != dev:
            raise ValueError(f"{where}: a tensor is on {t.device}, the call runs on {dev}")


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    if t.dtype == torch.float32:
        return SPEC_F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _i32(t, name):
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    return t


class Handle:
    """Owner of a ``spec_handle`` (workspace for B <= max_B, N <= max_N, V <= max_V)."""

    def __init__(self, max_B: int, max_N: int, max_V: int, device: int = 0):
        h = ctypes.c_void_p()
        _check(load().spec_verify_init(ctypes.byref(h), int(max_B), int(max_N), int(max_V),
                                       int(device)), "spec_verify_init")
        self.ptr = h
        self.device = int(device)
        self.torch_device = torch.device("cuda", self.device)
        self.max_B, self.max_N, self.max_V = int(max_B), int(max_N), int(max_V)
        self.attention_sizes = None     # sizes that attention_bytes (a workspace) belongs to
        self.attention_bytes = 0

    def close(self):
        if self.ptr is not None and self.ptr.value:
            load().spec_verify_destroy(self.ptr)
        self.ptr = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def spec_verify_init(max_B: int, max_N: int, max_V: int, device: int = 0) -> Handle:
    return Handle(max_B, max_N, max_V, device)


def spec_verify_destroy(h: Handle):
    h.close()


def spec_build_tree_mask(h: Handle, parent, anc_mask, depth, status, stream=None):
    """parent int32 [B, N] -> anc_mask int64 [B, N] (uint64 bit patterns), depth int32 [B, N],
    status int32 [B]."""
    B, N = parent.shape
    _same_device((parent, anc_mask, depth, status), _hdev(h), "spec_build_tree_mask")
    if anc_mask.dtype not in (torch.int64, getattr(torch, "uint64", torch.int64)):
        raise TypeError("anc_mask must be a 64-bit integer tensor")
    _check(load().spec_build_tree_mask(h.ptr, _ptr(_i32(parent, "parent")), B, N, _ptr(anc_mask),
                                       _ptr(_i32(depth, "depth")), _ptr(_i32(status, "status")),
                                       _stream(stream, parent.device)), "spec_build_tree_mask")


def spec_verify_greedy(h: Handle, logits, draft_token, parent, accept_len, out_tokens, kv_commit,
                       bonus, status, stream=None):
    B, N, V = logits.shape
    _same_device((logits, draft_token, parent, accept_len, out_tokens, kv_commit, bonus, status),
                 _hdev(h), "spec_verify_greedy")
    _check(load().spec_verify_greedy(
        h.ptr, _ptr(logits), _dtype_code(logits), B, N, V,
        _ptr(_i32(draft_token, "draft_token")), _ptr(_i32(parent, "parent")),
        _ptr(accept_len), _ptr(out_tokens), _ptr(kv_commit), _ptr(bonus), _ptr(status),
        _stream(stream, logits.device)), "spec_verify_greedy")


def spec_verify_sample(h: Handle, logits, draft_token, parent, temperature: float, uniforms,
                       accept_len, out_tokens, kv_commit, bonus, status, draft=None,
                       draft_kind: int = SPEC_DRAFT_POINT, stream=None):
    B, N, V = logits.shape
    _same_device((logits, draft_token, parent, uniforms, accept_len, out_tokens, kv_commit,
                  bonus, status, draft), _hdev(h), "spec_verify_sample")
    ddt = 0
    if draft is not None and draft_kind == SPEC_DRAFT_LOGITS:
        ddt = _dtype_code(draft)
    if draft is not None and draft_kind == SPEC_DRAFT_PROBS_F32 and draft.dtype != torch.float32:
        raise TypeError("draft probabilities must be float32")
    _check(load().spec_verify_sample(
        h.ptr, _ptr(logits), _dtype_code(logits), B, N, V,
        _ptr(_i32(draft_token, "draft_token")), _ptr(_i32(parent, "parent")), _ptr(draft),
        int(draft_kind), ddt, float(temperature), _ptr(uniforms), _ptr(accept_len),
        _ptr(out_tokens), _ptr(kv_commit), _ptr(bonus), _ptr(status),
        _stream(stream, logits.device)), "spec_verify_sample")


def spec_verify_greedy_lazy(h: Handle, logits, draft_token, parent, accept_len, out_tokens,
                            kv_commit, bonus, status, stream=None):
    """Greedy verification reading only the rows on the accepted path."""
    B, N, V = logits.shape
    _same_device((logits, draft_token, parent, accept_len, out_tokens, kv_commit, bonus, status),
                 _hdev(h), "spec_verify_greedy_lazy")
    _check(load().spec_verify_greedy_lazy(
        h.ptr, _ptr_dev_or_pinned(logits), _dtype_code(logits), B, N, V,
        _ptr(_i32(draft_token, "draft_token")), _ptr(_i32(parent, "parent")),
        _ptr(accept_len), _ptr(out_tokens), _ptr(kv_commit), _ptr(bonus), _ptr(status),
        _stream(stream, draft_token.device)), "spec_verify_greedy_lazy")


def spec_verify_sample_lazy(h: Handle, logits, draft_token, parent, temperature: float, uniforms,
                            accept_len, out_tokens, kv_commit, bonus, status, draft=None,
                            draft_kind: int = SPEC_DRAFT_POINT, stream=None):
    """Sampling verification reading only the rows the walk visits."""
    B, N, V = logits.shape
    _same_device((logits, draft_token, parent, uniforms, accept_len, out_tokens, kv_commit,
                  bonus, status, draft), _hdev(h), "spec_verify_sample_lazy")
    ddt = 0
    if draft is not None and draft_kind == SPEC_DRAFT_LOGITS:
        ddt = _dtype_code(draft)
    if draft is not None and draft_kind == SPEC_DRAFT_PROBS_F32 and draft.dtype != torch.float32:
        raise TypeError("draft probabilities must be float32")
    _check(load().spec_verify_sample_lazy(
        h.ptr, _ptr_dev_or_pinned(logits), _dtype_code(logits), B, N, V,
        _ptr(_i32(draft_token, "draft_token")), _ptr(_i32(parent, "parent")),
        _ptr_dev_or_pinned(draft), int(draft_kind), ddt, float(temperature), _ptr(uniforms),
        _ptr(accept_len), _ptr(out_tokens), _ptr(kv_commit), _ptr(bonus), _ptr(status),
        _stream(stream, draft_token.device)), "spec_verify_sample_lazy")


def spec_row_stats(h: Handle, logits, N: int, temperature: float, row_max, row_sum, row_argmax,
                   row_flags, draft_token=None, parent=None, child_prob=None, stream=None):
    """logits [rows, V] (or [B, N, V]) -> per-row max, sum, argmax, flags; optional gather of
    p_parent(token) at every child into child_prob [B, N]."""
    V = logits.shape[-1]
    rows = logits.numel() // V
    _same_device((logits, row_max, row_sum, row_argmax, row_flags, draft_token, parent,
                  child_prob), _hdev(h), "spec_row_stats")
    _check(load().spec_row_stats(
        h.ptr, _ptr(logits), _dtype_code(logits), rows, int(N), V, float(temperature),
        _ptr(draft_token), _ptr(parent), _ptr(row_max), _ptr(row_sum), _ptr(row_argmax),
        _ptr(row_flags), _ptr(child_prob), _stream(stream, logits.device)), "spec_row_stats")


def _kv_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return SPEC_F16
    return _dtype_code(t)


def spec_kv_commit(h: Handle, src_k, src_v, kv_commit, accept_len, cache_k, cache_v, layout: int,
                   block_table, seq_pos, cache_kind: int = SPEC_CACHE_SAME, k_scale=None,
                   v_scale=None, commit_status=None, stream=None):
    """Copy the K/V of the root and the accepted nodes ([B, N, H, D]) into a paged cache
    (NHD [blocks, block_size, H, D] or HND [blocks, H, block_size, D]); fp8 caches are uint8.
    Scales: float32 tensors of one element, or [B, N] (one per source token)."""
    B, N, H, D = src_k.shape
    _same_device((src_k, src_v, kv_commit, accept_len, cache_k, cache_v, block_table, seq_pos,
                  k_scale, v_scale, commit_status), _hdev(h), "spec_kv_commit")
    if layout == SPEC_KV_NHD:
        num_blocks, block_size = cache_k.shape[0], cache_k.shape[1]
    else:
        num_blocks, block_size = cache_k.shape[0], cache_k.shape[2]
    scale_mode = SPEC_SCALE_TENSOR
    given = [sc for sc in (k_scale, v_scale) if sc is not None]
    if any(sc.dtype != torch.float32 for sc in given):
        raise TypeError("scales must be float32")
    if any(sc.numel() != 1 for sc in given):
        if not all(tuple(sc.shape) == (B, N) for sc in given):
            raise ValueError("scales must all be single values or all [B, N]")
        scale_mode = SPEC_SCALE_PER_TOKEN
    _check(load().spec_kv_commit(
        h.ptr, _ptr(src_k), _ptr(src_v), _kv_dtype(src_k), B, N, H, D,
        _ptr(_i32(kv_commit, "kv_commit")), _ptr(_i32(accept_len, "accept_len")), _ptr(cache_k),
        _ptr(cache_v), int(cache_kind), int(layout), int(block_size), int(num_blocks),
        _ptr(_i32(block_table, "block_table")), int(block_table.shape[1]),
        _ptr(_i32(seq_pos, "seq_pos")), _ptr(k_scale), _ptr(v_scale), scale_mode,
        _ptr(commit_status),
        _stream(stream, src_k.device)), "spec_kv_commit")


# ---- the tree step over a 4-bit cache ----------------------------------------------------------
# A small call of these is shorter on the GPU than its argument checks once were on the host, so
# the checks compare whole shapes and integer device indices, and find words only on failure.

class Fp4Cache:
    """A 4-bit paged K/V cache (spec_fp4_cache): uint8 codes k, v [num_blocks, block_size, H,
    D/2] (SPEC_KV_NHD) or [num_blocks, H, block_size, D/2] (SPEC_KV_HND), uint8 e4m3 block
    scales k_sf, v_sf of the same shape but D/16, and float32 tensor scales of one element
    (None = 1). Holds the tensors; block tables come with each call."""

    def __init__(self, k, v, k_sf, v_sf, layout: int = SPEC_KV_NHD, k_scale=None, v_scale=None):
        if layout != SPEC_KV_NHD and layout != SPEC_KV_HND:
            raise ValueError("layout must be SPEC_KV_NHD or SPEC_KV_HND")
        u8 = torch.uint8
        if k.dtype != u8 or v.dtype != u8 or k_sf.dtype != u8 or v_sf.dtype != u8 or k.dim() != 4:
            raise TypeError("k, v, k_sf and v_sf must be 4-dimensional uint8 tensors")
        shape = k.shape
        if shape != v.shape or k_sf.shape != v_sf.shape or \
                shape != (*k_sf.shape[:-1], 8 * k_sf.shape[-1]):
            raise ValueError("k, v: [..., D/2], k_sf, v_sf: [..., D/16] of one shape")
        for s in (k_scale, v_scale):
            if s is not None and (s.dtype != torch.float32 or s.numel() != 1):
                raise TypeError("tensor scales must be float32 of one element")
        self.k, self.v, self.k_sf, self.v_sf = k, v, k_sf, v_sf
        self.k_scale, self.v_scale, self.layout = k_scale, v_scale, int(layout)
        if layout == SPEC_KV_NHD:
            self.num_blocks, self.block_size, self.H, half = shape
        else:
            self.num_blocks, self.H, self.block_size, half = shape
        self.D = 2 * half

    @classmethod
    def empty(cls, num_blocks: int, block_size: int, H: int, D: int, device,
              layout: int = SPEC_KV_NHD, k_scale=None, v_scale=None) -> "Fp4Cache":
        """A cache of zeros."""
        if D % 16 != 0:
            raise ValueError("D must be a multiple of 16")
        shape = (num_blocks, block_size, H) if layout == SPEC_KV_NHD else \
            (num_blocks, H, block_size)
        one = [torch.zeros(shape + (n,), dtype=torch.uint8, device=device)
               for n in (D // 2, D // 2, D // 16, D // 16)]
        return cls(*one, layout, k_scale, v_scale)

    def struct(self, block_table, B: int, device: int) -> Fp4CacheStruct:
        """The library's view of the cache on GPU `device`, with the block table int32
        [B, max_blocks]."""
        if block_table.dtype != torch.int32:
            raise TypeError("block_table must be int32")
        if block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError(f"block_table must be [{B}, max_blocks]")
        return Fp4CacheStruct(
            _addr(self.k, device), _addr(self.v, device), _addr(self.k_sf, device),
            _addr(self.v_sf, device), _addr(self.k_scale, device), _addr(self.v_scale, device),
            self.num_blocks, self.layout, self.block_size, self.H, self.D,
            _addr(block_table, device), block_table.shape[1])


def _addr(t, device: int):
    """Address of a contiguous tensor on GPU `device` (None for None)."""
    if t is None:
        return None
    if t.get_device() != device:
        raise ValueError(f"a tensor is on {t.device}, the call runs on cuda:{device}")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return t.data_ptr()


def _rows(t, device: int, name: str):
    """(address, token stride) of rows [B, N, H, D], contiguous or columns of a wider matrix."""
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the call runs on cuda:{device}")
    B, N, H, D = t.shape
    if t.is_contiguous():
        return t.data_ptr(), H * D
    sb, sn, sh, sd = t.stride()
    token = sn if N > 1 else sb if B > 1 else H * D
    if (sd != 1 and D > 1) or (sh != D and H > 1) or (B > 1 and N > 1 and sb != N * sn) or \
            token < H * D:
        raise ValueError(f"{name}: heads and elements must be contiguous, and tokens evenly "
                         "spaced")
    return t.data_ptr(), token


def _refuse(where: str, **wanted):
    """Raises for the first tensor that is not what `wanted` gives as name=(tensor, shape,
    dtype); a tensor may be None, a dtype too (any)."""
    for name, (t, shape, dtype) in wanted.items():
        if t is None:
            continue
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{where}: {name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{where}: {name} must be {list(shape)}, got {list(t.shape)}")


def _bad(t, shape, dtype) -> bool:
    return t is not None and (t.dtype != dtype or t.shape != shape)


def _raw_stream(stream, device: int):
    """The cudaStream_t of `stream`, or of the device's current stream."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream


_ROW_CODES = {torch.float32: SPEC_F32, torch.bfloat16: SPEC_BF16, torch.float16: SPEC_F16}


def _row_code(dtype, where: str) -> int:
    code = _ROW_CODES.get(dtype)
    if code is None:
        raise TypeError(f"{where}: rows must be float32, bfloat16 or float16, got {dtype}")
    return code


def spec_qk_norm_rope(h: Handle, q, k, inv_freq, seq_pos, depth, q_out, k_out, q_weight=None,
                      k_weight=None, eps: float = 1e-6, style: int = SPEC_ROPE_HALVES,
                      stream=None):
    """Norm of every query and key head and the rotation by seq_pos[b] + depth[b][n], in one
    pass. q [B, N, Hq, D], k [B, N, Hkv, D]; inv_freq float32 [rot/2] (None: no rotation);
    depth int32 [B, N] or None (n itself); weights [D] or None (no norm). q_out, k_out may be
    q and k."""
    where, i32, dt = "spec_qk_norm_rope", torch.int32, q.dtype
    qs = q.shape
    B, N, Hq, D = qs
    Hkv = k.shape[2]
    ks = (B, N, Hkv, D)
    if _bad(k, ks, dt) or _bad(q_out, qs, dt) or _bad(k_out, ks, dt) or \
            _bad(q_weight, (D,), dt) or _bad(k_weight, (D,), dt) or \
            _bad(seq_pos, (B,), i32) or _bad(depth, (B, N), i32) or \
            (inv_freq is not None and inv_freq.dtype != torch.float32):
        _refuse(where, k=(k, ks, dt), q_out=(q_out, qs, dt), k_out=(k_out, ks, dt),
                q_weight=(q_weight, (D,), dt), k_weight=(k_weight, (D,), dt),
                seq_pos=(seq_pos, (B,), i32), depth=(depth, (B, N), i32),
                inv_freq=(inv_freq, inv_freq.shape if inv_freq is not None else (),
                          torch.float32))
    dev = h.device
    qa, qt = _rows(q, dev, "q")
    ka, kt = _rows(k, dev, "k")
    qo, qot = _rows(q_out, dev, "q_out")
    ko, kot = _rows(k_out, dev, "k_out")
    _check(load().spec_qk_norm_rope(
        h.ptr, qa, qt, ka, kt, _row_code(dt, where), B, N, Hq, Hkv, D, _addr(q_weight, dev),
        _addr(k_weight, dev), eps, _addr(inv_freq, dev),
        0 if inv_freq is None else 2 * inv_freq.numel(), style, _addr(seq_pos, dev),
        _addr(depth, dev), qo, qot, ko, kot, _raw_stream(stream, dev)), where)


def spec_kv_commit_fp4(h: Handle, src_k, src_v, cache: Fp4Cache, block_table, seq_pos,
                       kv_commit=None, accept_len=None, commit_status=None, stream=None):
    """K/V rows [B, N, H, D] into the 4-bit cache: the root and the accepted nodes of a verify
    call (kv_commit, accept_len), or rows 0..accept_len[b] in order (kv_commit None; all N
    without accept_len), at positions seq_pos[b] + j."""
    where, i32, dt = "spec_kv_commit_fp4", torch.int32, src_k.dtype
    B, N = src_k.shape[:2]
    rows, one, dev = (B, N, cache.H, cache.D), (B,), h.device
    if _bad(src_k, rows, dt) or _bad(src_v, rows, dt) or _bad(seq_pos, one, i32) or \
            _bad(kv_commit, (B, N), i32) or _bad(accept_len, one, i32) or \
            _bad(commit_status, one, i32):
        _refuse(where, src_k=(src_k, rows, dt), src_v=(src_v, rows, dt),
                seq_pos=(seq_pos, one, i32), kv_commit=(kv_commit, (B, N), i32),
                accept_len=(accept_len, one, i32), commit_status=(commit_status, one, i32))
    view = cache.struct(block_table, B, dev)
    ka, kt = _rows(src_k, dev, "src_k")
    va, vt = _rows(src_v, dev, "src_v")
    _check(load().spec_kv_commit_fp4(
        h.ptr, ka, kt, va, vt, _row_code(dt, where), B, N, view, _addr(kv_commit, dev),
        _addr(accept_len, dev), _addr(seq_pos, dev), _addr(commit_status, dev),
        _raw_stream(stream, dev)), where)


def spec_kv_load_fp4(h: Handle, cache: Fp4Cache, block_table, start, count, out_k, out_v,
                     status=None, stream=None):
    """Positions start[b] .. start[b] + count[b] - 1 of the 4-bit cache into out_k, out_v
    [B, max_len, H, D]; rows at and after count[b] become zero."""
    where, i32, dt = "spec_kv_load_fp4", torch.int32, out_k.dtype
    B, max_len = out_k.shape[:2]
    rows, one, dev = (B, max_len, cache.H, cache.D), (B,), h.device
    if _bad(out_k, rows, dt) or _bad(out_v, rows, dt) or _bad(start, one, i32) or \
            _bad(count, one, i32) or _bad(status, one, i32):
        _refuse(where, out_k=(out_k, rows, dt), out_v=(out_v, rows, dt),
                start=(start, one, i32), count=(count, one, i32), status=(status, one, i32))
    _check(load().spec_kv_load_fp4(
        h.ptr, cache.struct(block_table, B, dev), B, _addr(start, dev), _addr(count, dev),
        max_len, _addr(out_k, dev), _addr(out_v, dev), _row_code(dt, where), _addr(status, dev),
        _raw_stream(stream, dev)), where)


def spec_tree_attention_workspace(h: Handle, B: int, N: int, Hq: int, H: int, D: int) -> int:
    """Bytes of workspace that spec_tree_attention_fp4 needs for these sizes."""
    n = ctypes.c_int64()
    _check(load().spec_tree_attention_workspace(h.ptr, int(B), int(N), int(Hq), int(H), int(D),
                                                ctypes.byref(n)),
           "spec_tree_attention_workspace")
    return n.value


def spec_tree_attention_fp4(h: Handle, q, k, v, cache: Fp4Cache, block_table, ctx_len, anc_mask,
                            scale: float, out, workspace, lse=None, status=None, stream=None):
    """Attention of the tree's nodes q [B, N, Hq, D] over positions 0..ctx_len[b]-1 of the
    4-bit cache and over the nodes k, v [B, N, H, D] that anc_mask (int64 [B, N] bit patterns,
    build_tree_mask) lets each see."""
    where, i32, dt = "spec_tree_attention_fp4", torch.int32, q.dtype
    B, N, Hq, D = q.shape
    full, rows, one, dev = (B, N, Hq, cache.D), (B, N, cache.H, cache.D), (B,), h.device
    bits = torch.int64 if anc_mask.dtype != getattr(torch, "uint64", None) else torch.uint64
    if _bad(q, full, dt) or _bad(k, rows, dt) or _bad(v, rows, dt) or _bad(out, full, dt) or \
            _bad(ctx_len, one, i32) or _bad(anc_mask, (B, N), bits) or \
            _bad(lse, (B, N, Hq), torch.float32) or _bad(status, one, i32):
        _refuse(where, q=(q, full, dt), k=(k, rows, dt), v=(v, rows, dt), out=(out, full, dt),
                ctx_len=(ctx_len, one, i32), anc_mask=(anc_mask, (B, N), bits),
                lse=(lse, (B, N, Hq), torch.float32), status=(status, one, i32))
    view = cache.struct(block_table, B, dev)
    qa, qt = _rows(q, dev, "q")
    ka, kt = _rows(k, dev, "k")
    va, vt = _rows(v, dev, "v")
    _check(load().spec_tree_attention_fp4(
        h.ptr, qa, qt, ka, kt, va, vt, _row_code(dt, where), B, N, Hq, view, _addr(ctx_len, dev),
        _addr(anc_mask, dev), scale, _addr(out, dev), _addr(lse, dev), _addr(status, dev),
        _addr(workspace, dev), workspace.numel() * workspace.element_size(),
        _raw_stream(stream, dev)), where)


def spec_set_node_budget(h: Handle, n_active):
    """Later verify calls on ``h`` verify request b as its first n_active[b] nodes (device
    int32 [>= B], read when the kernels run); None verifies every node."""
    if n_active is not None:
        _i32(n_active, "n_active")
    _check(load().spec_set_node_budget(h.ptr, _ptr(n_active)), "spec_set_node_budget")
    h.n_active = n_active   # keep the array alive while the handle reads it


def spec_budget_update(h: Handle, params: BudgetParams, accept_len, status, parent, state,
                       n_active, stream=None):
    """One controller update on the device; ``state`` is a tensor from budget_state()."""
    B, N = parent.shape
    _same_device((accept_len, status, parent, state, n_active), _hdev(h), "spec_budget_update")
    if state.dtype != torch.float64 or state.numel() != 2:
        raise TypeError("state must be the float64 [2] tensor made by budget_state()")
    _check(load().spec_budget_update(
        h.ptr, ctypes.byref(params), _ptr(_i32(accept_len, "accept_len")),
        _ptr(_i32(status, "status")), _ptr(_i32(parent, "parent")), B, N, _ptr(state),
        _ptr(_i32(n_active, "n_active")), _stream(stream, parent.device)), "spec_budget_update")


def budget_state(ema: float, budget: int, device, steps: int = 0) -> torch.Tensor:
    """A device spec_budget_state {double ema; int32 budget; int32 steps} in a float64 [2]."""
    t = torch.zeros(2, dtype=torch.float64)
    t[0] = float(ema)
    t[1:].view(torch.int32)[0] = int(budget)
    t[1:].view(torch.int32)[1] = int(steps)
    return t.to(device)


def read_budget_state(state: torch.Tensor):
    """-> (ema, budget, steps) of a state tensor (synchronises with the device)."""
    t = state.cpu()
    iv = t[1:].view(torch.int32)
    return float(t[0]), int(iv[0]), int(iv[1])


def spec_profile_begin(h: Handle):
    _check(load().spec_profile_begin(h.ptr), "spec_profile_begin")


def spec_profile_end(h: Handle):
    """-> {kernel class: (total ms, launches)} for the launches since spec_profile_begin."""
    ms = (ctypes.c_float * len(KERNEL_CLASSES))()
    n = (ctypes.c_int32 * len(KERNEL_CLASSES))()
    _check(load().spec_profile_end(h.ptr, ms, n), "spec_profile_end")
    return {k: (float(ms[i]), int(n[i])) for i, k in enumerate(KERNEL_CLASSES)}


# ---- convenience: allocate outputs -----------------------------------------------------------

def _new(device, stream, *specs, returned=True):
    """Tensors (shape, dtype) for a call on ``stream``, from that stream's memory: torch hands out
    freed memory again at once on the stream it belongs to, whose earlier work on it may not have
    run yet when another stream starts. `returned`: the caller gets them and may use and free
    them on the current stream, which is noted too."""
    if stream is None:
        return [torch.empty(shape, dtype=dtype, device=device) for shape, dtype in specs]
    if not isinstance(stream, torch.cuda.Stream):      # anything that has a cudaStream_t
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device)
    here = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        new = [torch.empty(shape, dtype=dtype, device=device) for shape, dtype in specs]
    if returned:
        for t in new:
            t.record_stream(here)
    return new


def alloc_outputs(B: int, N: int, device, stream=None) -> dict:
    """The outputs of a verify call on ``stream`` (None: the current one)."""
    one, all_nodes = ((B,), torch.int32), ((B, N), torch.int32)
    accept_len, out_tokens, kv_commit, bonus, status = _new(device, stream, one, all_nodes,
                                                            all_nodes, one, one)
    return dict(accept_len=accept_len, out_tokens=out_tokens, kv_commit=kv_commit, bonus=bonus,
                status=status)


def verify_greedy(h: Handle, logits, draft_token, parent, out: dict | None = None,
                  stream=None) -> dict:
    B, N, _ = logits.shape
    out = out or alloc_outputs(B, N, logits.device, stream)
    spec_verify_greedy(h, logits, draft_token, parent, out["accept_len"], out["out_tokens"],
                       out["kv_commit"], out["bonus"], out["status"], stream)
    return out


def verify_sample(h: Handle, logits, draft_token, parent, temperature, uniforms, draft=None,
                  draft_kind=SPEC_DRAFT_POINT, out: dict | None = None, stream=None) -> dict:
    B, N, _ = logits.shape
    out = out or alloc_outputs(B, N, logits.device, stream)
    spec_verify_sample(h, logits, draft_token, parent, temperature, uniforms, out["accept_len"],
                       out["out_tokens"], out["kv_commit"], out["bonus"], out["status"], draft,
                       draft_kind, stream)
    return out


def verify_greedy_lazy(h: Handle, logits, draft_token, parent, out: dict | None = None,
                       stream=None) -> dict:
    B, N, _ = logits.shape
    out = out or alloc_outputs(B, N, draft_token.device, stream)
    spec_verify_greedy_lazy(h, logits, draft_token, parent, out["accept_len"], out["out_tokens"],
                            out["kv_commit"], out["bonus"], out["status"], stream)
    return out


def verify_sample_lazy(h: Handle, logits, draft_token, parent, temperature, uniforms, draft=None,
                       draft_kind=SPEC_DRAFT_POINT, out: dict | None = None, stream=None) -> dict:
    B, N, _ = logits.shape
    out = out or alloc_outputs(B, N, draft_token.device, stream)
    spec_verify_sample_lazy(h, logits, draft_token, parent, temperature, uniforms,
                            out["accept_len"], out["out_tokens"], out["kv_commit"], out["bonus"],
                            out["status"], draft, draft_kind, stream)
    return out


def build_tree_mask(h: Handle, parent, stream=None) -> dict:
    B, N = parent.shape
    anc_mask, depth, status = _new(parent.device, stream, ((B, N), torch.int64),
                                   ((B, N), torch.int32), ((B,), torch.int32))
    out = dict(anc_mask=anc_mask, depth=depth, status=status)
    spec_build_tree_mask(h, parent, out["anc_mask"], out["depth"], out["status"], stream)
    return out


def qk_norm_rope(h: Handle, q, k, inv_freq, seq_pos, depth=None, q_weight=None, k_weight=None,
                 eps: float = 1e-6, style: int = SPEC_ROPE_HALVES, stream=None):
    """-> new contiguous (q, k), normalised and rotated (see spec_qk_norm_rope)."""
    qo, ko = _new(h.torch_device, stream, (q.shape, q.dtype), (k.shape, k.dtype))
    spec_qk_norm_rope(h, q, k, inv_freq, seq_pos, depth, qo, ko, q_weight, k_weight, eps, style,
                      stream)
    return qo, ko


def kv_load_fp4(h: Handle, cache: Fp4Cache, block_table, start, count, max_len: int,
                dtype=torch.bfloat16, stream=None, status=None):
    """-> (k, v) rows [B, max_len, H, D] of ``dtype`` (see spec_kv_load_fp4). status int32 [B]:
    what each request met (None: it stays unknown)."""
    shape = (block_table.shape[0], int(max_len), cache.H, cache.D)
    k, v = _new(h.torch_device, stream, (shape, dtype), (shape, dtype))
    spec_kv_load_fp4(h, cache, block_table, start, count, k, v, status, stream)
    return k, v


def tree_attention_fp4(h: Handle, q, k, v, cache: Fp4Cache, block_table, ctx_len, anc_mask,
                       scale: float, workspace=None, stream=None, status=None):
    """-> (out [B, N, Hq, D], lse float32 [B, N, Hq]) (see spec_tree_attention_fp4). Without a
    workspace one is taken from torch's allocator for the call. status int32 [B]: what each
    request met (None: it stays unknown)."""
    if workspace is None:
        B, N, Hq, D = q.shape
        sizes = (B, N, Hq, cache.H, D)
        if h.attention_sizes != sizes:      # the size depends on these alone
            h.attention_bytes = spec_tree_attention_workspace(h, *sizes)
            h.attention_sizes = sizes
        workspace, = _new(h.torch_device, stream, ((h.attention_bytes,), torch.uint8),
                          returned=False)
    out, lse = _new(h.torch_device, stream, (q.shape, q.dtype), (q.shape[:3], torch.float32))
    spec_tree_attention_fp4(h, q, k, v, cache, block_table, ctx_len, anc_mask, scale, out,
                            workspace, lse, status, stream)
    return out, lse


# ---- greedy verification without device allocation --------------------------------------------

SPEC_NOALLOC_MAX_ROWS = 16384


def spec_verify_greedy_noalloc(logits, draft_token, parent, accept_len, out_tokens, kv_commit,
                               bonus, status, stream=None):
    """Greedy verification whose scratch is a static device array (no cudaMalloc anywhere),
    for callers that must not allocate device memory. Runs on the tensors' device, which must
    be the current device; B*N <= SPEC_NOALLOC_MAX_ROWS. Calls share the scratch, so calls
    that overlap on the GPU race."""
    lib = load()
    fn = lib.spec_verify_greedy_noalloc
    if fn.argtypes is None:
        P, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        fn.argtypes = [P, i32, i32, i32, i64, P, P, P, P, P, P, P, P]
    B, N, V = logits.shape
    tensors = (logits, draft_token, parent, accept_len, out_tokens, kv_commit, bonus, status)
    _same_device(tensors, logits.device, "spec_verify_greedy_noalloc")
    # the library runs on the current device: make it the tensors' device for the call
    with torch.cuda.device(logits.device):
        _check(fn(_ptr(logits), _dtype_code(logits), B, N, V,
                  _ptr(_i32(draft_token, "draft_token")), _ptr(_i32(parent, "parent")),
                  _ptr(accept_len), _ptr(out_tokens), _ptr(kv_commit), _ptr(bonus),
                  _ptr(status), _stream(stream, logits.device)),
               "spec_verify_greedy_noalloc")


# ---- debug flavour -------------------------------------------------------------------------

def spec_debug_build() -> bool:
    """True when the loaded library is the checked (SPEC_DEBUG) build."""
    return bool(load().spec_debug_build())


def spec_debug_inject_arrival(h: Handle, row: int, value: int):
    """Debug builds: the next split row-statistics launch on ``h`` finds ``value`` in the
    arrival counter of ``row`` (a test of the counter check)."""
    _check(load().spec_debug_inject_arrival(h.ptr, int(row), int(value)),
           "spec_debug_inject_arrival")


def spec_debug_inject_lost_wait(h: Handle):
    """Debug builds: if the next tree attention on ``h`` runs on the tcgen05 tensor cores, all its
    waits give up at once (a test of lost results)."""
    _check(load().spec_debug_inject_lost_wait(h.ptr), "spec_debug_inject_lost_wait")


def spec_debug_words(h: Handle, B: int, stream=None) -> torch.Tensor:
    """Debug builds: the violation bits (DBG_*) of requests 0..B-1 in the handle's last call."""
    words, = _new(h.torch_device, stream, ((B,), torch.int32))
    _check(load().spec_debug_words(h.ptr, _ptr(words), int(B), _stream(stream, words.device)),
           "spec_debug_words")
    return words
