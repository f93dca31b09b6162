"""Refusals of the tree-step entry points that need no GPU: the library's without a handle,
and the binding's checks of shapes, types and strides (CPU tensors: none reaches the library)."""
import ctypes

import pytest
import torch

from speculative_decoding_tree_mask_gb300 import binding as G
from speculative_decoding_tree_mask_gb300 import build as B


class NoHandle:
    device, ptr = 0, None


H = NoHandle()


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def cache(D=64, heads=2):
    return G.Fp4Cache.empty(5, 4, heads, D, "cpu")


@pytest.fixture(scope="module")
def lib():
    B.build()
    return G.load()


def test_library_refuses_a_null_handle(lib):
    n = ctypes.c_int64()
    assert lib.spec_qk_norm_rope(None, None, 0, None, 0, 1, 1, 1, 1, 1, 64, None, None, 0.0, None,
                                 0, 0, None, None, None, 0, None, 0, None) == G.SPEC_ERR_ARG
    assert lib.spec_kv_commit_fp4(None, None, 0, None, 0, 1, 1, 1, None, None, None, None, None,
                                  None) == G.SPEC_ERR_ARG
    assert lib.spec_kv_load_fp4(None, None, 1, None, None, 1, None, None, 1, None,
                                None) == G.SPEC_ERR_ARG
    assert lib.spec_tree_attention_workspace(None, 1, 1, 1, 1, 64,
                                             ctypes.byref(n)) == G.SPEC_ERR_ARG
    assert lib.spec_tree_attention_fp4(None, None, 0, None, 0, None, 0, 1, 1, 1, 1, None, None,
                                       None, 1.0, None, None, None, None, 0,
                                       None) == G.SPEC_ERR_ARG


def test_cache_shapes():
    c = G.Fp4Cache.empty(5, 4, 3, 96, "cpu", G.SPEC_KV_HND)
    assert (c.num_blocks, c.block_size, c.H, c.D) == (5, 4, 3, 96)
    c = G.Fp4Cache.empty(5, 4, 3, 96, "cpu", G.SPEC_KV_NHD)
    assert (c.num_blocks, c.block_size, c.H, c.D) == (5, 4, 3, 96)
    with pytest.raises(ValueError):
        G.Fp4Cache.empty(5, 4, 3, 40, "cpu")
    with pytest.raises(ValueError):
        G.Fp4Cache(c.k, c.v, c.k_sf, c.v_sf, layout=2)
    with pytest.raises(TypeError):
        G.Fp4Cache(c.k.int(), c.v, c.k_sf, c.v_sf)
    with pytest.raises(ValueError):
        G.Fp4Cache(c.k, c.v, c.k_sf[..., :2], c.v_sf[..., :2])
    with pytest.raises(TypeError):
        G.Fp4Cache(c.k, c.v, c.k_sf, c.v_sf, k_scale=torch.ones(2))


def rope_args(**kw):
    a = dict(q=bf(2, 3, 4, 64), k=bf(2, 3, 2, 64), inv_freq=torch.ones(32), seq_pos=i32(2),
             depth=i32(2, 3), q_out=bf(2, 3, 4, 64), k_out=bf(2, 3, 2, 64))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,err", [
    (dict(k=bf(2, 4, 2, 64)), ValueError), (dict(k=bf(2, 3, 2, 32)), ValueError),
    (dict(q_out=bf(2, 3, 4, 32)), ValueError), (dict(k=bf(2, 3, 2, 64).float()), TypeError),
    (dict(q_weight=bf(32), k_weight=bf(64)), ValueError),
    (dict(q_weight=bf(64).float(), k_weight=bf(64)), TypeError),
    (dict(inv_freq=torch.ones(32).double()), TypeError), (dict(seq_pos=i32(3)), ValueError),
    (dict(depth=i32(2, 3).long()), TypeError), (dict(depth=i32(3, 2)), ValueError),
    (dict(), ValueError)])            # everything right but the memory: not CUDA tensors
def test_qk_norm_rope_refusals(kw, err):
    with pytest.raises(err):
        G.spec_qk_norm_rope(H, **rope_args(**kw))


@pytest.mark.parametrize("kw,err", [
    (dict(src_k=bf(2, 3, 2, 32)), ValueError), (dict(src_v=bf(2, 3, 1, 64)), ValueError),
    (dict(src_v=bf(2, 3, 2, 64).half()), TypeError), (dict(block_table=i32(3, 4)), ValueError),
    (dict(seq_pos=i32(2).long()), TypeError), (dict(kv_commit=i32(2, 2)), ValueError),
    (dict(accept_len=i32(3)), ValueError), (dict(), ValueError)])
def test_kv_commit_fp4_refusals(kw, err):
    a = dict(src_k=bf(2, 3, 2, 64), src_v=bf(2, 3, 2, 64), cache=cache(), block_table=i32(2, 4),
             seq_pos=i32(2))
    a.update(kw)
    with pytest.raises(err):
        G.spec_kv_commit_fp4(H, **a)


@pytest.mark.parametrize("kw,err", [
    (dict(out_k=bf(2, 7, 2, 32)), ValueError), (dict(out_v=bf(2, 6, 2, 64)), ValueError),
    (dict(out_v=bf(2, 7, 2, 64).float()), TypeError), (dict(count=i32(1)), ValueError),
    (dict(start=i32(2).long()), TypeError), (dict(), ValueError)])
def test_kv_load_fp4_refusals(kw, err):
    a = dict(cache=cache(), block_table=i32(2, 4), start=i32(2), count=i32(2),
             out_k=bf(2, 7, 2, 64), out_v=bf(2, 7, 2, 64))
    a.update(kw)
    with pytest.raises(err):
        G.spec_kv_load_fp4(H, **a)


@pytest.mark.parametrize("kw,err", [
    (dict(q=bf(2, 3, 4, 32)), ValueError), (dict(k=bf(2, 3, 4, 64)), ValueError),
    (dict(v=bf(2, 3, 2, 64).half()), TypeError), (dict(out=bf(2, 3, 2, 64)), ValueError),
    (dict(ctx_len=i32(2).long()), TypeError), (dict(ctx_len=i32(3)), ValueError),
    (dict(anc_mask=i32(2, 3)), TypeError),
    (dict(anc_mask=torch.zeros(2, 4, dtype=torch.int64)), ValueError),
    (dict(lse=torch.zeros(2, 3, 4).double()), TypeError),
    (dict(lse=torch.zeros(2, 3, 2)), ValueError), (dict(status=i32(3)), ValueError),
    (dict(), ValueError)])
def test_tree_attention_fp4_refusals(kw, err):
    a = dict(q=bf(2, 3, 4, 64), k=bf(2, 3, 2, 64), v=bf(2, 3, 2, 64), cache=cache(),
             block_table=i32(2, 4), ctx_len=i32(2),
             anc_mask=torch.zeros(2, 3, dtype=torch.int64), scale=0.125, out=bf(2, 3, 4, 64),
             workspace=torch.zeros(1024, dtype=torch.uint8))
    a.update(kw)
    with pytest.raises(err):
        G.spec_tree_attention_fp4(H, **a)
