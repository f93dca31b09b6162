"""Refusals of the paged step and of token log probabilities that need no GPU: the library's without
a handle, and the binding's checks of shapes, types and strides (CPU tensors: none reaches the
library). And the oracle against plain loops."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import paged_step as S
from speculative_decoding_tree_mask_gb300 import binding as G
from speculative_decoding_tree_mask_gb300 import build as B


class NoHandle:
    device, ptr = 0, None


H = NoHandle()


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def f32(*shape):
    return torch.zeros(shape)


def cache(dtype=torch.bfloat16, D=64, heads=2, **kw):
    return G.KvCache.empty(5, 4, heads, D, dtype, "cpu", **kw)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return G.load()


def test_library_refuses_a_null_handle(lib):
    n = ctypes.c_int64()
    assert lib.spec_kv_append(None, None, 0, None, 0, None, 0, 1, 1, 1, 0, None, None, None, None,
                              None, 0.0, None, 0, 0, None, 0, None, None) == G.SPEC_ERR_ARG
    assert lib.spec_paged_attention_workspace(None, 1, 1, 1, 1, 1, 64,
                                              ctypes.byref(n)) == G.SPEC_ERR_ARG
    assert lib.spec_paged_attention(None, None, 0, 1, 1, 1, 1, 0, None, None, None, 1.0, 0, 0, None,
                                    None, None, None, 0, None) == G.SPEC_ERR_ARG
    assert lib.spec_token_logprobs(None, None, 1, 1, 1, 10, None, 1, None, 0, 1.0, None, None, 0,
                                   None, None, None, None) == G.SPEC_ERR_ARG


def test_cache_shapes():
    c = G.KvCache.empty(5, 4, 3, 96, torch.float16, "cpu", G.SPEC_KV_HND)
    assert (c.num_blocks, c.block_size, c.H, c.D, c.kind) == (5, 4, 3, 96, G.SPEC_CACHE_SAME)
    c = cache(torch.float8_e5m2)
    assert (c.num_blocks, c.block_size, c.H, c.D, c.kind) == (5, 4, 2, 64, G.SPEC_CACHE_FP8_E5M2)
    u8 = torch.zeros((5, 4, 2, 64), dtype=torch.uint8)
    assert G.KvCache(u8, u8, kind=G.SPEC_CACHE_FP8_E4M3).kind == G.SPEC_CACHE_FP8_E4M3
    both = bf(5, 2, 4, 2, 64)
    assert G.KvCache(both[:, 0], both[:, 1]).block_size == 4
    for kw, err in ((dict(layout=2), ValueError), (dict(kind=3), ValueError),
                    (dict(kind=G.SPEC_CACHE_FP8_E4M3), TypeError), (dict(v=bf(5, 4, 2, 32)), TypeError),
                    (dict(v=bf(5, 4, 2, 64).half()), TypeError), (dict(k_scale=f32(2)), TypeError),
                    (dict(k=u8, v=u8), TypeError), (dict(k=u8, v=u8, kind=0), TypeError),
                    (dict(k=bf(4, 2, 64), v=bf(4, 2, 64)), TypeError)):
        a = dict(k=bf(5, 4, 2, 64), v=bf(5, 4, 2, 64))
        a.update(kw)
        with pytest.raises(err):
            G.KvCache(**a)


@pytest.mark.parametrize("kw,err", [
    (dict(k=bf(6, 2, 32)), ValueError), (dict(v=bf(5, 2, 64)), ValueError),
    (dict(v=bf(6, 2, 64).half()), TypeError), (dict(q=bf(5, 4, 64)), ValueError),
    (dict(q_out=bf(6, 2, 64)), ValueError), (dict(q_out=None), ValueError),
    (dict(q_weight=bf(32), k_weight=bf(64)), ValueError), (dict(row_start=i32(2)), ValueError),
    (dict(row_start=i32(3).long()), TypeError), (dict(seq_pos=i32(2).long()), TypeError),
    (dict(inv_freq=f32(32).double()), TypeError), (dict(status=i32(3)), ValueError),
    (dict(cache=cache(torch.float16)), TypeError), (dict(block_table=i32(3, 4)), ValueError),
    (dict(block_table=i32(2, 4).long()), TypeError), (dict(), ValueError)])   # not CUDA tensors
def test_kv_append_refusals(kw, err):
    a = dict(q=bf(6, 4, 64), k=bf(6, 2, 64), v=bf(6, 2, 64), cache=cache(), block_table=i32(2, 4),
             seq_pos=i32(2), q_out=bf(6, 4, 64))
    a.update(kw)
    with pytest.raises(err):
        G.spec_kv_append(H, **a)


@pytest.mark.parametrize("kw,err", [
    (dict(q=bf(6, 4, 32)), ValueError), (dict(out=bf(6, 2, 64)), ValueError),
    (dict(out=bf(6, 4, 64).half()), TypeError), (dict(seq_pos=i32(2).long()), TypeError),
    (dict(row_start=i32(4)), ValueError), (dict(lse=f32(6, 2)), ValueError),
    (dict(lse=f32(6, 4).double()), TypeError), (dict(status=i32(3)), ValueError),
    (dict(cache=cache(torch.float16)), TypeError), (dict(), ValueError)])
def test_paged_attention_refusals(kw, err):
    a = dict(q=bf(6, 4, 64), cache=cache(), block_table=i32(2, 4), seq_pos=i32(2), scale=0.125,
             out=bf(6, 4, 64), workspace=torch.zeros(1024, dtype=torch.uint8))
    a.update(kw)
    with pytest.raises(err):
        G.spec_paged_attention(H, **a)


@pytest.mark.parametrize("kw,err", [
    (dict(node=i32(2, 3).long()), TypeError), (dict(node=i32(3, 3)), ValueError),
    (dict(tokens=i32(2, 4)), ValueError), (dict(logprob=f32(2, 4)), ValueError),
    (dict(logprob=None), ValueError), (dict(entropy=f32(3)), ValueError),
    (dict(top_ids=i32(2, 3, 5)), ValueError),
    (dict(top_ids=i32(2, 3, 5), top_logprobs=f32(2, 3, 4)), ValueError),
    (dict(flags=f32(2, 3)), TypeError), (dict(), ValueError)])
def test_token_logprobs_refusals(kw, err):
    a = dict(logits=f32(2, 7, 100), node=i32(2, 3), tokens=i32(2, 3), temperature=1.0,
             logprob=f32(2, 3))
    a.update(kw)
    with pytest.raises(err):
        G.spec_token_logprobs(H, **a)


# ---- the oracle ---------------------------------------------------------------------------------

def test_visible():
    assert S.visible(5, 8, 0, 0).tolist() == [True] * 6 + [False] * 2
    assert S.visible(5, 8, 2, 1).tolist() == [True] + [False] * 3 + [True] * 2 + [False] * 2
    assert S.visible(-1, 4, 0, 0).sum() == 0
    assert S.visible(9, 4, 3, 9).tolist() == [True] * 4


def test_attention_oracle_is_the_formula():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((2, 4, 8)), rng.standard_normal((6, 2, 8)), rng.standard_normal(
        (6, 2, 8))
    there = np.array([True, True, False, True, True, True])
    r = S.attention(q, k, v, [3, 5], there, 0.3, 2, 1)
    for i, keys in ((0, [0, 3]), (1, [0, 4, 5])):
        for h in range(4):
            w = np.exp([0.3 * float(q[i, h] @ k[j, h // 2]) for j in keys])
            want = sum(a * v[j, h // 2] for a, j in zip(w, keys)) / w.sum()
            np.testing.assert_allclose(r["out"][i, h], want, rtol=1e-12)
            np.testing.assert_allclose(r["lse"][i, h], np.log(w.sum()), rtol=1e-12)


def test_logprobs_oracle_is_the_formula():
    row = np.array([1.0, 3.0, -np.inf, 3.0, 0.5])
    r = S.logprobs(row, 2.0, [1, -1, 2, 7], 5)
    p = np.exp(row / 2) / np.exp(row / 2).sum()
    np.testing.assert_allclose(r["logprob"][0], np.log(p[1]))
    assert r["logprob"][1] == 0 and r["logprob"][2] == -np.inf and np.isnan(r["logprob"][3])
    assert r["ids"].tolist() == [1, 3, 0, 4, -1] and r["top"][4] == -np.inf
    assert r["flags"] == S.ROW_BAD_TOKEN
    np.testing.assert_allclose(r["entropy"], -(p[p > 0] * np.log(p[p > 0])).sum())
    assert S.logprobs(np.array([np.nan, 1.0]), 1.0, [0], 0)["flags"] == S.ROW_NAN
    assert S.logprobs(np.full(3, -np.inf), 1.0, [0], 0)["flags"] == S.ROW_ALL_NEGINF
