"""New tokens into the paged cache at the edges of what a call may say (needs a GB300)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import paged_step as S
from speculative_decoding_tree_mask_gb300 import binding as G

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def h():
    G.load()
    with G.Handle(2048, 64, 1 << 10, 0) as handle:
        yield handle


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


# ---- row_start that falls or leaves the rows ------------------------------------------------------

def dealt(start, T):
    """Request of each row, -1 for none; status of each request. Row ranges do not meet."""
    owner, status = np.full(T, -1), np.zeros(len(start) - 1, int)
    for b, (s, e) in enumerate(zip(start[:-1], start[1:])):
        if s < 0 or e > T or s > e:
            status[b] = S.BAD_RANGE
        else:
            assert (owner[s:e] == -1).all()
            owner[s:e] = b
    return owner, status


@pytest.mark.parametrize("T,start", [
    (8, [0, 3, 100, 3, 8]), (8, [0, 3, -1, 3, 8]), (8, [0, 2, 8, 5, 5]), (8, [9, 0, 3, 8, 8]),
    (8, [-5, 0, 8, 20, -7]), (12, [0, 4, 90, 4, 4, 9, -3, 9, 12]), (6, [100, 100, 100]),
    (300, list(range(0, 151)) + [999] + list(range(151, 301))),
    (300, [999 if b % 3 == 2 else b - (b + 1) // 3 for b in range(451)])])
def test_valid_requests_beside_bad_ones(h, T, start):
    """Every request whose own rows are within those given takes part, whatever stands beside it;
    the others' rows are left and reported."""
    start = np.array(start, np.int32)
    B = len(start) - 1
    owner, status = dealt(start, T)
    k = torch.randn((T, 1, 64), device=DEV).half()
    q = torch.randn((T, 2, 64), device=DEV).half()
    bs = 16 if T < 100 else 64
    cache = G.KvCache.empty(B, bs, 1, 64, torch.float16, DEV)
    qo = torch.full_like(q, 7.0)
    st = torch.full((B,), 9, dtype=torch.int32, device=DEV)
    G.spec_kv_append(h, q, k, k, cache, gpu(np.arange(B, dtype=np.int32)[:, None]),
                     gpu(np.full(B, 1, np.int32)), qo, gpu(start), status=st)
    assert st.tolist() == status.tolist()
    want = torch.zeros_like(cache.k)
    for r, b in enumerate(owner):
        if b >= 0:
            want[b, 1 + r - start[b]] = k[r]
    assert torch.equal(cache.k, want) and torch.equal(cache.v, want)
    mine = gpu(owner >= 0)
    assert torch.equal(qo[mine], q[mine]) and (qo[~mine] == 7).all()


# ---- no rows --------------------------------------------------------------------------------------

@pytest.mark.parametrize("B", [0, 1, 3])
@pytest.mark.parametrize("queries", [True, False])
@pytest.mark.parametrize("given", [True, False])
def test_no_rows(h, B, queries, given):
    """Nothing is launched and the statuses are 0, with and without queries."""
    cache = G.KvCache.empty(4, 16, 2, 64, torch.bfloat16, DEV)
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device=DEV) if queries else None
    k = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    st = torch.full((B,), 9, dtype=torch.int32, device=DEV)
    zeros = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    qo = G.kv_append(h, q, k, k, cache, torch.zeros((B, 4), dtype=torch.int32, device=DEV), zeros[:B],
                     zeros if given else None, torch.ones(32, device=DEV), status=st)
    assert (qo.shape == q.shape) if queries else qo is None
    assert st.tolist() == [0] * B and not cache.k.any()


# ---- refusals at the C entry ------------------------------------------------------------------------

@pytest.mark.parametrize("rot,want", [(63, G.SPEC_ERR_ARG), (65, G.SPEC_ERR_ARG), (-2, G.SPEC_ERR_ARG),
                                      (66, G.SPEC_ERR_ARG), (64, 0)])
def test_rotated_elements(h, rot, want):
    """An odd, negative or too large number of rotated elements is refused."""
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device=DEV)
    cache = G.KvCache.empty(4, 16, 2, 64, torch.bfloat16, DEV)
    table, pos = (torch.zeros(s, dtype=torch.int32, device=DEV) for s in ((2, 4), (2,)))
    freq = torch.zeros(64, device=DEV)
    view = cache.struct(table, 2, 0, torch.bfloat16)
    rc = G.load().spec_kv_append(
        h.ptr, x.data_ptr(), 128, x.data_ptr(), 128, x.data_ptr(), 128, G.SPEC_BF16, 2, 2, 2, None,
        pos.data_ptr(), ctypes.byref(view), None, None, 1e-6, freq.data_ptr(), rot, 0, x.data_ptr(), 128,
        None, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == want
