"""A paged attention whose warps give up waiting for one another says so (needs a GB300). The debug
flavour gives all waits up before any product is issued: nothing hangs, faults or runs on."""
import numpy as np
import pytest
import torch

import test_gpu_paged_attention as T
from oracle import paged_step as S
from speculative_decoding_tree_mask_gb300 import binding as G
from speculative_decoding_tree_mask_gb300 import build as Build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    with G.use_library(Build.build(debug=True)):
        with G.Handle(64, 64, 1 << 10, 0) as handle:
            yield handle


@pytest.mark.parametrize("dt,cache", [("bf16", "same"), ("f16", "e4m3")])
@pytest.mark.parametrize("Gq,D", [(2, 64), (4, 128), (2, 256)])
def test_lost_results_are_not_numbers(h, dt, cache, Gq, D):
    """Whole items and cut ones: every row is NaN and every request has its status; the next call is
    as ever."""
    c = T.Case(np.random.default_rng(D), [90, 40, 130], [3000, 0, 50], 2, Gq, D, dt, cache)
    st = torch.full((3,), 9, dtype=torch.int32, device=T.DEV)
    G.spec_debug_inject_lost_wait(h)
    out, lse = c.run(h, st, max_new=260 // 3 + 100)
    torch.cuda.synchronize()
    assert st.tolist() == [G.SPEC_REQ_INTERNAL] * 3
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    out, lse = c.run(h, st)
    assert st.tolist() == [0, 0, 0]
    c.check(out, lse)
    assert S.BAD_SLOT != G.SPEC_REQ_INTERNAL
