"""A tree attention whose warps give up waiting for one another says so (needs a GB300). The debug
flavour gives all waits up before any product is issued: nothing hangs, faults or runs on."""
import numpy as np
import pytest
import torch

import test_gpu_tree_step as T
from oracle import tree_step as S
from speculative_decoding_tree_mask_gb300 import binding as G
from speculative_decoding_tree_mask_gb300 import build as Build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    with G.use_library(Build.build(debug=True)):
        with G.Handle(64, 64, 1 << 10, 0) as handle:
            yield handle


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("N,Gq,D", [(40, 2, 64), (64, 1, 128), (64, 4, 128), (64, 4, 64)])
def test_lost_results_are_not_numbers(h, dt, N, Gq, D):
    """Whole items and cut ones, with and without a context: every row is NaN and every request
    has its status, a request with a bad page too; the next call is as ever."""
    rng = np.random.default_rng(N + D)
    c = T.Case(rng, 3, N, 2, Gq, D, dt, S.NHD, 16, [3000, 0, 50])
    c.table[2, 1] = -1
    st = torch.full((3,), 9, dtype=torch.int32, device=T.DEV)
    G.spec_debug_inject_lost_wait(h)
    out, lse = c.run(h, status=st)
    assert st.tolist() == [G.SPEC_REQ_INTERNAL] * 3
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    out, lse = c.run(h, status=st)
    assert st.tolist() == [0, 0, S.BAD_SLOT]
    T.check_attention(out, lse, c.requests(), c.scale, dt)


def test_a_call_of_few_rows_has_no_such_waits(h):
    """The injection is for one call, whichever kernel it runs on."""
    rng = np.random.default_rng(3)
    c = T.Case(rng, 2, 4, 2, 2, 64, "bf16", S.NHD, 16, [300, 20])
    big = T.Case(rng, 2, 40, 2, 2, 64, "bf16", S.NHD, 16, [300, 20])
    st = torch.full((2,), 9, dtype=torch.int32, device=T.DEV)
    G.spec_debug_inject_lost_wait(h)
    for x in (c, big):
        out, lse = x.run(h, status=st)
        assert st.tolist() == [0, 0]
        T.check_attention(out, lse, x.requests(), x.scale, "bf16")
