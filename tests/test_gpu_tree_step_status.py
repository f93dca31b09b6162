"""The convenience calls of the tree step tell what a request met (needs a GB300)."""
import numpy as np
import pytest
import torch

import test_gpu_tree_step as T
from oracle import tree_step as S
from speculative_decoding_tree_mask_gb300 import binding as G

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("N", [3, 64])
def test_status_of_the_convenience_calls(N):
    rng = np.random.default_rng(91)
    c = T.Case(rng, 4, N, 1, 4, 128, "bf16", S.NHD, 16, [100, 100, 100, 112])
    c.table[1, 2] = c.cache.num_blocks          # a page outside the cache
    c.ctx[2] = -1                               # a length below zero
    c.ctx[3] = 113                              # a length past the table
    st = torch.full((4,), 9, dtype=torch.int32, device=DEV)
    with G.Handle(4, 64, 16, 0) as h:
        c.run(h, status=st)
        want = [0, S.BAD_SLOT, S.BAD_SLOT, S.BAD_SLOT]
        assert st.tolist() == want
        st.fill_(9)
        G.kv_load_fp4(h, c.cache, T.gpu(c.table), T.gpu(np.zeros(4, np.int32)), T.gpu(c.ctx), 112,
                      status=st)
        assert st.tolist() == want
