"""Log probabilities of the longest rows that a CTA takes alone (needs a GB300). Tolerances are those
of test_gpu_token_logprobs."""
import numpy as np
import pytest
import torch

import test_gpu_token_logprobs as T
from speculative_decoding_tree_mask_gb300 import binding as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    G.load()
    with G.Handle(64, 64, 1 << 21, 0) as handle:
        yield handle


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("top", [0, 20])
def test_longest_rows_of_one_cta(h, dt, top):
    """2^21 logits in so many slots that a row has a CTA of its own: 2^13 of them a thread."""
    V, P = 1 << 21, 1000
    rng = np.random.default_rng(top)
    t, x = T.rows(rng, 1, 2, V, dt)
    node = (np.arange(P) % 2).astype(np.int32)[None]
    tokens = np.repeat(rng.integers(0, V, (1, 2)).astype(np.int32), P // 2, 0).reshape(1, P)
    got = G.token_logprobs(h, t, T.gpu(tokens), T.gpu(node), top=top)
    T.check({k: v[:, :2] for k, v in got.items()}, x, node[:, :2], tokens[:, :2], 1.0, top)
    for k, v in got.items():
        assert torch.equal(v, v[:, :2].repeat(1, P // 2, *[1] * (v.dim() - 2))), k
