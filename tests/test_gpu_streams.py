"""Convenience calls on a stream of their own beside a busy current stream (needs a GB300)."""
import numpy as np
import pytest
import torch

import test_gpu_tree_step as T
from oracle import tree_step as S
from speculative_decoding_tree_mask_gb300 import binding as G

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BUSY = 40_000_000     # clocks: about 20 ms


@pytest.fixture(scope="module")
def calls():
    rng = np.random.default_rng(5)
    c = T.Case(rng, 4, 40, 2, 2, 64, "bf16", S.NHD, 16, [600, 0, 1, 333])
    table, ctx, mask = T.gpu(c.table), T.gpu(c.ctx), T.gpu(c.mask.view(np.int64))
    zero = T.gpu(np.zeros(4, np.int32))
    freq = T.gpu(np.float32([1.0, 0.1, 0.01, 0.001]))
    logits, _ = T.rows(rng, 4, 40, 1, 512, "bf16")
    logits = logits.view(4, 40, 512)
    token = T.gpu(rng.integers(0, 512, (4, 40)).astype(np.int32))
    parent = T.gpu(np.tile(np.arange(-1, 39, dtype=np.int32), (4, 1)))
    with G.Handle(4, 40, 512, 0) as h:
        yield {
            "attend": lambda s: G.tree_attention_fp4(h, c.q, c.tk, c.tv, c.cache, table, ctx, mask,
                                                     c.scale, stream=s),
            "load": lambda s: G.kv_load_fp4(h, c.cache, table, zero, ctx, 600, stream=s),
            "rope": lambda s: G.qk_norm_rope(h, c.q, c.tk, freq, ctx, stream=s),
            "mask": lambda s: G.build_tree_mask(h, parent, stream=s).values(),
            "greedy": lambda s: G.verify_greedy(h, logits, token, parent, stream=s).values()}


@pytest.mark.parametrize("name", ["attend", "load", "rope", "mask", "greedy"])
def test_memory_that_the_current_stream_has_still_to_write(calls, name):
    """Blocks of every output's and of the workspace's size are freed with writes to them still
    to run on the current stream: the call on another stream does not take them."""
    call = calls[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        sizes = [t.numel() * t.element_size() for t in want] * 2 + [1 << 22, 1 << 24, 1 << 25]
        blocks = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]
        torch.cuda._sleep(BUSY)
        for b in blocks:
            b.fill_(0x7F)
        del blocks, b
        got = list(call(s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del got


@pytest.mark.parametrize("name", ["attend", "load", "rope", "mask", "greedy"])
def test_results_freed_while_the_current_stream_has_still_to_read_them(calls, name):
    call = calls[name]
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = list(call(s))
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(BUSY)
        kept = [t.clone() for t in got]
        del got
        with torch.cuda.stream(s):
            for t in want:                  # what the next calls on s write
                torch.empty_like(t).fill_(3)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))
