"""Paged attention at the edges of what a call may say (needs a GB300). Tolerances are those of
test_gpu_paged_attention, whose cases these are built from."""
import numpy as np
import pytest
import torch

import test_gpu_paged_attention as T
from oracle import paged_step as S
from speculative_decoding_tree_mask_gb300 import binding as G

pytestmark = pytest.mark.gpu
DEV = T.DEV


@pytest.fixture(scope="module")
def h():
    G.load()
    with G.Handle(4096, 64, 1 << 10, 0) as handle:
        yield handle


def cut_table(c, pages):
    """The first `pages` of each request's table, and of what the oracle knows."""
    c.table = np.ascontiguousarray(c.table[:, :pages])
    for all_ in (c.k64, c.v64):
        all_[:] = [x[:pages * c.bs] for x in all_]


# ---- positions past the table -------------------------------------------------------------------

@pytest.mark.parametrize("dt,cache", [("bf16", "same"), ("f16", "e4m3")])
@pytest.mark.parametrize("n,Gq,D", [(8, 2, 64), (8, 2, 128), (8, 1, 256), (80, 2, 64), (150, 2, 128),
                                    (80, 2, 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (4, 0), (4, 3), (40, 1), (100, 0), (3, 500)])
def test_windows_of_rows_past_the_table(h, dt, cache, n, Gq, D, window, sinks):
    """A row whose position the table does not have sees the window that ends with that position, as
    far as the table goes, and the sinks; rows whose whole window is past it see nothing else."""
    rng = np.random.default_rng(D + n)
    pos = [254, 250 - n, 300]             # the table ends at 256: all but two rows, some, all
    c = T.Case(rng, [n] * 3, pos, 2, Gq, D, dt, cache, S.HND, 16, window, sinks)
    cut_table(c, 16)
    st = torch.full((3,), 9, dtype=torch.int32, device=DEV)
    out, lse = c.run(h, st)
    assert st.tolist() == [S.BAD_SLOT, 0, S.BAD_SLOT]
    c.check(out, lse)


@pytest.mark.parametrize("n,Gq", [(8, 2), (80, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (2 ** 31 - 1, 0), (2 ** 31 - 1, 5), (2 ** 31 - 100, 0),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (7, 2)])
def test_positions_near_two_to_the_31(h, n, Gq, window, sinks):
    """Positions up to and beyond 2^31 and windows as large: sums of the two stay exact."""
    rng = np.random.default_rng(n)
    c = T.Case(rng, [n, n], [100, 200], 2, Gq, 64, "bf16", "same", S.NHD, 16, window, sinks)
    cut_table(c, 6)
    c.pos = [2 ** 31 - 1, 2 ** 31 - 4]
    st = torch.full((2,), 9, dtype=torch.int32, device=DEV)
    out, lse = c.run(h, st)
    assert st.tolist() == [S.BAD_SLOT, S.BAD_SLOT]
    c.check(out, lse)


# ---- rows that are not a request's ---------------------------------------------------------------

@pytest.mark.parametrize("dt,cache", [("bf16", "same"), ("f16", "same"), ("bf16", "e4m3")])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,Gq", [(21, 2), (67, 4)])
@pytest.mark.parametrize("value", [float("nan"), 1e30, float("inf")])
def test_queries_of_others_change_nothing(h, dt, cache, D, n, Gq, value):
    """A request's results are the same bits whatever stands in the rows behind it, those of no
    request and those of the next."""
    c = T.Case(np.random.default_rng(D), [n, n], [400, 30], 2, Gq, D, dt, cache, spare=70)
    c.q[2 * n:] = 0
    first = c.run(h)
    c.q[2 * n:] = value
    again = c.run(h)
    assert all(torch.equal(x[:2 * n], y[:2 * n]) for x, y in zip(first, again))
    c.check(*again)
    c.q[n:2 * n] = value
    again = c.run(h)
    assert all(torch.equal(x[:n], y[:n]) for x, y in zip(first, again))


# ---- infinities in many short parts ---------------------------------------------------------------

@pytest.mark.parametrize("D,n,Gq", [(64, 40, 1), (128, 40, 1), (128, 70, 2), (256, 40, 1)])
def test_infinities_in_short_items(h, D, n, Gq):
    """Thousands of items of a tile each, dealt several to a CTA, an infinity that the last row alone
    sees in every third request: it is in that row's element and nowhere else."""
    B, bs = 4000, 128
    g = torch.Generator(device=DEV)
    g.manual_seed(D)
    k, v = (torch.randn((B, bs, 1, D), generator=g, device=DEV).half() for _ in range(2))
    pos = torch.randint(0, bs - n + 1 - n, (B,), generator=g, device=DEV) if bs >= 2 * n else \
        torch.zeros(B, dtype=torch.int64, device=DEV)
    b = torch.arange(0, B, 3, device=DEV)
    v[b, pos[b] + n - 1, 0, b % D] = float("inf")
    q = torch.randn((B * n, Gq, D), generator=g, device=DEV).half()
    table = torch.arange(B, dtype=torch.int32, device=DEV)[:, None]
    want = torch.zeros((B, n, Gq, D), dtype=torch.bool, device=DEV)
    want[b, n - 1, :, b % D] = True
    for _ in range(5):
        out, _ = G.paged_attention(h, q, G.KvCache(k, v), table, pos.int(), D ** -0.5, max_new=n)
        assert torch.equal(torch.isposinf(out.view(B, n, Gq, D)), want)
        assert torch.equal(torch.isfinite(out.view(B, n, Gq, D)), ~want)


# ---- alignment ------------------------------------------------------------------------------------

@pytest.mark.parametrize("dt,cache", [("bf16", "same"), ("f16", "e5m2")])
@pytest.mark.parametrize("counts,Gq,D", [([3, 1], 2, 64), ([1], 4, 96), ([2], 2, 256), ([70, 2], 2, 64),
                                         ([200], 2, 128), ([50, 1], 3, 80), ([60], 1, 256)])
@pytest.mark.parametrize("q_off,out_off", [(1, 1), (4, 4), (8, 8), (0, 3), (5, 0)])
def test_queries_and_results_at_any_address(h, dt, cache, counts, Gq, D, q_off, out_off):
    """Queries whose rows begin off 16-byte boundaries, and an output that begins anywhere; what is
    beside it stays."""
    rng = np.random.default_rng(q_off)
    c = T.Case(rng, counts, [500, 40][:len(counts)], 2, Gq, D, dt, cache, pad=16)
    wide = torch.zeros((len(c.q), c.Hq * D + 16 + q_off % 2), dtype=c.q.dtype, device=DEV)
    wide[:, q_off:q_off + c.Hq * D] = c.q.flatten(1)
    c.q = wide[:, q_off:q_off + c.Hq * D].unflatten(1, (c.Hq, D))
    n = c.q.numel()
    flat = torch.full((n + 32,), 7.0, dtype=c.q.dtype, device=DEV)
    out = flat[out_off:out_off + n].view(c.q.shape)
    lse = torch.empty(c.q.shape[:2], device=DEV)
    size = G.spec_paged_attention_workspace(h, len(counts), len(c.q), 0, c.Hq, 2, D)
    work = torch.empty(size, dtype=torch.uint8, device=DEV)
    G.spec_paged_attention(h, c.q, c.cache(), T.gpu(c.table), T.gpu(np.array(c.pos, np.int32)), c.scale,
                           out, work, T.gpu(c.start), lse=lse)
    c.check(out, lse)
    assert (flat[:out_off] == 7).all() and (flat[out_off + n:] == 7).all()
