"""The tree-step oracle against closed forms and hand-worked values (CPU)."""
import numpy as np
import pytest

from oracle import tree_step as S


def test_rotation_turns_pairs_by_the_angle():
    x = np.zeros((1, 1, 1, 8))
    x[..., 0] = 1.0                                    # pair 0: (0, 4) halves, (0, 1) pairs
    f = np.float32([0.5, 0.25, 0.125])
    y = S.norm_rope(x[..., :6], None, 0.0, f, np.array([[3]]), pairs=False)
    assert np.allclose(y[0, 0, 0], [np.cos(1.5), 0, 0, np.sin(1.5), 0, 0])
    y = S.norm_rope(x, None, 0.0, f, np.array([[3]]), pairs=True)
    assert np.allclose(y[0, 0, 0], [np.cos(1.5), np.sin(1.5), 0, 0, 0, 0, 0, 0])


def test_rotation_keeps_relative_positions():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 1, 16))
    f = (100.0 ** -(np.arange(8) / 8)).astype(np.float32)
    dots = [(S.norm_rope(q, None, 0, f, np.array([[p + 5]]), False) *
             S.norm_rope(k, None, 0, f, np.array([[p]]), False)).sum() for p in (0, 7, 1000)]
    assert np.allclose(dots, dots[0], rtol=1e-9)


def test_norm_gives_unit_mean_square():
    x = np.random.default_rng(2).standard_normal((2, 3, 4, 32)) * 7
    y = S.norm_rope(x, np.ones(32), 0.0, np.float32([]), np.zeros((2, 3)), False)
    assert np.allclose((y * y).mean(-1), 1.0)


def test_e2m1_rounding_ties_to_even_codes():
    x = np.zeros(16, np.float32)
    x[:14] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.75, -5.0, 0.2501, 0.2499, 5.01, 4.99]
    codes, sf = S.quantise(x)                          # amax 6: scale 1
    assert S.E4M3[sf[0]] == 1.0
    assert codes.tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 10, 14, 1, 0, 7, 6, 0, 0]


def test_quantised_values_are_fixed_points_and_near():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((50, 64)) * 10.0 ** rng.uniform(-2, 2, (50, 1))).astype(np.float32)
    for ts in (1.0, 0.37):
        codes, sf = S.quantise(x, ts)
        v = S.values(codes, sf, ts)
        # half of the widest step (2 of 6) under a scale within half a step (2^-4) of amax / 6
        amax = np.abs(x.reshape(50, 4, 16)).max(-1, keepdims=True)
        bound = amax / 6 * (1 + 2.0 ** -4) * 1.0 + amax * 2.0 ** -4
        assert np.all(np.abs(v - x).reshape(50, 4, 16) <= bound)
        c2, s2 = S.quantise(v.astype(np.float32), ts)
        if ts == 1.0:
            full = np.abs(S.E2M1[codes & 7]).reshape(50, 4, 16).max(-1) == 6
            assert np.array_equal(S.values(c2, s2, ts).reshape(50, 4, 16)[full],
                                  v.reshape(50, 4, 16)[full])


def test_special_blocks():
    x = np.zeros((4, 16), np.float32)
    x[1, 3] = np.nan
    x[2, 0], x[2, 1] = np.inf, 1.0
    x[3] = 1e-12                                       # below the smallest scale: zeros
    codes, sf = S.quantise(x)
    v = S.values(codes, sf)
    assert np.all(v[0] == 0) and np.all(np.isnan(v[1])) and np.all(v[3] == 0)
    assert v[2, 0] == 448 * 6 and v[2, 1] == 0
    assert np.array_equal(S.unpack(S.pack(codes)), codes)


@pytest.mark.parametrize("ctx", [0, 1, 5])
def test_attention_by_enumeration(ctx):
    rng = np.random.default_rng(4)
    N, Hq, H, D = 3, 4, 2, 16
    q, tk, tv = (rng.standard_normal(s) for s in ((N, Hq, D), (N, H, D), (N, H, D)))
    k, v = rng.standard_normal((2, ctx, H, D))
    mask = np.array([1, 3, 0], np.uint64)              # node 2 sees no node, not even itself
    out, lse, _, _ = S.attend(q, tk, tv, k, v, mask, 0.25)
    for n in range(N):
        for h in range(Hq):
            rows = [(k[t, h // 2], v[t, h // 2]) for t in range(ctx)] + \
                [(tk[j, h // 2], tv[j, h // 2]) for j in range(N) if int(mask[n]) >> j & 1]
            w = np.array([np.exp(0.25 * (q[n, h] * a).sum()) for a, _ in rows])
            if not rows:
                assert np.all(out[n, h] == 0) and lse[n, h] == -np.inf
                continue
            assert np.allclose(out[n, h], sum(x * b for x, (_, b) in zip(w, rows)) / w.sum())
            assert np.isclose(lse[n, h], np.log(w.sum()))
