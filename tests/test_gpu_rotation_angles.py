"""The sines and cosines of spec_qk_norm_rope against angles reduced in exact integers (needs a
GB300): rows of (1, 0) pairs come out as (cos, sin)."""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_tree_mask_gb300 import binding as G

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BITS = 256


def _arctan_inverse(n):
    """arctan(1/n) times 2^(BITS + 32), by its power series."""
    term = (1 << (BITS + 32)) // n
    total, k = term, 1
    while term:
        term //= -n * n
        k += 2
        total += term // k
    return total


# Machin's formula
PI = (16 * _arctan_inverse(5) - 4 * _arctan_inverse(239)) >> 32


def turns(pos, f):
    """pos * f / (2 pi) modulo 1, in [-1/2, 1/2], from exact integers."""
    num, den = float(f).as_integer_ratio()
    scaled = ((pos * num) << (2 * BITS)) // (den * 2 * PI)      # in units of 2^-BITS
    part = scaled & ((1 << BITS) - 1)
    if part >> (BITS - 1):
        part -= 1 << BITS
    return part / 2.0 ** BITS


@pytest.mark.parametrize("D,rot,pairs", [(128, 128, False), (128, 128, True), (128, 90, False),
                                         (33, 32, False)])
@pytest.mark.parametrize("largest", [1.0, 40.0])
def test_cosines_and_sines(D, rot, pairs, largest):
    """The turn errs by |position| (|inv_freq| + 1) 2^-64 and 2^-34; its float32 by 2^-24 of at
    most an eighth turn, sincospif by a step (2^-23): below 2^-22 of the value together."""
    rng = np.random.default_rng(rot + int(largest))
    half, B, N = rot // 2, 4, 64
    f = (largest * 10000.0 ** -rng.uniform(0, 1, half)).astype(np.float32)
    f[0] = largest
    f[1] = -f[1]
    pos = np.int32([0, 1000, 1 << 20, (1 << 31) - 1 - 3 * N])
    depth = rng.integers(0, 3 * N, (B, N)).astype(np.int32)
    a = np.arange(half) * (2 if pairs else 1)
    c = a + (1 if pairs else half)
    x = torch.zeros((B, N, 1, D), device=DEV)
    x[..., torch.from_numpy(a)] = 1.0
    with G.Handle(B, 64, 64, 0) as h:
        y, k = G.qk_norm_rope(h, x, x, torch.from_numpy(f).to(DEV), torch.from_numpy(pos).to(DEV),
                              torch.from_numpy(depth).to(DEV),
                              style=G.SPEC_ROPE_PAIRS if pairs else G.SPEC_ROPE_HALVES)
        assert torch.equal(y, k)
        y = y[:, :, 0].double().cpu().numpy()
    for b in range(B):
        for n in range(N):
            p = int(pos[b]) + int(depth[b, n])
            t = np.array([turns(p, v) for v in f])
            err = 2 * math.pi * (2.0 ** -34 + abs(p) * (np.abs(f) + 1) * 2.0 ** -64)
            for got, ref in ((y[b, n, a], np.cos(2 * math.pi * t)),
                             (y[b, n, c], np.sin(2 * math.pi * t))):
                tol = 2.0 ** -22 * np.abs(ref) + err + 2.0 ** -50
                assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / tol)
