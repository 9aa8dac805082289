"""Angles of far positions and of any frequency, against whole-number arithmetic.

Bounds.  The pair (1, 0) turns into (cos, sin).  The angle is off by 2^-28 of a
turn where it is rounded to float32 and by 2^-32 before: 2 pi (2^-28 + 2^-32) <
2^-25.  The series leave out 2^-28, their first terms and coefficients, of values
below 0.31, round by 2^-25 in all, and their sum rounds by 2^-25.  Together less
than 2^-23.
"""
import math
from fractions import Fraction

import pytest
import torch

from block_sparse_masked_blockmask_gb300 import flexattn as fa

pytestmark = pytest.mark.gpu
BITS = 320


def arctan_of_inverse(n):
    """arctan(1 / n) in units of 2^-BITS."""
    power, total, k, sign = (1 << BITS) // n, 0, 1, 1
    while power:
        total += sign * (power // k)
        power, k, sign = power // (n * n), k + 2, -sign
    return total


PI = Fraction(4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239)), 1 << BITS)
FREQUENCIES = [0.7499, 1.0, 0.1, -0.3, 10000.0 ** (-2 / 128), 10000.0 ** (-126 / 128), 500000.0 ** (-62 / 64), 1e-7, -1e-20,
               1e-300, 0.0, math.pi, 2 * math.pi, 99.9, 1000.7, 2.0**20 / 3, -(2.0**39) / 7]
POSITIONS = [0, 1, -1, 7, 4095, 131071, 1048577, 2**30 + 3, 2**31 - 1, -(2**31), -(2**31) + 5, 123456789, -987654321]


@pytest.mark.parametrize("layout", [fa.FLEX_ROPE_HALF, fa.FLEX_ROPE_INTERLEAVED])
def test_angles(layout):
    S, n = len(POSITIONS), 32
    f = (FREQUENCIES * 2)[:n]
    x = torch.zeros((1, 1, S, 64))
    x[..., :n if layout == fa.FLEX_ROPE_HALF else None:1 if layout == fa.FLEX_ROPE_HALF else 2] = 1.0
    at = torch.tensor(POSITIONS, dtype=torch.int32, device="cuda")[None]
    inv = torch.tensor(f, dtype=torch.float64, device="cuda")
    y, _ = fa.flex_rope_fwd(x.cuda(), None, inv, at, layout=layout)
    back, _ = fa.flex_rope_bwd(x.cuda(), None, inv, at, layout=layout)
    for y, sign in ((y, 1), (back, -1)):
        y = y[0, 0].double().cpu()
        cos, sin = (y[:, :n], y[:, n:]) if layout == fa.FLEX_ROPE_HALF else (y[:, 0::2], y[:, 1::2])
        for s, p in enumerate(POSITIONS):
            for i, w in enumerate(f):
                turns = Fraction(w) * p / (2 * PI)
                angle = 2 * math.pi * float(turns - math.floor(turns))
                assert abs(float(cos[s, i]) - math.cos(angle)) < 2.0**-23, (p, w)
                assert abs(float(sin[s, i]) - sign * math.sin(angle)) < 2.0**-23, (p, w)
