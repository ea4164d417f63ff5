"""Angles of positions beyond 2^39: the frequency is held in multiples of 2^-64 of a turn, so the
angle is off by up to the position times that, and by no more."""
import math
from fractions import Fraction

import numpy as np
import pytest

from tests.gpu_util import tensor_f64

pytestmark = pytest.mark.gpu
# from pi's published digits
PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923, 10**64)


@pytest.mark.parametrize("freq", [1.0, -1.0, 0.75, 1e-4, 2.5, 30.0, 1000.0])
@pytest.mark.parametrize("position", [2**39, 2**44 + 12345, 2**50 - 1, -(2**53) - 7, 2**60, 2**62 + 3])
def test_far_positions_within_the_bound(position, freq):
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q = torch.zeros(1, 1, 8, device="cuda")
    q[..., :4] = 1.0
    inv = torch.tensor([freq, freq / 4, freq / 16, 0.0], dtype=torch.float64)
    y, _ = B.flce_rope_forward(q, q, inv.cuda(), torch.tensor([position], device="cuda"))
    y = tensor_f64(y).reshape(2, 4)  # cosines, sines
    for j, f in enumerate(inv.tolist()):
        angle = 2 * math.pi * float(Fraction(f) * position / (2 * PI) % 1)
        # less than one multiple is cut off, and the constant 2^66 / 2 pi, rounded up to an integer, is
        # 0.02 too large; from 4 on each doubling of the frequency doubles both
        off = 2 * math.pi * abs(position) * 2.0**-64 * max(1.0, abs(f) / 2) * 1.02
        got = math.atan2(y[1, j], y[0, j])
        diff = abs((got - angle + math.pi) % (2 * math.pi) - math.pi)
        assert diff <= off + 1e-6, (position, f, diff, off)
        assert np.hypot(*y[:, j]) == pytest.approx(1.0, abs=1e-6)
