"""On the CPU: differences along the gradient tell a wrong gradient apart."""

import numpy as np
import pytest

from score_differences import SHARP, along_the_gradient, sharp


@pytest.mark.parametrize("case", SHARP)
def test_differences_tell_a_wrong_gradient(case):
    """What rounding may take is a small part of the slope, so that a gradient
    that is zero, of the other sign, or a tenth too small is told apart."""
    q, k, v, do, kw, cap = sharp(**case)
    rows, b = along_the_gradient(q, k, v, do, kw, cap)
    for n, step, slope, room in rows:
        assert room < 0.05 * abs(slope), (n, room / slope)
        g = b["d" + n]
        assert abs(np.sum(g * step) - slope) <= 1e-5 * abs(slope)
        for wrong in (0 * g, -g, 0.9 * g):
            assert abs(np.sum(wrong * step) - slope) > room
