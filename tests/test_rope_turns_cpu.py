"""The fractions of a turn that the rotary table holds, against exact arithmetic, to the bound that pagedkv.h states."""
from fractions import Fraction

import numpy as np
import pytest

from test_tree_cpu import _pkv

# 2 pi to 60 digits
TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


def turns(f):
    pkv = _pkv()
    f = np.ascontiguousarray(np.asarray(f, dtype=np.float64))
    out = np.empty(len(f), dtype=np.uint64)
    assert pkv.lib().pkv_rope_turns(out.ctypes.data, f.ctypes.data, len(f)) == 0
    return [int(t) for t in out]


@pytest.mark.parametrize("base", [10000.0, 500000.0, 2.0 ** 40])
@pytest.mark.parametrize("position", [1, 131071, 999_999, (1 << 31) + 5, (1 << 40) + 3, (1 << 50) + 1, -4097])
def test_angle_of_a_position(base, position):
    """position * turns mod 2^64 is off by at most |position| * (2^-52 f / 2 pi + 2^-64) turns: two roundings of the quotient
    f / 2 pi (2 pi's own and the division's, 2^-54 and 2^-53 of it), and the cut to 64 bits."""
    f = base ** (-np.arange(0, 128, 2, dtype=np.float64) / 128)
    for x, t in zip(f, turns(f)):
        exact = position * Fraction(float(x)) / TWO_PI
        got = Fraction(position * t % (1 << 64), 1 << 64)
        off = (got - exact) % 1
        off = min(off, 1 - off)
        assert off <= abs(position) * (Fraction(float(x)) / TWO_PI / (1 << 52) + Fraction(1, 1 << 64)), (x, position)
