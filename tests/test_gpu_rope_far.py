"""Rotations at far positions against exact angles, to the error that pagedkv.h states for the table of frequencies."""
import math
from fractions import Fraction

import pytest
import torch

pytestmark = pytest.mark.gpu

TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
FAR = [0, 1, 131071, 999_999, (1 << 31) + 5, (1 << 36) + 11, (1 << 40) + 3, -4097, -(1 << 40)]


@pytest.mark.parametrize("base", [10000.0, 500000.0])
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(base, interleaved):
    """Beside the table's |position| (2^-52 f + 2^-61): the turn's fraction in 32 bits (2^-25 half turns), the sine and the
    cosine (2 units in the last place: 2^-22 together with it, in radians 2^-21), three fp32 roundings; each of both elements of
    a pair."""
    import paged_kv_gqa_03_gb300 as pkv
    D = 128
    x = torch.randn(len(FAR), 3, D, generator=torch.Generator().manual_seed(1))
    table = pkv.RopeTable(D, base=base, interleaved=interleaved)
    out = torch.empty_like(x, device="cuda")
    pkv.paged_rope(x.cuda(), None, torch.tensor(FAR).cuda(), table, q_out=out)
    out, y = out.cpu().double(), x.double()
    pairs = (lambda t: (t[..., 0::2], t[..., 1::2])) if interleaved else (lambda t: (t[..., :D // 2], t[..., D // 2:]))
    a, b = pairs(y)
    got_a, got_b = pairs(out)
    for t, position in enumerate(FAR):
        for i, f in enumerate(table.frequencies):
            turn = float(position * Fraction(float(f)) / TWO_PI % 1)
            c, s = math.cos(2 * math.pi * turn), math.sin(2 * math.pi * turn)
            off = abs(position) * (f * 2.0 ** -52 + 2.0 ** -61) + 2.0 ** -21 + 3 * 2.0 ** -24
            tol = off * (a[t, :, i].abs() + b[t, :, i].abs())
            assert ((got_a[t, :, i] - (a[t, :, i] * c - b[t, :, i] * s)).abs() <= tol).all(), (position, i)
            assert ((got_b[t, :, i] - (b[t, :, i] * c + a[t, :, i] * s)).abs() <= tol).all(), (position, i)
