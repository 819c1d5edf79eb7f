"""Factors of the scores (scale, the keys' unit, a power of two per bf16 query row) whose product leaves 32 bits'
normal numbers, above or below, while each of them is allowed."""
import math

import pytest
import torch

from test_gpu_kv4_attention import Case, pkv  # noqa: F401
from test_gpu_kv4_large_scores import check, exact_case

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_len,Hq", [(1, 8), (4, 8)])
@pytest.mark.parametrize("reach,unit,scale", [(2.0 ** -72, 2.0 ** -64, None), (2.0 ** -60, 1.0, 1e-30), (2.0 ** -120, 1.0, 1e-4)])
def test_scores_of_almost_nothing(pkv, D, q_len, Hq, reach, unit, scale):  # noqa: F811
    """All weights alike; contexts and windows that end inside a tile, and rows that see nothing."""
    c = Case(pkv, [100, 31, 500, 2000, 1, 0], q_len, Hq, 2, D, BF16, seed=6, unit=(unit, 1.0))
    q = (c.q.float() * reach).to(BF16)
    scale = c.scale if scale is None else scale
    for window in (0, 50):
        out = c.check(window=window, q=q, scale=scale, four=True)
        assert torch.isfinite(out).all()


@pytest.mark.parametrize("lens", [[100, 31, 260], [9000, 333]])
@pytest.mark.parametrize("scale", [1e15, 1e30])
def test_scores_beyond_32_bits(pkv, lens, scale):  # noqa: F811
    """Queries near 2^100: scale times the row's power of two is past the largest number."""
    check(exact_case(pkv, lens, 2, 8, 2, 128, BF16, 7, queries=2.0 ** 100), scale)


def test_negative_scale(pkv):  # noqa: F811
    c = Case(pkv, [100, 31, 260], 1, 8, 2, 64, BF16, seed=8)
    c.check(q=(c.q.float() * 2.0 ** -70).to(BF16), scale=-1e-20)
    assert math.isfinite(c.scale)
