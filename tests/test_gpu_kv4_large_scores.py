"""paged_kv4_decode_attention on scores of any size: the weights are those of the scores' differences from the largest,
so that a row whose largest scores stand far above the others gives the mean of their values, never inf or NaN."""
import pytest
import torch

import kv4_reference as ref
from test_gpu_kv4_attention import Case, pkv  # noqa: F401

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def exact_case(pkv, lens, q_len, Hq, Hkv, D, dtype, seed, keys=1.0, queries=1.0):
    """Keys that the cache holds as they are and queries of few bits: every score is a multiple of keys * queries / 2
    that 32 bits hold, in any order of its sum.  The keys are drawn from 37 rows, so that a row's largest score comes
    up many times, all over the context."""
    c = Case(pkv, lens, q_len, Hq, Hkv, D, dtype, seed=seed)
    g = torch.Generator().manual_seed(seed)
    pool = LEVELS[torch.randint(0, 8, (37, Hkv, D), generator=g)] * (1 - 2.0 * torch.randint(0, 2, (37, Hkv, D), generator=g))
    pool[..., ::16] = 6.0       # each group's scale is exactly `keys`
    n = c.k.shape[0]
    c.k = (pool[torch.randint(0, 37, (n, 16), generator=g)] * keys).transpose(1, 2).contiguous().to(BF16)
    assert torch.equal(ref.quantised(c.k), c.k.double())
    c.q = (torch.randint(-3, 4, c.q.shape, generator=g) * queries).to(dtype)
    return c


def check(c, scale, window=0, **kw):
    """Scores are exact, the next score is so far below the largest that its weight is 0 in any type, and the weights of
    the largest are the same power of two: what is left are the additions of n equal weights and of n weighted values
    (2^-23 of the sum of magnitudes each), two factors, and the rounding of the output."""
    out = c.call(scale=scale, window=window, four=True, **kw)
    assert c.status == (0, 0)
    vq = ref.quantised(c.v, c.unit[1])
    for b, ctx in enumerate(c.lens):
        ids = c.table[b, :(ctx + 15) // 16].long()
        kb, vb = (x[ids].transpose(1, 2).reshape(-1, c.Hkv, c.D)[:ctx] for x in (c.k.double(), vq))
        want = ref.attention(c.q[b], kb, vb, scale, window)
        most = float(vb.abs().amax()) if ctx else 0.0
        tol = (2 * ctx * 2.0 ** -23 + 2.0 ** -20) * most + torch.finfo(out.dtype).eps / 2 * want.abs() + torch.finfo(out.dtype).tiny
        err = (out[b].double() - want).abs()
        assert (err <= tol).all(), (b, ctx, float((err - tol).nan_to_num(9e9).max()))


SCALES = [1e6, 1e9, -1e9, 1e30, 2e36]      # (the last: scores beyond 32 bits)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, F16)])
@pytest.mark.parametrize("q_len,Hq,Hkv", [(1, 8, 2), (2, 8, 8), (3, 8, 2), (1, 16, 4)])
def test_whole_units(pkv, scale, D, dtype, q_len, Hq, Hkv):  # noqa: F811
    check(exact_case(pkv, [100, 31, 260, 64, 1, 0], q_len, Hq, Hkv, D, dtype, 1), scale)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("D,dtype,q_len,Hq,Hkv", [(128, BF16, 1, 8, 1), (128, F16, 3, 8, 2), (64, BF16, 1, 8, 4), (64, F16, 4, 4, 1)])
def test_units_cut_between_warps_and_ctas(pkv, scale, D, dtype, q_len, Hq, Hkv):  # noqa: F811
    check(exact_case(pkv, [12000, 3, 4001, 700], q_len, Hq, Hkv, D, dtype, 2), scale)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("splits", [0, 1, 7])
def test_one_long_context(pkv, scale, splits):  # noqa: F811
    check(exact_case(pkv, [20000], 1, 8, 1, 128, BF16, 3), scale, num_splits=splits)


@pytest.mark.parametrize("window", [16, 100, 1000])
def test_windows(pkv, window):  # noqa: F811
    check(exact_case(pkv, [2000, 90, 333], 2, 8, 2, 128, BF16, 4), 1e8, window=window)


def test_large_queries_and_keys_at_the_usual_scale(pkv):  # noqa: F811
    """f16 queries to 6000 on keys to 2688."""
    c = exact_case(pkv, [100, 3000], 1, 8, 2, 128, F16, 5, keys=448.0, queries=2000.0)
    check(c, c.scale)
