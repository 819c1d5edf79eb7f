"""Tree attention on fp8 caches whose block scales are not ordinary numbers, and
queries that are not; and how near the kernels come when the scales are small
or differ."""
import numpy as np
import pytest
import torch

from gpu_helpers import routes
from tree_reference import BLOCK, TORCH, Inputs, attention, seen_positions, to_i64

pytestmark = pytest.mark.gpu


def _call(x, window=0):
    import paged_kv_gqa_03_gb300 as pkv
    dev = "cuda"
    up = lambda t: None if t is None else t.to(dev)  # noqa: E731
    out = torch.full(x.q.shape, 7.0, dtype=x.q.dtype, device=dev)
    ws = pkv.paged_tree_attention(
        out, x.q.to(dev), x.kc.to(dev), x.vc.to(dev), torch.from_numpy(x.table).to(dev),
        torch.tensor(x.ctx, dtype=torch.int32, device=dev), x.mask.to(dev), x.scale,
        tree_lens=torch.tensor(x.nodes, dtype=torch.int32, device=dev), k_scale=up(x.ks), v_scale=up(x.vs), window=window)
    assert pkv.paged_decode_status(ws) == (0, 0)
    return out.double().cpu().numpy()


def _overflowed(D, q_dtype, Hq, Hkv, n, opens, tree_of):
    """A tree whose node `opens` opens a block, on contexts from the tree alone
    (after the block before it) to one that is split over the GPU."""
    ctx = [16 - opens + n, 16 * 9 - opens + n, 16 * 300 - opens + n]
    x = Inputs(33, ctx, n, Hq, Hkv, D, "fp8_e4m3", q_dtype, stale=False)
    x.masks = [tree_of] * 3
    x.mask = torch.stack([to_i64(tree_of)] * 3)
    return x


@pytest.mark.parametrize("route", ["tiles", "units"])
@pytest.mark.parametrize("D,q_dtype,Hq,Hkv", [(128, "bf16", 4, 1), (64, "bf16", 2, 2), (128, "f16", 16, 2), (64, "f16", 3, 1)])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), -float("inf")])
@pytest.mark.parametrize("which", ["k", "v", "both"])
def test_a_scale_that_is_not_finite_stays_in_its_branch(route, D, q_dtype, Hq, Hkv, value, which):
    """A drafted branch whose values overflowed opens a block: its scale is an
    infinity or a NaN.  Rows that see nothing of that block get what the formula
    gives; those that see it (infinities and NaN in the formula) are NaN."""
    n, opens = 11, 5
    masks = [1 << i | (1 if i else 0) for i in range(n)]      # a star: node 0 and the node itself
    x = _overflowed(D, q_dtype, Hq, Hkv, n, opens, masks)
    for b in range(x.B):
        blk = int(x.table[b, (x.ctx[b] - n + opens) // 16])
        for s in {"k": [x.ks], "v": [x.vs], "both": [x.ks, x.vs]}[which]:
            s[blk] = value
    with routes(tree=route):
        got = _call(x)
    with np.errstate(invalid="ignore"):
        ref, bound = attention(x)
    for b in range(x.B):
        assert np.isfinite(ref[b, :opens]).all()
        err = np.abs(got[b, :opens] - ref[b, :opens])
        assert (err <= bound[b, :opens]).all(), f"sequence {b}: {int(np.isnan(got[b, :opens]).sum())} NaN"
        assert np.isnan(got[b, opens:]).all()


def test_an_overflowed_draft_through_the_append():
    """The same from the append: a V row with an infinity at the opener of a block."""
    import paged_kv_gqa_03_gb300 as pkv
    n, opens, Hq, D = 9, 4, 4, 128
    masks = [1 << i | (1 if i else 0) for i in range(n)]
    for route in ("tiles", "units"):
        x = _overflowed(D, "bf16", Hq, 1, n, opens, masks)
        g = torch.Generator().manual_seed(2)
        kn, vn = (torch.randn(x.B, n, 1, D, generator=g).bfloat16() for _ in range(2))
        vn[:, opens, 0, 17] = float("inf")
        slots = torch.tensor([[int(x.table[b, p // 16]) * 16 + p % 16 for p in range(x.ctx[b] - n, x.ctx[b])] for b in range(x.B)])
        dev = [t.cuda() for t in (x.kc, x.vc, x.ks, x.vs)]
        pkv.paged_kv_append(kn.view(-1, 1, D).cuda(), vn.view(-1, 1, D).cuda(), dev[0], dev[1], slots.view(-1).cuda(), dev[2], dev[3])
        x.kc, x.vc, x.ks, x.vs = (t.cpu() for t in dev)
        assert np.isinf(x.vs.numpy()).any()
        with routes(tree=route):
            got = _call(x)
        with np.errstate(invalid="ignore"):
            ref, bound = attention(x)
        assert (np.abs(got[:, :opens] - ref[:, :opens]) <= bound[:, :opens]).all()
        assert np.isnan(got[:, opens:]).all()


@pytest.mark.parametrize("route", ["tiles", "units"])
@pytest.mark.parametrize("dtype,q_dtype", [("fp8_e4m3", "bf16"), ("fp8_e4m3", "f16"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("window", [0, 1])
def test_a_query_that_is_not_finite_and_sees_nothing(route, dtype, q_dtype, window):
    """A row that sees nothing gives 0, whatever its query holds."""
    n = 6
    ctx = [n, n] if window == 0 else [n + 300, n + 17]       # (window 1: a node without a mask sees nothing)
    x = Inputs(71, ctx, n, 4, 2, 128, dtype, q_dtype)
    x.masks = [[m if i % 2 == 0 else 0 for i, m in enumerate(ms)] for ms in x.masks]
    x.mask = torch.stack([to_i64(m) for m in x.masks])
    x.q[:, 1, :, 3] = float("nan")
    x.q[:, 3, :, 5] = float("inf")
    x.q[:, 4, 1, 0] = float("nan")
    with routes(tree=route):
        got = _call(x, window)
    assert (got[:, 1::2] == 0).all()
    assert np.isnan(got[:, 4, 1]).all() and np.isfinite(got[:, [0, 2]]).all()


@pytest.mark.parametrize("route", ["tiles", "units"])
@pytest.mark.parametrize("D", [64, 128])
def test_tiny_queries_on_tiny_scales(route, D):
    """Scores whose factor leaves 32 bits: the visible positions weigh the same,
    the hidden ones nothing."""
    n = 7
    x = Inputs(72, [n, 140, 500], n, 4, 1, D, "fp8_e4m3")
    x.q = (x.q.float() * 2.0 ** -110).bfloat16()
    x.ks = torch.full_like(x.ks, 2.0 ** -50)
    ref, bound = attention(x)
    with routes(tree=route):
        got = _call(x)
    assert (np.abs(got - ref) <= bound).all()


def tight_bound(x, window=0):
    """(out, bound [B, n, Hq, D]): the definition in 64 bits and how far a kernel
    may be from it: a bound that counts the weights' steps against the largest weight
    times scale of the row, not against the largest value a byte can stand for.  As
    attention()'s bound (half a step of the output; 2^-13 of
    A = sum w |v| for the scores and the fp32 sums; 2^-11 of A for weights rounded to
    f16), but for weights below f16's normal range: with v_b the block scales a weight
    enters as 2^(s + log2 v_b - m), m a running maximum of that exponent, so the weight is
    at most 1 (2^8 before a maximum is taken over) and what it stands for is
    w v_b / max(w v_b); half a subnormal step is 2^-25 of max(w v_b), against the
    decoded value, for every position.  A running maximum that is still below the
    last one makes the step smaller, not larger."""
    out, _ = attention(x, window)
    bound = np.full_like(out, np.inf)
    G, half = x.Hq // x.Hkv, torch.finfo(TORCH[x.q_dtype]).eps / 2
    q = x.q.double().numpy()
    for b in range(x.B):
        for h in range(x.Hkv):
            K, V = (x.rows(b, h, w, np.arange(x.ctx[b])) for w in (0, 1))
            vb = x.vs.double().numpy()[x.table[b, np.arange(x.ctx[b]) // BLOCK], h]
            for i in range(x.nodes[b]):
                t = seen_positions(x, b, i, window)
                if not t:
                    bound[b, i, h * G:(h + 1) * G] = 0
                    continue
                s = q[b, i, h * G:(h + 1) * G] @ K[t].T * x.scale
                w = np.exp(s - s.max(-1, keepdims=True))
                l = w.sum(-1, keepdims=True)
                A = w / l @ np.abs(V[t])
                dec = (np.abs(V[t]) / vb[t][:, None]).sum(0)
                step = 2.0 ** -25 * (w * vb[t]).max(-1, keepdims=True) * dec / l
                o = out[b, i, h * G:(h + 1) * G]
                bound[b, i, h * G:(h + 1) * G] = half * np.abs(o) + (2.0 ** -13 + 2.0 ** -11) * A + step
    return out, bound


def _blind(ref, bound):
    """The part of the outputs for which 0 would be within the bound."""
    return float((np.abs(ref) <= bound).mean())


@pytest.mark.parametrize("route", ["tiles", "units"])
@pytest.mark.parametrize("D,q_dtype,n", [(128, "bf16", 9), (64, "f16", 9), (128, "f16", 3), (64, "bf16", 2)])
@pytest.mark.parametrize("spread,level", [(0.0, 1.0), (0.0, 2.0 ** -12), (2.0, 2.0 ** -12), (3.0, 1.0), (1.0, 2.0 ** 20), (0.0, 2.0 ** -40)])
def test_every_scale_meets_the_same_bound(route, D, q_dtype, n, spread, level):
    x = Inputs(50 + n, [n, 130, 400, 1000], n, 8, 2, D, "fp8_e4m3", q_dtype)
    g = torch.Generator().manual_seed(7)
    x.ks = (x.ks * torch.exp2(0.3 * spread * torch.randn(x.ks.shape, generator=g))).contiguous()
    x.vs = (x.vs * level * torch.exp2(spread * torch.randn(x.vs.shape, generator=g))).contiguous()
    if level not in (1.0, 2.0 ** -12):   # (outputs outside f16's range)
        x.q_dtype = "bf16"
        x.q = x.q.bfloat16()
    ref, bound = tight_bound(x)
    if spread == 0:
        assert _blind(ref, bound) < 0.05
    with routes(tree=route):
        got = _call(x)
    # (outputs below the output type's normal range: half its subnormal step)
    tiny = torch.finfo(TORCH[x.q_dtype]).smallest_normal * torch.finfo(TORCH[x.q_dtype]).eps / 2
    err = np.abs(got - ref) - tiny
    bad = ~(err <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} out of bound, worst {np.nanmax(err / bound):.3g} of it"


@pytest.mark.parametrize("route", ["tiles", "units"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("power", [40, 17, -17, -40, -100])
def test_queries_of_any_size(route, D, power):
    """bf16 queries reach far beyond f16 both ways; the scale undoes the factor, so
    the formula's outputs are those of ordinary queries."""
    x = Inputs(91, [9, 140, 1500], 9, 6, 2, D, "fp8_e4m3")
    x.q = (x.q.float() * 2.0 ** power).bfloat16()
    x.scale *= 2.0 ** -power
    ref, bound = tight_bound(x)
    with routes(tree=route):
        got = _call(x)
    assert (np.abs(got - ref) <= bound).all()
