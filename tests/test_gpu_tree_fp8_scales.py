"""Tree attention on fp8 caches whose block scales are not ordinary numbers, and
queries that are not."""
import numpy as np
import pytest
import torch

from gpu_helpers import routes
from tree_reference import Inputs, attention, to_i64

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
