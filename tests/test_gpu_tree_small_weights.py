"""Values that are not finite under weights that 32 bits round to 0."""
import numpy as np
import pytest
import torch

from gpu_helpers import routes
from tree_reference import Inputs, seen_positions

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("route", ["tiles", "units"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "fp8_e4m3", "f32"])
@pytest.mark.parametrize("Hq,D", [(2, 128), (8, 64)])
def test_a_value_that_is_seen_is_not_lost_under_a_small_weight(route, dtype, Hq, D):
    """A weight is positive, however small: an infinity or NaN in the V row of a
    node reaches that element of every row that sees the node, and of no other."""
    import paged_kv_gqa_03_gb300 as pkv
    n, dev = 9, "cuda"
    x = Inputs(37, [n, 130, 2500], n, Hq, 1, D, dtype)
    x.scale = 12.0                      # scores hundreds apart: most weights are below 2^-149
    cols = {2: 5, 5: 40, 8: 63}
    for b in range(x.B):
        for node, col in cols.items():
            t = x.ctx[b] - n + node
            if dtype == "fp8_e4m3":
                x.vc.view(torch.uint8)[x.table[b, t // 16], 0, t % 16, col] = 0x7F
            else:
                x.vc[x.table[b, t // 16], 0, t % 16, col] = float("inf")
    up = lambda t: None if t is None else t.to(dev)  # noqa: E731
    out = torch.empty(x.q.shape, dtype=x.q.dtype, device=dev)
    with routes(tree=route):
        pkv.paged_tree_attention(out, up(x.q), up(x.kc), up(x.vc), torch.from_numpy(x.table).to(dev),
                                 torch.tensor(x.ctx, dtype=torch.int32, device=dev), up(x.mask), x.scale, k_scale=up(x.ks),
                                 v_scale=up(x.vs))
    got = np.isfinite(out.float().cpu().numpy())
    for b in range(x.B):
        for i in range(n):
            wild = {col for node, col in cols.items() if x.ctx[b] - n + node in seen_positions(x, b, i)}
            want = np.array([d not in wild for d in range(D)])
            assert (got[b, i] == want).all(), (b, i, sorted(wild))
