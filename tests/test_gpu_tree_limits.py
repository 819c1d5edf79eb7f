"""Tree attention at the ends of what its counts hold."""
import numpy as np
import pytest
import torch

from tree_reference import Inputs, check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
def test_wide_trees_under_long_tables(dtype):
    """64 sequences with room for 131072 positions each and the widest tree:
    short contexts, tables of 8192 entries."""
    import paged_kv_gqa_03_gb300 as pkv
    B, n, Hq, Hkv, D = 64, 64, 64, 8, 128
    rng = np.random.default_rng(1)
    x = Inputs(4, [int(c) for c in rng.integers(n, 200, B)], n, Hq, Hkv, D, dtype)
    x.table = np.concatenate([x.table, np.full((B, 8192 - x.table.shape[1]), -1, dtype=np.int32)], 1)
    dev = "cuda"
    up = lambda t: None if t is None else t.to(dev)  # noqa: E731
    out = torch.full(x.q.shape, 7.0, dtype=x.q.dtype, device=dev)
    ws = pkv.paged_tree_attention(out, up(x.q), up(x.kc), up(x.vc), torch.from_numpy(x.table).to(dev),
                                  torch.tensor(x.ctx, dtype=torch.int32, device=dev), up(x.mask), x.scale,
                                  k_scale=up(x.ks), v_scale=up(x.vs))
    assert pkv.paged_decode_status(ws) == (0, 0)
    check_attention(out, x)
