"""paged_tree_attention against its definition in 64 bits, through the binding:
types, head layouts, tree shapes, lengths, masks, windows, and the calls around
it (streams, graphs, status)."""
import copy

import numpy as np
import pytest
import torch

from gpu_helpers import routes
from tree_reference import Inputs, attention, check_attention, masks_of, to_i64

pytestmark = pytest.mark.gpu


def _pkv():
    import paged_kv_gqa_03_gb300 as pkv
    return pkv


def _call(x, window=0, mask=None, fill=7.0, lens=True, **kw):
    pkv, dev = _pkv(), "cuda"
    out = torch.full(x.q.shape, fill, dtype=x.q.dtype, device=dev)
    up = lambda t: None if t is None else t.to(dev)  # noqa: E731
    ws = pkv.paged_tree_attention(
        out, x.q.to(dev), x.kc.to(dev), x.vc.to(dev), torch.from_numpy(x.table).to(dev),
        torch.tensor(x.ctx, dtype=torch.int32, device=dev), up(x.mask if mask is None else mask), x.scale,
        tree_lens=torch.tensor(x.nodes, dtype=torch.int32, device=dev) if lens else None,
        k_scale=up(x.ks), v_scale=up(x.vs), window=window, **kw)
    return out, ws


def _run(x, window=0, **kw):
    out, ws = _call(x, window, **kw)
    rc, flags = _pkv().paged_decode_status(ws)
    assert (rc, flags) == (0, 0)
    check_attention(out, x, window, untouched=7.0)
    return out


TYPES = [("bf16", "bf16"), ("f16", "f16"), ("fp8_e4m3", "bf16"), ("fp8_e4m3", "f16"), ("f32", "f32")]


@pytest.mark.parametrize("dtype,q_dtype", TYPES, ids=["-".join(t) for t in TYPES])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (6, 2, 64), (4, 4, 128), (14, 2, 128)])
@pytest.mark.parametrize("n", [1, 5, 17])
def test_types_and_heads(dtype, q_dtype, Hq, Hkv, D, n):
    """Contexts of the tree alone, inside one block, ending at and inside tiles."""
    _run(Inputs(11 + n, [n, n + 1, 16 + n, 128, 150 + n, 300], n, Hq, Hkv, D, dtype, q_dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "fp8_e4m3", "f32"])
@pytest.mark.parametrize("n,kind", [(64, "random"), (64, "star"), (33, "chain"), (2, "random")])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 2, 128), (3, 1, 64)])
def test_tree_sizes(dtype, n, kind, Hq, Hkv, D):
    """The widest trees (R = 512 and 192 rows per kv head), every tile boundary inside them."""
    _run(Inputs(5, [64, 100, 128 + 64, 129 + 63, 257, 700], n, Hq, Hkv, D, dtype, kind=kind))


@pytest.mark.parametrize("dtype,Hq,Hkv,D,n", [("bf16", 8, 2, 128, 12), ("bf16", 16, 1, 128, 40), ("f16", 4, 2, 64, 9),
                                              ("fp8_e4m3", 8, 2, 128, 21), ("f32", 4, 2, 64, 7)])
def test_ragged_trees_leave_the_other_rows(dtype, Hq, Hkv, D, n):
    nodes = [0, 1, n, n // 2, 3, n]
    # (a context shorter than its tree: the positions before 0 do not exist)
    _run(Inputs(2, [2, 0, n - 1, 200, 1, 515], n, Hq, Hkv, D, dtype, nodes=nodes))
    _run(Inputs(3, [90, 1, n, 200, 131, 515], n, Hq, Hkv, D, dtype, nodes=nodes))
    _run(Inputs(4, [90, 1, n, 200, 131, 515], n, Hq, Hkv, D, dtype, nodes=nodes, shared=True))


def test_all_sequences_empty():
    x = Inputs(9, [40, 0, 3], 4, 8, 2, 128, "bf16", nodes=[0, 0, 0])
    _run(x)


@pytest.mark.parametrize("dtype,Hq,D,n", [("bf16", 8, 128, 6), ("bf16", 8, 128, 30), ("f16", 8, 64, 6),
                                          ("fp8_e4m3", 8, 128, 6), ("f32", 8, 64, 6)])
def test_masks_that_are_no_tree(dtype, Hq, D, n):
    """Rows that see nothing (an empty mask on a context that is the tree
    alone) give 0; rows without their own node; a node that sees later ones;
    bits past the nodes are ignored."""
    x = Inputs(21, [n, n, 140, 256 + n], n, Hq, 1, D, dtype)
    rng = np.random.default_rng(2)
    x.masks = [[0] * n, [int(v) for v in rng.integers(0, 1 << n, n)], [0] * n,
               [int(v) | (0xABCD << n) & ((1 << 64) - 1) for v in rng.integers(0, 1 << n, n)]]
    x.mask = torch.stack([to_i64(m) for m in x.masks])
    out = _run(x)
    assert torch.all(out[0] == 0)


def test_bit_63():
    x = Inputs(8, [64, 300], 64, 4, 1, 128, "bf16")
    x.masks = [[(1 << 63) | (1 << i) for i in range(64)]] * 2
    x.mask = to_i64(x.masks[0])
    _run(x)


@pytest.mark.parametrize("dtype,Hq,Hkv,D,n", [("bf16", 8, 2, 128, 6), ("bf16", 16, 2, 128, 24), ("f16", 2, 2, 64, 5),
                                              ("fp8_e4m3", 8, 2, 128, 6), ("f32", 4, 2, 128, 6)])
@pytest.mark.parametrize("window", [1, 7, 16, 100, 1000, 2**31 - 1])
def test_sliding_window(dtype, Hq, Hkv, D, n, window):
    """Deep and shallow nodes reach back differently; blocks before every
    row's window are -1 in the table and are not read."""
    x = Inputs(31, [n, n + 3, 130, 260, 517], n, Hq, Hkv, D, dtype)
    for b in range(x.B):
        first = max(0, x.ctx[b] - n + 1 - window) // 16
        x.table[b, :first] = -1
    _run(x, window)


def test_chain_is_the_causal_multi_query_decode():
    pkv = _pkv()
    x = Inputs(2, [40, 7, 300], 7, 8, 2, 128, "bf16", kind="chain")
    out, _ = _call(x)
    ref = torch.empty_like(out)
    dev = "cuda"
    pkv.paged_decode_attention(ref, x.q.to(dev), x.kc.to(dev), x.vc.to(dev), torch.from_numpy(x.table).to(dev),
                               torch.tensor(x.ctx, dtype=torch.int32, device=dev), x.scale)
    check_attention(ref, x)
    check_attention(out, x)


@pytest.mark.parametrize("B", [1, 3, 260, 2100])
def test_batch_sizes(B):
    """One sequence to more than the in-kernel plans hold."""
    rng = np.random.default_rng(B)
    _run(Inputs(1, [int(c) for c in rng.integers(3, 60, B)], 3, 2, 1, 128, "bf16"))


def test_long_context_is_split_and_joined():
    """One sequence, few rows: the context is cut over the whole GPU."""
    for dtype, n, Hq in (("bf16", 2, 2), ("bf16", 9, 8), ("bf16", 40, 8), ("fp8_e4m3", 2, 4), ("f16", 3, 1)):
        _run(Inputs(6, [20011], n, Hq, 1, 128, dtype, stale=False))


def test_bad_entries_are_flagged_and_read_as_zeros():
    pkv = _pkv()
    for Hq in (8, 64):
        x = Inputs(14, [200, 64], 10, Hq, 1, 128, "bf16")
        x.table[0, 3] = x.num_blocks + 5
        x.table[1, 0] = -4
        out, ws = _call(x)
        rc, flags = pkv.paged_decode_status(ws)
        assert rc == pkv.PKV_ERANGE and flags == pkv.PKV_FLAG_BAD_BLOCK
        assert torch.isfinite(out).all()
        x = Inputs(14, [200, 64], 10, Hq, 1, 128, "bf16")
        x.nodes = [10, 11]
        out, ws = _call(x)
        rc, flags = pkv.paged_decode_status(ws)
        assert rc == pkv.PKV_ERANGE and flags == pkv.PKV_FLAG_BAD_LEN
        x.nodes = [10, 10]
        check_attention(out, x)


def test_infinite_and_nan_values_in_hidden_places():
    """K / V rows that no row sees may hold anything, also inside the tree."""
    for Hq in (4, 64):
        x = Inputs(15, [70, 133], 6, Hq, 1, 128, "bf16")
        x.masks = [[0b000001, 0b000011, 0b000101, 0b000011, 0b000001, 0b000101]] * 2
        x.mask = to_i64(x.masks[0])
        for b in range(2):
            for j in (3, 4, 5):
                t = x.ctx[b] - 6 + j
                x.kc[x.table[b, t // 16], :, t % 16] = float("inf")
        _run(x)


def test_on_a_side_stream_and_from_a_graph():
    pkv, dev = _pkv(), "cuda"
    for Hq, n in ((8, 5), (16, 40)):
        x = Inputs(17, [300, 45, 128], n if n < 45 else 40, Hq, 1, 128, "bf16")
        st = torch.cuda.Stream()
        args = [t.to(dev) for t in (x.q, x.kc, x.vc, torch.from_numpy(x.table), torch.tensor(x.ctx, dtype=torch.int32), x.mask)]
        out = torch.empty_like(args[0])
        ws = torch.empty(pkv.paged_tree_workspace_bytes(x.B, x.n, Hq, 1, 128, torch.bfloat16, torch.bfloat16),
                         dtype=torch.uint8, device=dev)
        torch.cuda.synchronize()
        call = pkv.paged_tree_attention(out, *args, x.scale, workspace=ws, stream=st, prepare=True)
        call()
        st.synchronize()
        check_attention(out, x)
        out.fill_(3.0)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            call()
        args[0].copy_(torch.flip(x.q, [0]).to(dev))       # another query in the same buffer
        x.q = torch.flip(x.q, [0])
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        check_attention(out, x)


def test_same_inputs_same_bits():
    for dtype, Hq, n in (("bf16", 8, 6), ("bf16", 16, 32), ("fp8_e4m3", 8, 6)):
        x = Inputs(19, [900, 77, 2000], n, Hq, 1, 128, dtype, stale=False)
        a, _ = _call(x)
        b, _ = _call(x)
        assert torch.equal(a, b)


@pytest.mark.parametrize("route", ["tiles", "units"])
@pytest.mark.parametrize("dtype,Hq,Hkv,D,n", [("bf16", 8, 2, 128, 3), ("bf16", 8, 2, 128, 16), ("f16", 6, 2, 128, 13),
                                              ("bf16", 2, 2, 64, 2), ("f16", 5, 1, 64, 33), ("bf16", 16, 1, 128, 64),
                                              ("bf16", 12, 4, 128, 1), ("fp8_e4m3", 8, 2, 128, 9), ("fp8_e4m3", 6, 2, 64, 5),
                                              ("fp8_e4m3", 16, 1, 128, 64), ("fp8_e4m3", 3, 1, 64, 1)])
def test_every_kernel_on_the_same_inputs(route, dtype, Hq, Hkv, D, n):
    """Each kernel where it applies (pkv_set_route), one tree size each side of
    its row tiles; windows, ragged trees, an empty context."""
    with routes(tree=route):
        ctx = [0, n, 127 + n, 128, 129 + n, 700, 2049]
        ctx = [max(c, n) if c else 0 for c in ctx]
        _run(Inputs(40, ctx, n, Hq, Hkv, D, dtype, nodes=[0, n, n, max(1, n - 1), n, n, 1]))
        _run(Inputs(41, ctx[1:], n, Hq, Hkv, D, dtype), window=130)
        _run(Inputs(42, [5000], n, Hq, Hkv, D, dtype, stale=False))
        _run(Inputs(43, [n + 3] * 170, n, Hq, Hkv, D, dtype))


def _rescaled(x, k, v):
    """The same stored bytes under other block scales."""
    x.ks, x.vs = (x.ks * k).contiguous(), (x.vs * v).contiguous()
    return x


@pytest.mark.parametrize("route", ["tiles", "units"])
@pytest.mark.parametrize("D,q_dtype", [(128, "bf16"), (64, "f16")])
def test_fp8_scales_of_all_sizes(route, D, q_dtype):
    """Block scales that differ by orders of magnitude between blocks and from
    1 (tiles: also values far below f16's normal range)."""
    with routes(tree=route):
        for seed, spread, level in ((1, 0.0, 1.0), (2, 3.0, 1.0), (3, 1.0, 2.0 ** 6)) + (((4, 2.0, 2.0 ** -12),) if route == "tiles" else ()):
            x = Inputs(50 + seed, [9, 130, 400, 1000], 9, 8, 2, D, "fp8_e4m3", q_dtype)
            g = torch.Generator().manual_seed(seed)
            f = lambda: torch.exp2(spread * torch.randn(x.vs.shape, generator=g))  # noqa: E731
            _run(_rescaled(x, torch.exp2(0.3 * spread * torch.randn(x.ks.shape, generator=g)), level * f()))


def test_fp8_zero_and_negative_scales():
    """A block may hold nothing (scale 0) or be stored with negative scales:
    the literal products."""
    for D in (128, 64):
        x = Inputs(61, [140, 400, 33], 12, 8, 2, D, "fp8_e4m3")
        x.ks[x.table[0, 1]] = 0.0
        x.vs[x.table[0, 2]] = 0.0
        x.vs[x.table[1, 5]] *= -1.0
        x.ks[x.table[1, 6]] *= -1.0
        x.vs[x.table[2, 0], 1] = 0.0
        _run(x)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("route", ["tiles", "units"])
def test_fp8_every_byte_value(route, D):
    """Blocks whose values run over all the numbers of the type, subnormal ones
    among them, one range of magnitudes per sequence; a NaN byte that a row
    sees is a NaN in its output, and in no other row's."""
    with routes(tree=route):
        x = Inputs(70, [16 * 3 + 12, 200, 77], 12, 2, 1, D, "fp8_e4m3", stale=False)
        g = torch.Generator().manual_seed(1)
        for b, (lo, hi) in enumerate(((0, 8), (0, 127), (100, 127))):
            for c in (x.kc, x.vc):
                raw = c.view(torch.uint8)
                for blk in x.table[b][x.table[b] >= 0].tolist():
                    raw[blk] = (torch.randint(lo, hi, raw[blk].shape, generator=g) | (torch.randint(0, 2, raw[blk].shape, generator=g) << 7)).to(torch.uint8)
        x.ks = torch.full_like(x.ks, 1.0 / 64)
        _run(x)
        # sequence 1's node 5: its V row holds a NaN at element 3
        t = x.ctx[1] - 12 + 5
        x.masks[1] = [m & ~(1 << 5) | ((1 << 5) if i in (5, 7) else 0) for i, m in enumerate(x.masks[1])]
        x.mask = torch.stack([to_i64(m) for m in x.masks])
        x.kc.view(torch.uint8)[x.table[1, t // 16], 0, t % 16, 3] = 0x7F
        out, _ = _call(x)
        bad = torch.isnan(out[1].float()).any(-1).any(-1).cpu()
        assert bad.tolist() == [i in (5, 7) for i in range(12)]
        assert torch.isfinite(out[0].float()).all() and torch.isfinite(out[2].float()).all()


@pytest.mark.parametrize("dtype,Hq,D,n", [("bf16", 2, 128, 3), ("bf16", 8, 128, 20), ("f16", 8, 64, 20), ("fp8_e4m3", 2, 128, 3),
                                          ("fp8_e4m3", 8, 128, 20), ("f32", 2, 64, 3)])
def test_a_nan_that_is_seen_is_not_lost(dtype, Hq, D, n):
    """One query row of NaN over a context that is split between CTAs: NaN in
    its output and in no other; the same for a K row that every node sees."""
    x = Inputs(80, [9000, 300], n, Hq, 1, D, dtype, stale=False)
    q = x.q.clone()
    x.q[0, 1, Hq - 1, 5] = float("nan")
    x.q[1, 0, 0, 0] = float("inf")
    out, _ = _call(x)
    bad = torch.isnan(out.float()).all(-1).cpu()
    assert bad[0, 1, Hq - 1] and bad[1, 0, 0] and int(bad.sum()) == 2
    assert int(torch.isnan(out.float()).any(-1).sum()) == 2
    x.q = q
    blk = x.table[0, 100]
    if dtype == "fp8_e4m3":
        x.kc.view(torch.uint8)[blk, 0, 7, 0] = 0xFF
    else:
        x.kc[blk, 0, 7, 0] = float("nan")
    out, _ = _call(x)
    assert torch.isnan(out[0].float()).all() and torch.isfinite(out[1].float()).all()


@pytest.mark.parametrize("D,q_dtype", [(128, "bf16"), (64, "bf16"), (128, "f16"), (64, "f16")])
def test_fp8_queries_of_all_sizes(D, q_dtype):
    """The tile kernel splits a query row into E4M3 parts under a scale of the
    row: rows whose elements differ by orders of magnitude, tiny and huge rows."""
    with routes(tree="tiles"):
        x = Inputs(90, [40, 300], 20, 8, 1, D, "fp8_e4m3", q_dtype)
        g = torch.Generator().manual_seed(3)
        mag = torch.exp2(3.0 * torch.randn(x.q.shape, generator=g))
        x.q = (x.q.float() * mag).to(x.q.dtype)
        x.q[0, 3] *= 2.0 ** -10
        x.q[0, 4] *= 2.0 ** 5
        x.q[1, 2] = 0
        x.scale /= 40
        _run(x)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64), ("fp8_e4m3", 128), ("fp8_e4m3", 64)])
def test_small_and_wide_trees_one_after_another(dtype, D):
    """A CTA's items alternate between trees that leave most of a row tile's
    warps without rows and trees that fill it, an odd number of tiles each: the
    warps' exchange keeps step with the tiles through both."""
    rng = np.random.default_rng(7)
    B, n = 240, 40
    nodes = [int(rng.choice([1, 2, 33, 40])) for _ in range(B)]
    ctx = [max(m, int(rng.choice([50, 128, 300]))) for m in nodes]
    with routes(tree="tiles"):
        _run(Inputs(51, ctx, n, 3, 3, D, dtype, nodes=nodes))


def _spoil(x, b, pos, h, cols, values):
    """V elements of a position that are not finite."""
    blk = int(x.table[b, pos // 16])
    if x.dtype == "fp8_e4m3":
        x.vc.view(torch.uint8)[blk, h, pos % 16, cols] = torch.tensor([0x7F, 0xFF] * len(cols), dtype=torch.uint8)[:len(cols)]
    else:
        x.vc[blk, h, pos % 16, cols] = torch.tensor([values[i % len(values)] for i in range(len(cols))], dtype=x.vc.dtype)


def _check_spoiled(out, x, window=0):
    with np.errstate(invalid="ignore"):
        ref, _ = attention(x, window)
    c = copy.copy(x)                                  # the bound of the other elements
    c.vc = torch.where(torch.isfinite(x.vc.float()), x.vc.float(), 0.0).to(x.vc.dtype)
    _, bound = attention(c, window)
    got = out.double().cpu().numpy()
    wild = ~np.isfinite(ref)
    assert wild.any() and not wild.all()
    for b in range(x.B):
        m = x.nodes[b]
        g, r, w = got[b, :m], ref[b, :m], wild[b, :m]
        assert np.array_equal(np.isnan(g[w]), np.isnan(r[w])) and np.array_equal(g[w] > 0, r[w] > 0)
        err = np.abs(g[~w] - r[~w])
        assert (err <= bound[b, :m][~w]).all(), f"sequence {b}: {int((~(err <= bound[b, :m][~w])).sum())} of {err.size}"


@pytest.mark.parametrize("route", ["tiles", "units"])
@pytest.mark.parametrize("dtype,Hq,Hkv,D,n", [("bf16", 8, 2, 128, 6), ("bf16", 16, 1, 128, 40), ("f16", 4, 2, 64, 9), ("f16", 4, 4, 128, 33),
                                              ("fp8_e4m3", 8, 2, 128, 6), ("fp8_e4m3", 4, 1, 64, 40), ("f32", 4, 2, 64, 9),
                                              ("f32", 2, 1, 128, 5)])
def test_values_that_are_not_finite_stay_in_their_branch(route, dtype, Hq, Hkv, D, n):
    """Infinities and NaN in the V rows of some nodes: rows that see such a node
    get what the formula gives, element by element; the others nothing of it."""
    inf, nan = float("inf"), float("nan")
    with routes(tree=route):
        x = Inputs(61, [n, n + 7, 130 + n, 128, 2000], n, Hq, Hkv, D, dtype, nodes=[n, n, n, max(2, n // 2), n])
        for b in range(x.B):
            start, m = x.ctx[b] - x.nodes[b], x.nodes[b]
            for k, node in enumerate((1, m - 1, m // 2)):
                for h in range(Hkv):
                    _spoil(x, b, start + node, h, [k, 7 + k, D // 2 + 5 * k, D - 1 - k], (inf, nan, -inf, inf))
        out, _ = _call(x)
        _check_spoiled(out, x)
        again, _ = _call(x)
        assert torch.equal(out.view(torch.uint8), again.view(torch.uint8))


@pytest.mark.parametrize("route", ["tiles", "units"])
@pytest.mark.parametrize("dtype,Hq,Hkv,D,n", [("bf16", 8, 2, 128, 7), ("f16", 16, 1, 64, 40), ("fp8_e4m3", 8, 2, 128, 7),
                                              ("fp8_e4m3", 4, 1, 64, 40), ("f32", 4, 2, 64, 7)])
@pytest.mark.parametrize("window", [5, 30, 200])
def test_values_that_are_not_finite_at_a_windows_edge(route, dtype, Hq, Hkv, D, n, window):
    """Cached positions before every row's window may hold anything; one that the
    windows of some rows have left touches only those that still see it."""
    inf, nan = float("inf"), float("nan")
    with routes(tree=route):
        x = Inputs(62, [n + 3, 130 + n, 517, 2000], n, Hq, Hkv, D, dtype)
        for b in range(x.B):
            start = x.ctx[b] - n
            first = max(0, start + 1 - window)
            for h in range(Hkv):
                for pos in range(first // 16 * 16, first):        # no row sees them
                    _spoil(x, b, pos, h, list(range(D)), (nan, inf))
                # (a position that every row sees has to be finite)
                for k, pos in enumerate(range(first, min(start + n - window, first + 3))):
                    _spoil(x, b, pos, h, [3 * k, D - 1 - k], (inf, nan))
        out, _ = _call(x, window)
        _check_spoiled(out, x, window)


@pytest.mark.parametrize("route", ["tiles", "units"])
@pytest.mark.parametrize("dtype,blocks", [("bf16", 140000), ("fp8_e4m3", 280000)])
def test_caches_beyond_32_bit_offsets(route, dtype, blocks):
    """Blocks whose bytes and elements lie past 2^32 and 2^31 of the cache."""
    pkv, dev = _pkv(), "cuda"
    Hq, Hkv, D, n = 16, 8, 128, 6
    assert blocks * Hkv * 16 * D * (1 if dtype == "fp8_e4m3" else 2) > 2 ** 32 and blocks * Hkv * 16 * D > 2 ** 31
    x = Inputs(71, [300, 77, n], n, Hq, Hkv, D, dtype)
    ids = torch.arange(x.num_blocks, device=dev) + (blocks - x.num_blocks)
    ids[::3] = torch.arange(len(ids[::3]), device=dev)          # some at the front as well
    big = []
    for c in (x.kc, x.vc):
        t = torch.empty((blocks,) + tuple(c.shape[1:]), dtype=torch.uint8 if dtype == "fp8_e4m3" else c.dtype, device=dev)
        t[ids] = (c.view(torch.uint8) if dtype == "fp8_e4m3" else c).to(dev)
        big.append(t.view(c.dtype))
    scales = [None, None]
    if dtype == "fp8_e4m3":
        scales = [torch.ones((blocks, Hkv), device=dev).index_copy_(0, ids, s.to(dev)) for s in (x.ks, x.vs)]
    table = torch.from_numpy(x.table).to(dev)
    table = torch.where(table >= 0, ids[table.clamp(min=0).long()].int(), table)
    out = torch.empty(x.q.shape, dtype=x.q.dtype, device=dev)
    with routes(tree=route):
        ws = pkv.paged_tree_attention(out, x.q.to(dev), *big, table, torch.tensor(x.ctx, dtype=torch.int32, device=dev),
                                      x.mask.to(dev), x.scale, k_scale=scales[0], v_scale=scales[1])
    assert pkv.paged_decode_status(ws) == (0, 0)
    check_attention(out, x)


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace, over one cache."""
    pkv, dev = _pkv(), "cuda"
    for dtype, Hq, n in (("bf16", 16, 40), ("fp8_e4m3", 8, 6), ("bf16", 4, 3)):
        x = Inputs(81, [3000, 45, 1280, 700], n, Hq, 2, 128, dtype)
        up = lambda t: None if t is None else t.to(dev)  # noqa: E731
        a = [up(t) for t in (x.q, x.kc, x.vc, torch.from_numpy(x.table), torch.tensor(x.ctx, dtype=torch.int32), x.mask)]
        ks, vs = up(x.ks), up(x.vs)
        streams = [torch.cuda.Stream() for _ in range(2)]
        outs = [[torch.full_like(a[0], 7.0) for _ in range(6)] for _ in streams]
        nbytes = pkv.paged_tree_workspace_bytes(x.B, n, Hq, 2, 128, x.kc.dtype, x.q.dtype)
        works = [torch.empty(nbytes, dtype=torch.uint8, device=dev) for _ in streams]
        torch.cuda.synchronize()
        for k in range(6):
            for s, o, w in zip(streams, outs, works):
                pkv.paged_tree_attention(o[k], *a, x.scale, k_scale=ks, v_scale=vs, workspace=w, stream=s)
        torch.cuda.synchronize()
        check_attention(outs[0][0], x)
        for o in outs:
            for t in o:
                assert torch.equal(t, outs[0][0])
