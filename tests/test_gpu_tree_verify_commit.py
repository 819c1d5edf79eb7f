"""paged_tree_verify and paged_tree_commit against their definitions, and the
three tree calls together as a speculative step uses them."""
import numpy as np
import pytest
import torch

from tree_reference import Inputs, commit, masks_of, random_parents, to_i64, verify

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _pkv():
    import paged_kv_gqa_03_gb300 as pkv
    return pkv


class Drafts:
    def __init__(self, seed, B, n, V, mode, dtype="f32", kind="random", noise=0.7, sharp=2.0, nodes=None, shared=False):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.nodes = [n] * B if nodes is None else nodes
        parents = [random_parents(n, rng, kind) for _ in range(B)]
        if shared:
            parents = [parents[0]] * B
        self.masks = [masks_of(p) for p in parents]
        self.mask = to_i64(self.masks[0]) if shared else torch.stack([to_i64(m) for m in self.masks])
        logits = sharp * torch.randn(B, n, V, generator=g)
        noisy = logits + noise * torch.randn(B, n, V, generator=g)
        self.target = (logits if mode == "greedy" else torch.softmax(logits, -1)).to(DT[dtype])
        self.draft = torch.softmax(noisy, -1).to(DT[dtype]) if mode == "sample" else None
        tokens = torch.zeros(B, n, dtype=torch.int64)
        for b in range(B):
            used = {}
            for i in range(1, n):
                p = parents[b][i]
                if mode == "sample":
                    tokens[b, i] = torch.multinomial(self.draft[b, p].float(), 1, generator=g)[0]
                else:
                    k = used[p] = used.get(p, -1) + 1
                    tokens[b, i] = noisy[b, p].topk(min(V, k + 1)).indices[-1]
        self.tokens = tokens
        self.u = None if mode == "greedy" else torch.rand(B, n, generator=g)

    def check(self, target=None, draft=None):
        pkv, dev = _pkv(), "cuda"
        B, n = self.tokens.shape
        path = torch.full((B, n), 9, dtype=torch.int32, device=dev)
        length = torch.full((B,), 9, dtype=torch.int32, device=dev)
        token = torch.full((B,), 9, dtype=torch.int64, device=dev)
        up = lambda t: None if t is None else t.to(dev)  # noqa: E731
        pkv.paged_tree_verify(path, length, token, self.tokens.to(dev), self.mask.to(dev),
                              up(self.target) if target is None else target,
                              draft_probs=up(self.draft) if draft is None else draft, uniforms=up(self.u),
                              tree_lens=torch.tensor(self.nodes, dtype=torch.int32, device=dev))
        f = lambda t: None if t is None else t.double().numpy()  # noqa: E731
        want = verify(self.masks, self.tokens.numpy(), f(self.target), f(self.draft), f(self.u), self.nodes)
        for got, ref, what in zip((path, length, token), want, ("path", "path_len", "next_token")):
            got = got.cpu().numpy()
            assert np.array_equal(got, ref), f"{what}: {np.argwhere(got != ref)[:3].tolist()} got {got[got != ref][:3]} want {ref[got != ref][:3]}"
        return want


@pytest.mark.parametrize("mode", ["sample", "topk", "greedy"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4097, 32000])
def test_modes_types_and_vocabularies(mode, dtype, V):
    for kind in ("chain", "random", "star"):
        Drafts(V + 3, 5, 7, V, mode, dtype, kind).check()


@pytest.mark.parametrize("mode", ["sample", "topk", "greedy"])
def test_tree_sizes(mode):
    lens = []
    for n in (1, 2, 33, 64):
        for seed in (1, 2):
            lens += Drafts(seed, 6, n, 500, mode, noise=0.4).check()[1].tolist()
    assert max(lens) >= 3   # the walks go somewhere


@pytest.mark.parametrize("mode", ["sample", "topk", "greedy"])
def test_ragged_and_shared_trees(mode):
    Drafts(4, 6, 12, 300, mode, nodes=[12, 0, 1, 5, 12, 3]).check()
    Drafts(5, 4, 12, 300, mode, shared=True).check()


def test_many_sequences():
    Drafts(6, 300, 4, 257, "sample").check()
    Drafts(7, 300, 4, 257, "greedy").check()


def test_large_vocabulary():
    for mode in ("sample", "topk", "greedy"):
        Drafts(8, 2, 4, 151936, mode, noise=2.0).check()


@pytest.mark.parametrize("mode", ["sample", "topk"])
def test_every_draft_accepted_and_every_draft_refused(mode):
    d = Drafts(9, 4, 6, 200, mode, kind="chain")
    d.u[:, 1:] = 0.0
    assert (d.check()[1] == 6).all()
    d.u[:, 1:] = 1.0 - 2.0 ** -24
    d.target = d.target * 0 + 1.0 / 200
    for b in range(4):
        for i in range(1, 6):
            d.target[b, i - 1, d.tokens[b, i]] = 0.0
    assert (d.check()[1] == 1).all()


@pytest.mark.parametrize("mode", ["sample", "topk"])
def test_the_draw_at_its_ends(mode):
    d = Drafts(10, 4, 5, 700, mode, kind="star")
    d.u[:, 0] = torch.tensor([0.0, 1.0 - 2.0 ** -24, 0.5, 1.0])
    d.check()


def test_repeated_and_impossible_tokens():
    """The same token twice at a node, and ids outside the vocabulary."""
    for mode in ("sample", "topk", "greedy"):
        d = Drafts(11, 4, 8, 50, mode, kind="star")
        d.tokens[:, 3] = d.tokens[:, 1]
        d.tokens[:, 4] = -1
        d.tokens[:, 5] = 50
        d.tokens[:, 6] = 2 ** 40
        d.check()


def test_no_weight_left():
    """The target puts everything on a refused token: nothing to draw."""
    d = Drafts(12, 1, 2, 40, "topk", kind="chain")
    d.target.zero_()
    assert d.check()[2][0] == -1


def test_greedy_ties_take_the_lowest_id():
    d = Drafts(13, 3, 4, 3000, "greedy", "bf16", kind="chain")
    d.target[:] = 1.0
    d.target[1, 0, 1234] = 2.0
    d.target[1, 0, 2999] = 2.0
    d.target[2] = float("-inf")
    d.tokens[0, 1:] = 0
    d.check()


def test_row_strides():
    """Rows of a wider (padded) vocabulary, at every alignment."""
    for mode in ("sample", "greedy", "topk"):
        for pad in (1, 3, 8):
            d = Drafts(14, 3, 5, 601, mode, "bf16" if pad == 3 else "f32")
            wide = lambda t: None if t is None else torch.cat(  # noqa: E731
                [t, torch.full((3, 5, pad), 5.0, dtype=t.dtype)], -1).cuda()[..., :601]
            d.check(target=wide(d.target), draft=wide(d.draft))


def test_borders_agree_with_double_precision():
    """A flat vocabulary of 100003 ids: the draws' borders are 1e-5 apart,
    and 32-bit partial sums (1e-7 of the total) would miss some in a hundred."""
    B, V = 64, 100003
    for mode in ("sample", "topk"):
        d = Drafts(15, B, 2, V, mode, kind="chain", sharp=0.02, noise=0.02)
        d.check()


# ---------------------------------------------------------------------------
def _commit(x, path, length, new=True, **kw):
    pkv, dev = _pkv(), "cuda"
    kc, vc = x.kc.to(dev), x.vc.to(dev)
    lens = torch.full((x.B,), -7, dtype=torch.int32, device=dev) if new else None
    up = lambda t: None if t is None else t.to(dev)  # noqa: E731
    pkv.paged_tree_commit(kc, vc, torch.from_numpy(path).to(dev), torch.from_numpy(length).to(dev),
                          torch.from_numpy(x.table).to(dev), torch.tensor(x.ctx, dtype=torch.int32, device=dev),
                          k_scale=up(x.ks), v_scale=up(x.vs),
                          tree_lens=torch.tensor(x.nodes, dtype=torch.int32, device=dev), new_lens=lens, **kw)
    for got, ref in zip((kc, vc), commit(x, path, length)):
        got = got.view(torch.uint8).cpu().numpy().reshape(ref.shape)
        assert np.array_equal(got, ref), f"{int((got != ref).any(-1).sum())} rows differ"
    if new:
        assert lens.tolist() == [max(0, x.ctx[b] - x.nodes[b] + min(max(int(length[b]), 0), x.nodes[b])) for b in range(x.B)]


def _paths(x, seed, longest):
    rng = np.random.default_rng(seed)
    path = np.full((x.B, x.n), -1, dtype=np.int32)
    length = np.zeros(x.B, dtype=np.int32)
    for b in range(x.B):
        m = x.nodes[b]
        if m:
            k = int(rng.integers(1, min(m, longest) + 1))
            path[b, :k] = [0] + sorted(rng.choice(np.arange(1, m), k - 1, replace=False).tolist())
            length[b] = k
    return path, length


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32", "fp8_e4m3"])
@pytest.mark.parametrize("Hkv,D", [(1, 64), (3, 128), (8, 64)])
@pytest.mark.parametrize("n", [1, 2, 17, 64])
def test_commit(dtype, Hkv, D, n):
    """Paths of all lengths, in place and across blocks."""
    x = Inputs(n, [n, n + 7, 16 + n, 100, 131], n, Hkv, Hkv, D, dtype,
               nodes=None if n < 3 else [n, n - 1, 1, 0, n])
    for seed in (1, 2):
        _commit(x, *_paths(x, seed, n))


def test_commit_shifts_a_long_chain():
    """[0, 2, 3, .., 63]: every row is both a destination and a source."""
    for dtype in ("bf16", "fp8_e4m3", "f32"):
        x = Inputs(3, [64, 70, 79], 64, 2, 2, 64 if dtype == "fp8_e4m3" else 128, dtype)
        path = np.tile(np.array([0] + list(range(2, 64)) + [-1], dtype=np.int32), (3, 1))
        _commit(x, path, np.full(3, 63, dtype=np.int32))


def test_commit_ignores_entries_that_are_no_path():
    x = Inputs(5, [40, 33, 64], 8, 2, 2, 128, "bf16")
    path = np.array([[0, 1, 9, -5, 2, 7, 2 ** 30, 7], [3, 3, 3, 3, 3, 3, 3, 3], [7, 6, 5, 4, 3, 2, 1, 0]], dtype=np.int32)
    _commit(x, path, np.array([8, 99, 8], dtype=np.int32))
    _commit(x, path, np.array([0, -3, 1], dtype=np.int32))
    x.table[0, -2:] = x.num_blocks + 1
    x2 = Inputs(5, [40, 33, 64], 8, 2, 2, 128, "bf16")
    pkv, dev = _pkv(), "cuda"
    kc, vc = x2.kc.to(dev), x2.vc.to(dev)
    x.table[:] = -1
    pkv.paged_tree_commit(kc, vc, torch.from_numpy(path).to(dev), torch.tensor([8, 8, 8], dtype=torch.int32, device=dev),
                          torch.from_numpy(x.table).to(dev), torch.tensor(x.ctx, dtype=torch.int32, device=dev))
    assert torch.equal(kc.view(torch.int16).cpu(), x2.kc.view(torch.int16))


def test_commit_large_batch_and_graph():
    pkv, dev = _pkv(), "cuda"
    x = Inputs(7, [20 + (b % 50) for b in range(300)], 9, 2, 2, 128, "fp8_e4m3")
    path, length = _paths(x, 3, 9)
    _commit(x, path, length)
    kc, vc = x.kc.to(dev), x.vc.to(dev)
    args = (torch.from_numpy(path).to(dev), torch.from_numpy(length).to(dev), torch.from_numpy(x.table).to(dev),
            torch.tensor(x.ctx, dtype=torch.int32, device=dev))
    ks, vs = x.ks.to(dev), x.vs.to(dev)
    st = torch.cuda.Stream()
    call = pkv.paged_tree_commit(kc, vc, *args, k_scale=ks, v_scale=vs, stream=st, prepare=True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    g.replay()
    torch.cuda.synchronize()
    for got, ref in zip((kc, vc), commit(x, path, length)):
        assert np.array_equal(got.view(torch.uint8).cpu().numpy().reshape(ref.shape), ref)


@pytest.mark.parametrize("dtype,blocks", [("bf16", 140000), ("fp8_e4m3", 280000)])
def test_commit_beyond_32_bit_offsets(dtype, blocks):
    """Rows whose bytes lie past 2^32 of the cache."""
    pkv, dev = _pkv(), "cuda"
    Hkv, D, n = 8, 128, 40
    x = Inputs(91, [n + 11, 700], n, 8, Hkv, D, dtype, stale=False)
    path, length = _paths(x, 3, 12)
    ids = torch.arange(x.num_blocks, device=dev) + (blocks - x.num_blocks)
    raw, big = [], []
    for c in (x.kc, x.vc):
        t = torch.empty((blocks,) + tuple(c.shape[1:]), dtype=torch.uint8 if dtype == "fp8_e4m3" else c.dtype, device=dev)
        t[ids] = (c.view(torch.uint8) if dtype == "fp8_e4m3" else c).to(dev)
        raw.append(t)
        big.append(t.view(c.dtype))
    scales = [None, None]
    if dtype == "fp8_e4m3":
        scales = [torch.ones((blocks, Hkv), device=dev).index_copy_(0, ids, s.to(dev)) for s in (x.ks, x.vs)]
    table = torch.from_numpy(x.table).to(dev)
    table = torch.where(table >= 0, ids[table.clamp(min=0).long()].int(), table)
    pkv.paged_tree_commit(*big, torch.as_tensor(path, dtype=torch.int32).to(dev), torch.as_tensor(length, dtype=torch.int32).to(dev), table,
                          torch.tensor(x.ctx, dtype=torch.int32, device=dev), k_scale=scales[0], v_scale=scales[1])
    for t, want in zip(raw, commit(x, path, length)):
        got = t[ids].contiguous().view(torch.uint8).cpu().numpy().reshape(want.shape)
        assert np.array_equal(got, want)
