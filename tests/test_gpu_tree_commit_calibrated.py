"""paged_tree_commit on caches of the calibrated fp8 append: byte for byte against
the rule, and through TreeStep: what a confirmed position holds survives the
move of the accepted rows, however different the drafted rows' magnitudes."""
import math

import numpy as np
import pytest
import torch

from tree_reference import BLOCK, Inputs, masks_of, random_parents, to_i64

pytestmark = pytest.mark.gpu


def _pkv():
    import paged_kv_gqa_03_gb300 as pkv
    return pkv


def _pow2(amax):
    m, e = math.frexp(float(amax))
    return math.ldexp(1.0, e - 9 if m <= 0.875 else e - 8)


def _decode(raw):
    return torch.from_numpy(np.ascontiguousarray(raw)).view(torch.float8_e4m3fn).float()


def _encode(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def commit_calibrated(raws, scales, table, ctx, nodes, path, length):
    """The caches' bytes [nb, Hkv, 16, D] and scales [nb, Hkv] after the call, by the rule."""
    raws, scales = [r.copy() for r in raws], [s.clone() for s in scales]
    for raw, sc in zip(raws, scales):
        for b in range(len(ctx)):
            start = ctx[b] - nodes[b]
            for k in range(min(int(length[b]), nodes[b])):
                f = int(path[b, k])
                if not k < f < nodes[b]:
                    continue
                sp, dp = start + f, start + k
                si, di = int(table[b, sp // BLOCK]), int(table[b, dp // BLOCK])
                for h in range(raw.shape[1]):
                    row = raw[si, h, sp % BLOCK].copy()
                    if si != di:
                        v = _decode(row)
                        top = float(v[~v.isnan()].abs().max() * sc[si, h]) if not v.isnan().all() else 0.0
                        if 0 < top < math.inf and _pow2(top) > float(sc[di, h]):
                            p = torch.tensor(_pow2(top))
                            used = min(BLOCK, ctx[b] - dp // BLOCK * BLOCK)
                            raw[di, h, :used] = _encode(_decode(raw[di, h, :used]) * sc[di, h] / p)
                            sc[di, h] = p
                        row = _encode(v * sc[si, h] / sc[di, h])
                    raw[di, h, dp % BLOCK] = row
    return raws, scales


def _run(x, path, length, new=True):
    pkv, dev = _pkv(), "cuda"
    kc, vc, ks, vs = (t.to(dev) for t in (x.kc, x.vc, x.ks, x.vs))
    lens = torch.full((x.B,), -7, dtype=torch.int32, device=dev) if new else None
    pkv.paged_tree_commit(kc, vc, torch.from_numpy(path).to(dev), torch.from_numpy(length).to(dev),
                          torch.from_numpy(x.table).to(dev), torch.tensor(x.ctx, dtype=torch.int32, device=dev), k_scale=ks,
                          v_scale=vs, tree_lens=torch.tensor(x.nodes, dtype=torch.int32, device=dev), new_lens=lens,
                          calibrated=True)
    raws = [c.view(torch.uint8).numpy().reshape(x.num_blocks, x.Hkv, BLOCK, x.D) for c in (x.kc, x.vc)]
    want, scales = commit_calibrated(raws, [x.ks, x.vs], x.table, x.ctx, x.nodes, path, length)
    for got, ref in zip((kc, vc), want):
        got = got.view(torch.uint8).cpu().numpy().reshape(ref.shape)
        assert np.array_equal(got, ref), f"{int((got != ref).any(-1).sum())} rows differ"
    for got, ref in zip((ks, vs), scales):
        assert torch.equal(got.cpu(), ref)
    if new:
        assert lens.tolist() == [max(0, x.ctx[b] - x.nodes[b] + min(max(int(length[b]), 0), x.nodes[b])) for b in range(x.B)]
    return raws, want, scales


def _paths(x, seed):
    rng = np.random.default_rng(seed)
    path = np.full((x.B, x.n), -1, dtype=np.int32)
    length = np.zeros(x.B, dtype=np.int32)
    for b in range(x.B):
        m = x.nodes[b]
        if m:
            k = int(rng.integers(1, m + 1))
            path[b, :k] = [0] + sorted(rng.choice(np.arange(1, m), k - 1, replace=False).tolist())
            length[b] = k
    return path, length


@pytest.mark.parametrize("powers", [True, False])
@pytest.mark.parametrize("Hkv,D", [(1, 64), (3, 128)])
@pytest.mark.parametrize("n", [2, 17, 64])
def test_bytes_and_scales(Hkv, D, n, powers):
    """Paths of all lengths over blocks whose scales differ by up to 2^10; scales
    of the calibrated append (powers of two) and of the plain one."""
    x = Inputs(n, [n, n + 7, 16 + n, 100, 131, n + 15], n, Hkv, Hkv, D, "fp8_e4m3",
               nodes=None if n < 3 else [n, n - 1, 1, 0, n, n])
    g = torch.Generator().manual_seed(n)
    for name in ("ks", "vs"):
        s = torch.exp2(torch.randint(-12, -1, (x.num_blocks, Hkv), generator=g).float())
        setattr(x, name, s if powers else s * (0.5 + torch.rand(s.shape, generator=g)))
    for seed in (1, 2):
        _run(x, *_paths(x, seed))
    # rows of zeros ask for no scale, entries that are no path move nothing
    x.kc.view(torch.uint8)[:, :, 1:] = 0
    path, length = _paths(x, 3)
    path[0, :2] = (n - 1, 0)
    length[1] = 99
    _run(x, path, length, new=False)


def test_overflowed_rows_raise_no_scale():
    x = Inputs(9, [30, 40], 8, 2, 1, 64, "fp8_e4m3")
    x.vs[int(x.table[0, 1])] = float("inf")
    x.ks[int(x.table[1, 2])] = float("nan")
    path = np.tile(np.array([0, 6, 7, -1, -1, -1, -1, -1], dtype=np.int32), (2, 1))
    pkv, dev = _pkv(), "cuda"
    ks, vs = x.ks.to(dev), x.vs.to(dev)
    pkv.paged_tree_commit(x.kc.to(dev), x.vc.to(dev), torch.from_numpy(path).to(dev), torch.tensor([3, 3], dtype=torch.int32, device=dev),
                          torch.from_numpy(x.table).to(dev), torch.tensor(x.ctx, dtype=torch.int32, device=dev), k_scale=ks,
                          v_scale=vs, calibrated=True)
    dst = [int(x.table[0, 1]), int(x.table[1, 2])]
    keep = [i for i in range(x.num_blocks) if i not in dst]
    assert torch.isfinite(ks.cpu()[keep]).all() and torch.isfinite(vs.cpu()[keep]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_other_caches_are_moved_as_they_are(dtype):
    pkv, dev = _pkv(), "cuda"
    x = Inputs(3, [30, 70], 9, 2, 2, 128, dtype, stale=False)
    path, length = _paths(x, 1)
    args = (torch.from_numpy(path).to(dev), torch.from_numpy(length).to(dev), torch.from_numpy(x.table).to(dev),
            torch.tensor(x.ctx, dtype=torch.int32, device=dev))
    out = []
    for calibrated in (False, True):
        kc, vc = x.kc.to(dev), x.vc.to(dev)
        pkv.paged_tree_commit(kc, vc, *args, calibrated=calibrated)
        out.append((kc, vc))
    assert all(torch.equal(a, b) for a, b in zip(*out))


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("D,Hkv,n", [(128, 2, 7), (64, 1, 20), (128, 1, 64)])
def test_steps_on_a_calibrated_cache(D, Hkv, n, graph):
    """TreeStep(calibrated=True), drafted rows of magnitudes from 2^-6 to 2^6, a
    path chosen at random in every step.  After a step the position that took node
    path[k]'s row holds what that node's position held before, and the confirmed
    prefix what it held, up to the roundings of re-quantising: half a step of a
    normal value, 2^-4 of it, once (scales are powers of two: a second
    re-quantisation of a normal value is exact), and half a subnormal step,
    2^-10 of the scale it is rounded under, once for the source's block and once for
    every raise of the destination's, each at least twice the one before: less than
    2 * 2^-10 of the last scale.  A clipped value would be off by its own size."""
    from paged_kv_gqa_03_gb300.step import TreeStep
    dev, V, Hq = "cuda", 50, 4 * Hkv
    g, rng = torch.Generator().manual_seed(5), np.random.default_rng(D + n)
    nb, prompts = 80, [13, 30, 16, 5]
    B = len(prompts)
    kc, vc = (torch.full((nb, Hkv, 16, D), 0x7F, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.ones(nb, Hkv, device=dev) for _ in range(2))
    step = TreeStep(kc, vc, Hq, torch.bfloat16, 40, n, ks, vs, stream=torch.cuda.Stream(), calibrated=True)
    pkv = _pkv()
    for seq in range(B):
        assert step.bm.allocate(seq, 0)
        slots, _ = step.bm.append_slots([seq] * prompts[seq])
        rows = [torch.randn(prompts[seq], Hkv, D, generator=g).bfloat16().to(dev) for _ in range(2)]
        pkv.paged_kv_append(*rows, kc, vc, torch.tensor(slots, device=dev), ks, vs, calibrated=True)
    step.seqs = list(range(B))
    torch.cuda.synchronize()

    def held(table, b, t):
        """Decoded K and V of position t, [2, Hkv, D], and the block's scales."""
        blk = int(table[b, t // 16])
        out = [c.view(torch.uint8)[blk, :, t % 16].view(torch.float8_e4m3fn).float().cpu() * s[blk].cpu()[:, None]
               for c, s in ((kc, ks), (vc, vs))]
        return torch.stack(out).double(), torch.stack([ks[blk], vs[blk]]).cpu().double()

    crossed = 0
    for _ in range(5):
        parents = [random_parents(n, rng) for _ in range(B)]
        masks = [masks_of(p) for p in parents]
        step.prepare(torch.stack([to_i64(m) for m in masks]).numpy())
        step.upload()
        mag = torch.exp2(torch.randint(-6, 7, (B, n, 1, 1), generator=g).float())
        kn, vn = ((torch.randn(B, n, Hkv, D, generator=g) * mag).bfloat16().to(dev) for _ in range(2))
        q = torch.randn(B, n, Hq, D, generator=g).bfloat16().to(dev)
        out = torch.empty_like(q)
        torch.cuda.synchronize()
        step.launch(q, kn, vn, out)
        step.stream.synchronize()
        # a path to a random deep node: its ancestors' tokens are each node's most likely ones
        target = torch.zeros(B, n, V)
        tokens = torch.randint(10, V, (B, n), generator=g)
        want = []
        for b in range(B):
            leaf = max(rng.integers(0, n, 4).tolist(), key=lambda i: bin(masks[b][i]).count("1"))
            path = [i for i in range(n) if (masks[b][leaf] >> i) & 1]
            for up, c in zip(path, path[1:]):
                target[b, up, 1] = 1.0
                tokens[b, c] = 1
            target[b, path[-1], 2] = 1.0
            want.append(path)
        table, lens = step.bm.export(step.seqs, 40)
        starts = [int(lens[b]) - n for b in range(B)]
        before = [[held(table, b, t) for t in range(starts[b], int(lens[b]))] for b in range(B)]
        prefix = [[held(table, b, t) for t in range(starts[b] // 16 * 16, starts[b])] for b in range(B)]
        args = tokens.to(dev), target.to(dev)
        torch.cuda.synchronize()
        if graph:
            body = torch.cuda.CUDAGraph()
            with torch.cuda.graph(body, stream=step.stream):
                step.verify(*args)
                step.commit()
            with torch.cuda.stream(step.stream):
                body.replay()
        else:
            step.verify(*args)
            step.commit()
        path_len, token = step.finish()
        assert token.tolist() == [2] * B and path_len.tolist() == [len(p) for p in want]
        for b in range(B):
            for k, (f, (was, p_src)) in [(k, (f, before[b][f])) for k, f in enumerate(want[b])]:
                crossed += (starts[b] + f) // 16 != (starts[b] + k) // 16
                now, p_dst = held(table, b, starts[b] + k)
                room = 2.0 ** -4 * was.abs() + 2.0 ** -10 * (p_src + 2 * p_dst)[:, :, None]
                assert ((now - was).abs() <= room).all(), (b, k, f)
            for t, (was, _) in zip(range(starts[b] // 16 * 16, starts[b]), prefix[b]):
                now, p = held(table, b, t)
                assert ((now - was).abs() <= 2.0 ** -4 * was.abs() + 2.0 ** -9 * p[:, :, None]).all(), (b, t)
    assert crossed >= 1
