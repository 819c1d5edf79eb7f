"""Speculative decoding with trees of drafted tokens through TreeStep: append,
attention, verification, commit and the host's release of the rejected
positions, several steps in a row.  A mirror of every sequence's K / V rows, one
list entry per confirmed position, follows the definitions in 64 bits; each
step's output, path, next token, lengths and cached rows are compared with it."""
import numpy as np
import pytest
import torch

from tree_reference import Inputs, check_attention, masks_of, random_parents, to_i64, verify

pytestmark = pytest.mark.gpu


class Mirror(Inputs):
    """The attention inputs of one step, K / V rows from per-sequence lists."""

    def __init__(self, q, rows, masks, nodes, n, Hq, Hkv, D, dtype):
        self.q, self.lists, self.masks, self.nodes = q, rows, masks, list(nodes)
        self.ctx = [len(r[0]) for r in rows]
        self.B, self.n, self.Hq, self.Hkv, self.D = len(rows), n, Hq, Hkv, D
        self.dtype = self.q_dtype = dtype
        self.scale = 1.0 / np.sqrt(D)

    def rows(self, b, h, which, positions):
        if len(positions) == 0:
            return np.zeros((0, self.D))
        return np.stack([self.lists[b][which][t][h] for t in positions])


def _drafts(rng, g, B, n, V, sampled, parents):
    logits = 2.0 * torch.randn(B, n, V, generator=g)
    noisy = logits + 0.5 * torch.randn(B, n, V, generator=g)
    target = torch.softmax(logits, -1) if sampled else logits
    draft = torch.softmax(noisy, -1) if sampled else None
    tokens = torch.zeros(B, n, dtype=torch.int64)
    for b in range(B):
        used = {}
        for i in range(1, n):
            p = parents[b][i]
            if sampled:
                tokens[b, i] = torch.multinomial(draft[b, p], 1, generator=g)[0]
            else:
                k = used[p] = used.get(p, -1) + 1
                tokens[b, i] = noisy[b, p].topk(k + 1).indices[-1]
    return target, draft, tokens, torch.rand(B, n, generator=g) if sampled else None


@pytest.mark.parametrize("from_host", [False, True])
@pytest.mark.parametrize("sampled,n,Hq,Hkv,D,window,ragged", [
    (False, 7, 8, 2, 128, 0, False), (True, 7, 8, 2, 128, 0, True), (True, 33, 16, 1, 128, 0, True),
    (False, 12, 4, 2, 64, 0, True), (True, 1, 4, 1, 128, 0, False), (False, 64, 2, 2, 64, 0, False),
    (True, 9, 8, 2, 128, 40, True)])
def test_steps_in_a_row(from_host, sampled, n, Hq, Hkv, D, window, ragged):
    from paged_kv_gqa_03_gb300.step import TreeStep
    dev, V, steps, dtype = "cuda", 300, 6, torch.bfloat16
    g, rng = torch.Generator().manual_seed(5), np.random.default_rng(5)
    nb, prompts = 96, [37, 5, 37, 130]
    kc, vc = (torch.full((nb, Hkv, 16, D), float("nan"), dtype=dtype, device=dev) for _ in range(2))
    step = TreeStep(kc, vc, Hq, dtype, 24, n, stream=torch.cuda.Stream(), window=window)
    B = len(prompts)
    for seq in (0, 1, 3):
        assert step.bm.allocate(seq, prompts[seq])
    assert step.bm.fork(0, 2)                     # sequence 2 shares 0's blocks, the last of them partly filled
    step.seqs = [0, 1, 2, 3]
    rows = [([], []) for _ in range(B)]
    table, _ = step.bm.export(step.seqs, 24)
    for b in (0, 1, 3):
        for t in range(prompts[b]):
            for which, c in ((0, kc), (1, vc)):
                r = torch.randn(Hkv, D, generator=g).to(dtype)
                c[table[b, t // 16], :, t % 16] = r.to(dev)
                rows[b][which].append(r.double().numpy())
    rows[2] = (list(rows[0][0]), list(rows[0][1]))
    torch.cuda.synchronize()
    free0, first_len = step.bm.num_free(), [len(r[0]) for r in rows]
    longest = 0
    for k in range(steps):
        parents = [random_parents(n, rng) for _ in range(B)]
        masks = [masks_of(p) for p in parents]
        nodes = [int(v) for v in rng.integers(0, n + 1, B)] if ragged else [n] * B
        q = torch.randn(B, n, Hq, D, generator=g).to(dtype)
        kn, vn = (torch.randn(B, n, Hkv, D, generator=g).to(dtype) for _ in range(2))
        mask = torch.stack([to_i64(m) for m in masks]).numpy()
        cow = step.prepare(mask, nodes)
        assert ragged or cow == (1 if k == 0 else 0)  # the first to write into the shared block copies it
        if from_host:
            out = torch.full((B, n, Hq, D), 9.0, dtype=dtype).pin_memory()
            step.stage_inputs(q, kn, vn)
            step.run(out)
        else:
            step.upload()
            out = torch.full((B, n, Hq, D), 9.0, dtype=dtype, device=dev)
            dq, dk, dv = q.to(dev), kn.to(dev), vn.to(dev)
            torch.cuda.synchronize()
            step.launch(dq, dk, dv, out)
        target, draft, tokens, u = _drafts(rng, g, B, n, V, sampled, parents)
        up = lambda t: None if t is None else t.to(dev)  # noqa: E731
        args = [up(tokens), up(target), up(draft), up(u)]
        torch.cuda.synchronize()
        step.verify(*args)
        step.commit()
        path_len, token = step.finish()

        for b in range(B):
            for which, new in ((0, kn), (1, vn)):
                rows[b][which].extend(new[b, i].double().numpy() for i in range(nodes[b]))
        check_attention(out, Mirror(q, rows, masks, nodes, n, Hq, Hkv, D, "bf16"), window, untouched=9.0)
        f = lambda t: None if t is None else t.double().numpy()  # noqa: E731
        path, want_len, want_token = verify(masks, tokens.numpy(), f(target), f(draft), f(u), nodes)
        assert np.array_equal(step.d_path.cpu().numpy(), path)
        assert np.array_equal(path_len, want_len) and np.array_equal(token, want_token)
        longest = max(longest, int(want_len.max()))
        for b in range(B):
            start = len(rows[b][0]) - nodes[b]
            for which in (0, 1):
                r = rows[b][which]
                r[start:] = [r[start + i] for i in path[b, :want_len[b]]]
        table, lens = step.bm.export(step.seqs, 24)
        assert lens.tolist() == [len(r[0]) for r in rows] == step.d_new_lens.tolist()
        for b in range(B):
            lo = max(0, len(rows[b][0]) + 1 - window) if window else 0
            for t in range(lo, len(rows[b][0])):
                for which, c in ((0, kc), (1, vc)):
                    assert np.array_equal(c[table[b, t // 16], :, t % 16].double().cpu().numpy(), rows[b][which][t]), (k, b, t)
    assert n == 1 or longest >= 2
    for seq in step.seqs:
        step.bm.free(seq)
    assert step.bm.num_free() == nb and free0 < nb and first_len == prompts


def test_two_layers_share_a_step():
    """The tables, masks and path of one step on a second layer's cache."""
    import paged_kv_gqa_03_gb300 as pkv
    from paged_kv_gqa_03_gb300.step import TreeStep
    dev, n, H, D = "cuda", 5, 2, 64
    g = torch.Generator().manual_seed(3)
    kc, vc, k2, v2 = (torch.randn(16, H, 16, D, generator=g).half().to(dev) for _ in range(4))
    step = TreeStep(kc, vc, 4, torch.float16, 4, n)
    assert step.bm.allocate(7, 14)
    step.seqs = [7]
    masks = masks_of([-1, 0, 0, 2, 2])
    step.prepare(masks)
    step.upload()
    q = torch.randn(1, n, 4, D, generator=g).half().to(dev)
    kn, vn = (torch.randn(1, n, H, D, generator=g).half().to(dev) for _ in range(2))
    out = torch.empty_like(q)
    step.launch(q, kn, vn, out)
    pkv.paged_kv_append(kn.view(-1, H, D), vn.view(-1, H, D), k2, v2, step.d_slots)
    probs = torch.zeros(1, n, 9, device=dev)
    for i, t in enumerate((4, 1, 6, 2, 3)):
        probs[0, i, t] = 1.0                       # node 0 -> token 4, node 2 -> 6, ...
    step.verify(torch.tensor([[0, 5, 4, 8, 6]], device=dev), probs)
    step.commit()
    step.commit(k2, v2)
    path_len, token = step.finish()
    assert step.d_path.tolist() == [[0, 2, 4, -1, -1]] and path_len.tolist() == [3] and token.tolist() == [3]
    table, lens = step.bm.export([7], 4)
    assert lens.tolist() == [17]
    for c, new in ((kc, kn), (vc, vn), (k2, kn), (v2, vn)):
        for t, i in ((14, 0), (15, 2), (16, 4)):
            assert torch.equal(c[table[0, t // 16], :, t % 16], new[0, i])


def test_refusals():
    from paged_kv_gqa_03_gb300.step import TreeStep
    dev = "cuda"
    kc, vc = (torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16, device=dev) for _ in range(2))
    step = TreeStep(kc, vc, 2, torch.bfloat16, 4, 4)
    assert step.bm.allocate(0, 50)
    step.seqs = [0]
    for masks, lens in (([1, 3, 5], None), ([[1, 3, 5, 7]] * 2, None), ([1, 3, 5, 7], [5]), ([1, 3, 5, 7], [-1]),
                        ([1, 3, 5, 7], [1, 1])):
        with pytest.raises(ValueError):
            step.prepare(masks, lens)
    assert step.bm.export([0], 4)[1].tolist() == [50]
    for _ in range(3):
        step.prepare([1, 3, 5, 9])
    with pytest.raises(MemoryError):               # 62 + 4 tokens do not fit 4 blocks
        step.prepare([1, 3, 5, 9])
    assert step.bm.export([0], 4)[1].tolist() == [62]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_a_step_captured_into_a_graph(dtype):
    """Append, attention, verification and commit as one graph, replayed on
    other inputs in the same buffers: the bits of the eager step."""
    from paged_kv_gqa_03_gb300.step import TreeStep
    dev, n, Hq, Hkv, D, V, B = "cuda", 9, 8, 2, 128, 1000, 3
    g, rng = torch.Generator().manual_seed(4), np.random.default_rng(4)
    fp8 = dtype == torch.float8_e4m3fn
    raw = [torch.randn(40, Hkv, 16, D, generator=g).to(dtype).to(dev) for _ in range(2)]
    kc, vc = (t.clone() for t in raw)
    sc = [torch.full((40, Hkv), 0.01, device=dev) for _ in range(2)] if fp8 else [None, None]
    st = torch.cuda.Stream()
    step = TreeStep(kc, vc, Hq, torch.bfloat16, 16, n, *sc, stream=st)
    step.seqs = [0, 1, 2]
    for seq, length in zip(step.seqs, (100, 7, 32)):
        assert step.bm.allocate(seq, length)
    parents = [random_parents(n, rng) for _ in range(B)]
    step.prepare(torch.stack([to_i64(masks_of(p)) for p in parents]).numpy(), [n, 4, n])
    step.upload()
    mk = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    buf = [mk(B, n, Hq, D).bfloat16().to(dev), mk(B, n, Hkv, D).bfloat16().to(dev), mk(B, n, Hkv, D).bfloat16().to(dev)]
    target, draft, tokens, u = (t.to(dev) for t in _drafts(rng, g, B, n, V, True, parents))
    out = torch.empty_like(buf[0])

    def body():
        step.launch(*buf, out)
        step.verify(tokens, target, draft, u)
        step.commit()

    def reset():
        for c, r in zip((kc, vc), raw):
            c.view(torch.uint8).copy_(r.view(torch.uint8))
        for s in sc:
            if s is not None:
                s.fill_(0.01)
        torch.cuda.synchronize()

    def results():
        st.synchronize()
        return [t.clone().view(torch.uint8) for t in (out, step.d_path, step.d_path_len, step.d_next_token, step.d_new_lens, kc, vc)]

    inputs = []
    for _ in range(3):
        t, d, k, x = _drafts(rng, g, B, n, V, True, parents)
        inputs.append([mk(B, n, Hq, D).bfloat16(), mk(B, n, Hkv, D).bfloat16(), mk(B, n, Hkv, D).bfloat16(), t, d, k, x])

    def fill(values):
        for b, v in zip(buf + [target, draft, tokens, u], values):
            b.copy_(v)
        reset()

    eager = []
    for values in inputs:
        fill(values)
        body()
        eager.append(results())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        body()
    for values, want in zip(inputs, eager):
        fill(values)
        with torch.cuda.stream(st):
            graph.replay()
        for a, b in zip(results(), want):
            assert torch.equal(a, b)
    assert any(not torch.equal(a, b) for a, b in zip(eager[0], eager[1]))
