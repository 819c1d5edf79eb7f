"""CPU checks of the tree calls: refusals at the C boundary and in the binding
(nothing is launched), the block manager's truncate, and the reference forms
that the GPU tests compare with."""
import ctypes
import os

import numpy as np
import pytest
import torch

import oracle
from tree_reference import (Inputs, attention, commit, masks_of, parent_of, random_parents, to_i64, verify_one)


def _pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_gqa_03_gb300 as pkv
    return pkv


def test_attention_refusals():
    pkv = _pkv()
    L = pkv.lib()

    def call(**kw):
        a = dict(out=16, q=16, qd=2, k=16, v=16, cd=2, ks=None, vs=None, bt=16, mb=4, cl=16, mask=16, per=1, tl=None,
                 B=2, n=4, w=0, Hq=8, Hkv=2, D=128, nb=10, scale=0.1, ws=256, wsb=0, st=None)
        a.update(kw)
        return L.paged_tree_attention(*a.values())
    for kw in (dict(n=0), dict(n=65), dict(B=-1), dict(Hq=6, Hkv=4), dict(Hkv=0), dict(nb=0), dict(mb=0), dict(w=-1),
               dict(per=2), dict(per=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(out=None), dict(q=None), dict(k=None), dict(v=None), dict(bt=None),
               dict(cl=None), dict(mask=None), dict(mask=20), dict(q=18), dict(out=8), dict(k=24), dict(qd=3, cd=3),
               dict(cd=9), dict(qd=-1), dict(cd=3, ks=16), dict(cd=3, vs=16)):
        assert call(**kw) == pkv.PKV_EINVAL, kw
    for kw in (dict(D=96), dict(qd=1), dict(cd=0), dict(cd=3, qd=0, ks=16, vs=16), dict(mb=(1 << 26) + 1),
               dict(nb=1 << 40)):
        assert call(**kw) == pkv.PKV_EUNSUPPORTED, kw
    assert call(B=0) == pkv.PKV_OK
    size = ctypes.c_size_t(0)
    assert L.paged_tree_workspace_bytes(2, 0, 8, 2, 128, 2, 2, ctypes.byref(size)) == pkv.PKV_EINVAL
    assert L.paged_tree_workspace_bytes(2, 4, 8, 2, 128, 2, 2, None) == pkv.PKV_EINVAL
    assert L.paged_tree_workspace_bytes(2, 4, 8, 2, 80, 2, 2, ctypes.byref(size)) == pkv.PKV_EUNSUPPORTED


def test_verify_refusals():
    pkv = _pkv()
    L = pkv.lib()

    def call(**kw):
        a = dict(path=16, plen=16, tok=16, draft_tokens=16, mask=16, per=1, tl=None, t=16, ldt=100, d=16, ldd=100, dt=0,
                 u=16, B=2, n=4, V=100, st=None)
        a.update(kw)
        return L.paged_tree_verify(*a.values())
    for kw in (dict(n=0), dict(n=65), dict(B=-1), dict(V=0), dict(per=2), dict(ldt=99), dict(ldd=99), dict(u=None),
               dict(path=None), dict(plen=None), dict(tok=None), dict(draft_tokens=None), dict(mask=None), dict(t=None),
               dict(t=18), dict(d=17), dict(mask=12), dict(dt=7)):
        assert call(**kw) == pkv.PKV_EINVAL, kw
    for kw in (dict(dt=3), dict(V=(1 << 30) + 1, ldt=1 << 31, ldd=1 << 31)):
        assert call(**kw) == pkv.PKV_EUNSUPPORTED, kw
    assert call(B=0) == pkv.PKV_OK


def test_commit_refusals():
    pkv = _pkv()
    L = pkv.lib()

    def call(**kw):
        a = dict(k=16, v=16, cd=2, ks=None, vs=None, path=16, plen=16, bt=16, mb=4, cl=16, tl=None, nl=None, B=2, n=4,
                 Hkv=2, D=128, nb=10, st=None)
        a.update(kw)
        return L.paged_tree_commit(*a.values())
    for kw in (dict(n=0), dict(n=65), dict(B=-1), dict(Hkv=0), dict(nb=0), dict(mb=0), dict(cd=5), dict(k=None),
               dict(v=None), dict(path=None), dict(plen=None), dict(bt=None), dict(cl=None), dict(k=24), dict(v=8),
               dict(cd=3, ks=16), dict(cd=3, vs=16)):
        assert call(**kw) == pkv.PKV_EINVAL, kw
    for kw in (dict(D=80), dict(mb=(1 << 26) + 1)):
        assert call(**kw) == pkv.PKV_EUNSUPPORTED, kw
    assert call(B=0) == pkv.PKV_OK


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on device 0: the binding's checks run
    without a GPU (the C call behind them is replaced)."""
    is_cuda = True

    def get_device(self):
        return 0


def _gpu(x):
    return x.as_subclass(OnGpu) if isinstance(x, torch.Tensor) else x


def _recorded(monkeypatch, pkv):
    """Replaces the C calls and what asks for a GPU; the list of calls made."""
    made = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: made.append((name, a)) or 0
    monkeypatch.setattr(pkv, "_L", Lib())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(pkv, "_stream", lambda s, d=None: 0)
    return made


def test_binding_refusals(monkeypatch):
    """Shapes, types, strides and places are checked before the call."""
    pkv = _pkv()
    x = Inputs(1, [40, 33], 4, 4, 2, 64, "bf16")
    made = _recorded(monkeypatch, pkv)
    table, lens = torch.from_numpy(x.table), torch.tensor(x.ctx, dtype=torch.int32)
    ones = torch.ones(x.num_blocks, 2)

    def refused(fn, base, exc, **kw):
        before = len(made)
        with pytest.raises(exc):
            fn(**{k: _gpu(v) for k, v in {**base, **kw}.items()})
        assert len(made) == before
        for name, v in kw.items():   # the same call is fine otherwise
            assert name in base or name in ("tree_lens", "k_scale", "uniforms", "draft_probs", "new_lens"), name
    good = dict(out=torch.empty_like(x.q), q=x.q, k_cache=x.kc, v_cache=x.vc, block_table=table, context_lens=lens,
                tree_mask=x.mask, scale=0.1, workspace=torch.empty(256, dtype=torch.uint8))
    f = pkv.paged_tree_attention
    f(**{k: _gpu(v) for k, v in good.items()})
    assert made[-1][0] == "paged_tree_attention" and made[-1][1][12] == 1       # one mask per sequence
    f(**{k: _gpu(v) for k, v in {**good, "tree_mask": x.mask[0].contiguous()}.items()})
    assert made[-1][1][12] == 0
    wide = torch.zeros(2, 4, 4, 128, dtype=torch.bfloat16)
    for kw in (dict(q=x.q[0]), dict(out=x.q[:, :3]), dict(v_cache=x.vc[:1]), dict(k_cache=x.kc[:, :, :8]),
               dict(block_table=table[0]), dict(block_table=table[:1]), dict(context_lens=lens[:1]),
               dict(tree_mask=x.mask[:, :3]), dict(tree_mask=x.mask[:1]), dict(tree_lens=lens[:1]),
               dict(k_scale=ones[:, :1]), dict(q=wide, out=wide), dict(q=x.q.transpose(1, 2).contiguous().transpose(1, 2)),
               dict(tree_mask=torch.stack([x.mask, x.mask], 1)[:, 0])):
        refused(f, good, ValueError, **kw)
    for kw in (dict(out=x.q.float()), dict(v_cache=x.vc.half()), dict(tree_mask=x.mask.int()), dict(context_lens=lens.long()),
               dict(block_table=table.long()), dict(tree_lens=lens.long()), dict(k_scale=ones.double())):
        refused(f, good, TypeError, **kw)
    for name in ("q", "k_cache", "v_cache", "block_table", "context_lens", "tree_mask", "workspace", "out"):
        with pytest.raises(ValueError):   # one tensor on the host
            f(**{k: v if k == name else _gpu(v) for k, v in good.items()})
    B, n, V = 2, 4, 50
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    good = dict(path=i32(B, n), path_len=i32(B), next_token=torch.zeros(B, dtype=torch.int64),
                draft_tokens=torch.zeros(B, n, dtype=torch.int64), tree_mask=x.mask, target_probs=torch.zeros(B, n, V))
    f = pkv.paged_tree_verify
    f(**{k: _gpu(v) for k, v in good.items()})
    for kw in (dict(path=i32(B, 3)), dict(path_len=i32(3)), dict(next_token=torch.zeros(3, dtype=torch.int64)),
               dict(draft_tokens=torch.zeros(8, dtype=torch.int64)), dict(uniforms=torch.zeros(B)),
               dict(target_probs=torch.zeros(B, V)), dict(tree_lens=lens[:1]), dict(draft_probs=torch.zeros(B, n, V + 1)),
               dict(target_probs=torch.zeros(B, n, 2 * V)[..., ::2])):
        refused(f, good, ValueError, **kw)
    for kw in (dict(draft_tokens=i32(B, n)), dict(next_token=i32(B)), dict(uniforms=torch.zeros(B, n).double()),
               dict(draft_probs=torch.zeros(B, n, V).half()), dict(path=i32(B, n).long())):
        refused(f, good, TypeError, **kw)
    good = dict(k_cache=x.kc, v_cache=x.vc, path=i32(B, n), path_len=i32(B), block_table=table, context_lens=lens)
    f = pkv.paged_tree_commit
    f(**{k: _gpu(v) for k, v in good.items()})
    for kw in (dict(path=i32(8)), dict(path_len=i32(1)), dict(block_table=table[:1]), dict(new_lens=i32(3)),
               dict(tree_lens=i32(1)), dict(k_cache=x.kc[0])):
        refused(f, good, ValueError, **kw)
    refused(f, good, TypeError, new_lens=torch.zeros(B, dtype=torch.int64))


def test_other_device_is_refused(monkeypatch):
    pkv = _pkv()
    x = Inputs(1, [40, 33], 4, 4, 2, 64, "bf16")
    made = _recorded(monkeypatch, pkv)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    path = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="current device"):
        pkv.paged_tree_commit(*(_gpu(t) for t in (x.kc, x.vc, path, path[:, 0], torch.from_numpy(x.table), path[:, 0])))
    assert made == []


def test_row_strides_of_probabilities():
    """_rows takes rows a fixed distance apart and nothing else."""
    pkv = _pkv()
    rows = lambda t: pkv._rows(_gpu(t), "t", t.dtype, *t.shape, 0)  # noqa: E731
    t = torch.zeros(3, 5, 40)
    assert rows(t)[1] == 40
    assert rows(t[..., :33])[1] == 40
    assert rows(t[:, :1, :33])[1] == 200
    assert rows(t[:1])[1] == 40
    for bad in (t[:, :4], t.transpose(0, 1).contiguous().transpose(0, 1), t[..., ::2], t[:, ::2], t[:1].expand(3, 5, 40),
                t[:, :1].expand(3, 5, 40)):
        with pytest.raises(ValueError):
            rows(bad)


# ---------------------------------------------------------------------------
def test_truncate():
    pkv = _pkv()
    bm = pkv.BlockManager(8)
    assert bm.allocate(1, 20)
    table, _ = bm.export([1], 8)
    slots, _ = bm.append_slots([1] * 40)                       # 20 .. 59: blocks 2 and 3 open
    assert bm.num_free() == 4 and bm.num_tokens(1) == 60
    bm.truncate(1, 60)
    assert bm.num_free() == 4
    bm.truncate(1, 33)
    assert bm.num_free() == 5 and bm.num_tokens(1) == 33
    assert bm.append_slots([1])[0] == [slots[13]]               # position 33 again, in its block
    bm.truncate(1, 32)
    assert bm.num_free() == 6
    assert bm.append_slots([1])[0] == [slots[12]]               # the block just released is the next one taken
    bm.truncate(1, 0)
    assert bm.num_free() == 8 and bm.num_tokens(1) == 0
    assert bm.export([1], 8)[1].tolist() == [0]


def test_truncate_shared_and_released_blocks():
    pkv = _pkv()
    bm = pkv.BlockManager(16)
    assert bm.allocate(1, 40) and bm.fork(1, 2)
    blocks = bm.export([1], 4)[0][0]
    bm.truncate(2, 20)
    assert bm.refcount(int(blocks[2])) == 1 and bm.refcount(int(blocks[1])) == 2 and bm.num_free() == 13
    slots, cow = bm.append_slots([2])                           # into a shared block: copy on write
    assert len(cow) == 1 and cow[0][0] == blocks[1]
    bm.free(1)
    bm.append_slots([2] * 60)
    bm.release_outside_window(2, 16)
    free = bm.num_free()
    bm.truncate(2, 70)
    assert bm.num_free() == free + 1
    bm.truncate(2, 0)                                           # -1 entries are skipped
    assert bm.num_free() == 16


def test_truncate_adopted_blocks_and_errors():
    pkv = _pkv()
    bm = pkv.BlockManager(4)
    bm.adopt(1, [3, 1], 30)
    bm.adopt(2, [3], 16)
    bm.truncate(1, 5)
    assert bm.num_free() == 3 and bm.refcount(3) == 2 and bm.refcount(1) == 0
    for seq, n, rc in ((1, -1, pkv.PKV_EINVAL), (1, 6, pkv.PKV_ERANGE), (9, 0, pkv.PKV_ENOTFOUND)):
        with pytest.raises(pkv.PagedKVError) as e:
            bm.truncate(seq, n)
        assert e.value.status == rc
    assert bm.num_tokens(1) == 5
    assert pkv.lib().pkv_bm_truncate(None, 0, 0) == pkv.PKV_EINVAL


# ---------------------------------------------------------------------------
def test_reference_chain_is_the_oracles_causal_decode():
    """A chain's tree attention is the multi-token causal decode."""
    for window in (0, 9):
        x = Inputs(3, [9, 40, 77], 5, 4, 2, 64, "f32", kind="chain", stale=False)
        ref = oracle.decode(x.q, "f32", x.kc, x.vc, "f32", x.table, np.array(x.ctx, dtype=np.int32), scale=x.scale,
                            window=window)
        if window:   # the chain's own tokens are the mask's; hide the ones out of the window
            x.masks = [[m & ~((1 << max(0, i + 1 - window)) - 1) for i, m in enumerate(ms)] for ms in x.masks]
        assert np.abs(attention(x, window)[0] - ref).max() < 1e-12


def test_reference_parents():
    rng = np.random.default_rng(0)
    for kind in ("chain", "random", "star"):
        p = random_parents(64, rng, kind)
        m = masks_of(p)
        assert [parent_of(m, i) for i in range(64)] == p
    assert to_i64([1 << 63]).tolist() == [-(1 << 63)]


@pytest.mark.parametrize("mode", ["sample", "topk"])
@pytest.mark.parametrize("kids", [1, 2, 3])
def test_reference_verification_keeps_the_targets_distribution(mode, kids):
    """Averaged over the drafts and the random numbers, the first token that
    comes out of a node is distributed as the target (the point of the rule):
    the children's numbers and the draw run over grids."""
    V, N = 3, 12
    rng = np.random.default_rng(4)
    p = rng.dirichlet(np.ones(V))
    q = rng.dirichlet(np.ones(V))
    masks = masks_of([-1] + [0] * kids)
    mid = (np.arange(N) + 0.5) / N
    got = np.zeros(V)
    target = np.tile(p, (kids + 1, 1))
    draft = np.tile(q, (kids + 1, 1)) if mode == "sample" else None
    picks = np.array(np.meshgrid(*[np.arange(V)] * kids)).reshape(kids, -1).T if mode == "sample" else [np.arange(kids)]
    us = np.array(np.meshgrid(*[mid] * kids)).reshape(kids, -1).T
    draws = (np.arange(200) + 0.5) / 200
    for pick in picks:
        weight = np.prod(q[pick]) if mode == "sample" else 1.0
        tokens = np.concatenate([[0], pick])
        for u in us:
            path, _ = verify_one(masks, tokens, target, draft, np.concatenate([[0.5], u]), kids + 1)
            if len(path) > 1:
                got[tokens[path[1]]] += weight / len(us)
            else:
                t = [verify_one(masks, tokens, target, draft, np.concatenate([[d], u]), kids + 1)[1] for d in draws[::10]]
                got += weight / len(us) * np.bincount(t, minlength=V) / len(t)
    # a grid of N numbers per child and 20 draws: within 1 / N per child and 1 / 20 of the draws
    assert np.abs(got - p).max() < kids / N / 2 + 1 / 40, (got, p)


def test_reference_commit_of_a_chain_with_a_hole():
    x = Inputs(6, [30], 6, 1, 1, 64, "f32", stale=False)
    path = np.array([[0, 2, 3, 5, -1, -1]], dtype=np.int32)
    k, _ = commit(x, path, np.array([4]))
    rows = lambda raw: [raw[x.table[0, t // 16], 0, t % 16].tobytes() for t in range(24, 30)]  # noqa: E731
    was = rows(x.kc.view(torch.uint8).numpy().reshape(k.shape))
    assert rows(k) == [was[0], was[2], was[3], was[5], was[4], was[5]]


def test_header_declares_the_tree_calls():
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "pagedkv.h")).read()
    for name in ("paged_tree_attention", "paged_tree_workspace_bytes", "paged_tree_verify", "paged_tree_commit",
                 "pkv_bm_truncate"):
        assert f"int {name}(" in src
