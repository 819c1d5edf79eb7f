"""CPU checks of what the tree calls refuse and keep: tensors that share memory,
limits of each route, and who owns a workspace.  Nothing is launched."""
import gc
import weakref

import pytest
import torch

from test_tree_cpu import OnGpu, _gpu, _pkv, _recorded
from tree_reference import Inputs


def test_commit_refuses_new_lens_on_the_memory_it_reads():
    """C: new_lens[b] is written by one warp while others still read the rest."""
    pkv = _pkv()
    L = pkv.lib()
    # pointers that nothing follows: the call ends before any launch
    at = dict(k=1 << 20, v=2 << 20, path=0x1000, plen=0x2000, bt=0x3000, cl=0x4000, tl=0x5000, nl=0x6000)

    def call(**kw):
        a = dict(at, **kw)
        return L.paged_tree_commit(a["k"], a["v"], 2, None, None, a["path"], a["plen"], a["bt"], 4, a["cl"], a["tl"], a["nl"],
                                   2, 8, 2, 128, 10, None)
    for name, size in (("cl", 8), ("tl", 8), ("plen", 8), ("path", 64), ("bt", 32)):
        for off in (0, 4, -4, size - 4):
            assert call(nl=at[name] + off) == pkv.PKV_EINVAL, (name, off)


def test_binding_refuses_new_lens_on_the_memory_it_reads(monkeypatch):
    pkv = _pkv()
    x = Inputs(1, [40, 33], 4, 4, 2, 64, "bf16")
    made = _recorded(monkeypatch, pkv)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    lens = i32(6)
    good = dict(k_cache=x.kc, v_cache=x.vc, path=i32(2, 4), path_len=lens[:2], block_table=torch.from_numpy(x.table),
                context_lens=lens[2:4], tree_lens=i32(2), new_lens=lens[4:])
    pkv.paged_tree_commit(**{k: _gpu(v) for k, v in good.items()})   # parts of one tensor that do not meet
    assert len(made) == 1
    for bad in (good["context_lens"], good["path_len"], good["tree_lens"], good["path"].view(-1)[2:4], lens[3:5],
                good["block_table"].view(-1)[:2]):
        with pytest.raises(ValueError, match="share memory"):
            pkv.paged_tree_commit(**{k: _gpu(v) for k, v in dict(good, new_lens=bad).items()})
    assert len(made) == 1


def _attention_calls(x):
    """The two calls that allocate a workspace when given none."""
    table, lens = torch.from_numpy(x.table), torch.tensor(x.ctx, dtype=torch.int32)
    common = dict(out=torch.empty_like(x.q), q=x.q, k_cache=x.kc, v_cache=x.vc, block_table=table, context_lens=lens, scale=0.1)
    return [("paged_tree_attention", dict(common, tree_mask=x.mask)), ("paged_decode_attention", common)]


def _allocations(monkeypatch):
    """Every torch.empty, on "device 0": a list of weak references."""
    made, real = [], torch.empty

    def empty(*a, **kw):
        t = real(*a, **kw).as_subclass(OnGpu)
        made.append(weakref.ref(t))
        return t
    monkeypatch.setattr(torch, "empty", empty)
    return made


@pytest.mark.parametrize("which", [0, 1])
def test_a_prepared_call_keeps_the_workspace_it_allocated(monkeypatch, which):
    pkv = _pkv()
    x = Inputs(1, [40, 33], 4, 4, 2, 64, "bf16")
    calls = _recorded(monkeypatch, pkv)
    monkeypatch.setattr(pkv, f"paged_{('tree', 'decode')[which]}_workspace_bytes", lambda *a, **kw: 4096)
    name, kw = _attention_calls(x)[which]
    kw = {k: _gpu(v) for k, v in kw.items()}
    made = _allocations(monkeypatch)
    call = getattr(pkv, name)(**kw, prepare=True)
    gc.collect()
    assert len(made) == 1 and made[0]() is not None and made[0]().data_ptr() in call.args
    assert call.workspace is made[0]()
    call()
    assert calls[-1][0].startswith(name) and made[0]().data_ptr() in calls[-1][1]
    own = torch.empty(4096, dtype=torch.uint8)
    assert getattr(pkv, name)(**kw, workspace=own, prepare=True).workspace is own
    del call
    gc.collect()
    assert made[0]() is None


@pytest.mark.parametrize("which", [0, 1])
def test_an_allocated_workspace_belongs_to_the_calls_stream(monkeypatch, which):
    """Allocated as the current stream's memory it would be handed out again,
    once dropped, while a call on another stream still runs."""
    pkv = _pkv()
    x = Inputs(1, [40, 33], 4, 4, 2, 64, "bf16")
    _recorded(monkeypatch, pkv)
    monkeypatch.setattr(pkv, f"paged_{('tree', 'decode')[which]}_workspace_bytes", lambda *a, **kw: 4096)
    name, kw = _attention_calls(x)[which]
    kw = {k: _gpu(v) for k, v in kw.items()}
    inside, at = [], []

    class Stream:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            inside.append(self.s)

        def __exit__(self, *a):
            inside.pop()
    monkeypatch.setattr(torch.cuda, "stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s, device=None: ("raw", s))
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: at.append(list(inside)) or real(*a, **k).as_subclass(OnGpu))
    side = object()
    for stream, want in ((None, []), (side, [side]), (77, [("raw", 77)])):
        getattr(pkv, name)(**kw, stream=stream)
        assert at.pop() == want and not at


@pytest.mark.parametrize("route,shape,over", [
    # 64 sequences with room for 131072 positions each, the widest tree on 64 / 8 heads
    ("auto", dict(B=64, mb=8192, Hq=64, Hkv=8, n=64, cd=2), False),
    ("auto", dict(B=64, mb=8192, Hq=64, Hkv=8, n=64, cd=3), False),
    # tiles: B * Hkv * ceil(mb / 8) either side of 2^31
    ("auto", dict(B=2048, mb=(1 << 20) - 8, Hq=64, Hkv=8, n=64, cd=2), False),
    ("auto", dict(B=2048, mb=1 << 20, Hq=64, Hkv=8, n=64, cd=2), True),
    ("tiles", dict(B=2048, mb=(1 << 20) - 8, Hq=8, Hkv=8, n=1, cd=1), False),
    # units: B * Hkv * ceil(R / rows) * mb, of 2 rows (fp32), 8 (16-bit) and 16 (fp8)
    ("auto", dict(B=4, mb=(1 << 18) - 1, Hq=64, Hkv=8, n=64, cd=0), False),
    ("auto", dict(B=4, mb=1 << 18, Hq=64, Hkv=8, n=64, cd=0), True),
    ("units", dict(B=64, mb=65535, Hq=64, Hkv=8, n=64, cd=2), False),
    ("units", dict(B=64, mb=65536, Hq=64, Hkv=8, n=64, cd=2), True),
    ("units", dict(B=64, mb=131071, Hq=64, Hkv=8, n=64, cd=3), False),
    ("units", dict(B=64, mb=131072, Hq=64, Hkv=8, n=64, cd=3), True),
    ("auto", dict(B=4096, mb=65535, Hq=8, Hkv=8, n=8, cd=2), False),   # more than the tile kernel's plan holds
    ("auto", dict(B=4096, mb=65536, Hq=8, Hkv=8, n=8, cd=2), True),
    # query rows
    ("auto", dict(B=2048, mb=1, Hq=16376, Hkv=8, n=64, cd=2), False),
    ("auto", dict(B=2048, mb=1, Hq=16384, Hkv=8, n=64, cd=2), True),
    ("auto", dict(B=1, mb=1, Hq=(1 << 31) - 8, Hkv=1, n=64, cd=2), True)])
def test_attention_refuses_what_its_route_cannot_count(route, shape, over):
    """A long table alone does not refuse a call that the route's counts hold."""
    pkv = _pkv()
    a = dict(out=16, q=16, qd=2, k=16, v=16, cd=2, ks=16, vs=16, bt=16, mb=4, cl=16, mask=16, per=1, tl=None, B=2, n=4, w=0,
             Hq=8, Hkv=2, D=128, nb=10, scale=0.1, ws=256, wsb=0, st=None)
    a.update(shape)
    a["qd"] = {3: 2}.get(a["cd"], a["cd"])
    was = pkv.pkv_set_route("tree", route)
    try:
        rc = pkv.lib().paged_tree_attention(*a.values())
    finally:
        pkv.pkv_set_route("tree", was)
    # (no workspace: a call that is not refused for its shape ends there, or without a GPU)
    assert rc == pkv.PKV_EUNSUPPORTED if over else rc in (pkv.PKV_EWORKSPACE, pkv.PKV_ECUDA), rc
