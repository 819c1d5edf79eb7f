"""CPU checks of the step objects' host side: what they refuse, what they keep and
which stream their memory belongs to.  Nothing is launched."""
import contextlib

import pytest
import torch

from test_tree_cpu import _gpu, _pkv, _recorded


def _step(monkeypatch, tree=True, B=2, **kw):
    """A step on "device 0" whose C calls are recorded; (step, calls)."""
    pkv = _pkv()
    from paged_kv_gqa_03_gb300 import step as mod
    kc, vc = (_gpu(torch.zeros(32, 2, 16, 64, dtype=torch.bfloat16)) for _ in range(2))
    args = (kc, vc, 4, torch.bfloat16, 8) + ((4,) if tree else ())
    s = (mod.TreeStep if tree else mod.DecodeStep)(*args, stream=object(), **kw)
    monkeypatch.setattr(type(s), "_workspace_bytes", lambda self, B: 256)
    monkeypatch.setattr(torch.cuda, "stream", lambda st: contextlib.nullcontext())
    for seq in range(B):
        assert s.bm.allocate(seq, 20)
    s.seqs = list(range(B))
    return s, pkv


def test_a_sequence_appears_once(monkeypatch):
    """Twice in one step its nodes would be appended behind each other, and both
    rows attend the second ones."""
    s, _ = _step(monkeypatch)
    for seqs in ([0, 0], [1, 0, 1]):
        with pytest.raises(ValueError, match="once"):
            s.prepare([1, 3, 5, 9], seqs=seqs)
    assert [s.bm.num_tokens(i) for i in (0, 1)] == [20, 20]
    s.prepare([1, 3, 5, 9], seqs=[1, 0])
    assert s.h_lens.tolist() == [24, 24]


@pytest.mark.parametrize("tree", [True, False])
def test_a_marshalled_call_is_not_reused_for_another_tensor_at_its_address(monkeypatch, tree):
    """The checks of the first call say nothing of a smaller, strided or otherwise
    typed tensor at the same address: it would be read or written past its end."""
    s, pkv = _step(monkeypatch, tree)
    if tree:
        s.prepare([1, 3, 5, 9])
    else:
        s.prepare()
    made = _recorded(monkeypatch, pkv)
    for name in ("d_table", "d_lens", "d_slots", "_ws") + (("d_mask", "d_tree_lens") if tree else ()):
        setattr(s, name, _gpu(getattr(s, name)))
    L = (4,) if tree else ()
    q, out = (_gpu(torch.zeros(2, *L, 4, 64, dtype=torch.bfloat16)) for _ in range(2))
    kn, vn = (_gpu(torch.zeros(2, *L, 2, 64, dtype=torch.bfloat16)) for _ in range(2))
    s.launch(q, kn, vn, out)
    assert len(made) == 2
    args = [m[1] for m in made]
    s.launch(q, kn, vn, out)
    assert [m[1] for m in made[2:]] == args          # the same buffers: the same call
    bad = [out[:1], out.view(torch.float16), out.transpose(-1, -2)]
    for o in bad:
        assert o.data_ptr() == out.data_ptr()
        before = len(made)
        if o.dtype != out.dtype and not tree:
            continue                                 # (the decode call takes its type from q)
        with pytest.raises((ValueError, TypeError)):
            s.attend(q, o)
        assert len(made) == before
    with pytest.raises((ValueError, TypeError, RuntimeError)):   # (several nodes' rows: refused by view)
        s.launch(q, kn.transpose(-1, -2), vn, out)


def test_a_graph_is_not_replayed_into_another_output(monkeypatch):
    """run() keeps one graph per output buffer: one of another shape at the same
    address gets its own."""
    s, pkv = _step(monkeypatch, False)
    s.prepare()
    h = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    monkeypatch.setattr(torch.Tensor, "is_pinned", lambda self: True)
    ran = []

    class Stream:
        cuda_stream = 5
    s.stream, s._ran = Stream(), True
    monkeypatch.setattr(s, "_graph_body", lambda o: ran.append(tuple(o.shape)))

    class Graph:
        def replay(self):
            pass

    class Event:
        def record(self, st):
            pass

    class Context:
        def __init__(self, *a, **kw):
            pass

        def __enter__(self):
            pass

        def __exit__(self, *a):
            pass
    for name, v in (("CUDAGraph", Graph), ("Event", Event), ("graph", Context), ("stream", Context)):
        monkeypatch.setattr(torch.cuda, name, v)
    s.run(h)
    s.run(h)
    assert ran == [(2, 4, 64)]
    s.run(h[:1])
    assert ran == [(2, 4, 64), (1, 4, 64)]


@pytest.mark.parametrize("tree", [True, False])
def test_device_buffers_are_the_steps_streams_memory(monkeypatch, tree):
    """Memory of the current stream may still be in use there when the step's
    stream writes it."""
    s, pkv = _step(monkeypatch, tree)
    inside, made, real = [], [], torch.empty

    class Context:
        def __init__(self, st):
            self.st = st

        def __enter__(self):
            inside.append(self.st)

        def __exit__(self, *a):
            inside.pop()

    def empty(*a, **kw):
        if kw.get("device") != s.device:
            return real(*a, **kw)
        made.append(list(inside))
        return real(*a, **dict(kw, device="cpu"))
    s.device = torch.device("cuda", 0)
    monkeypatch.setattr(torch.cuda, "stream", Context)
    monkeypatch.setattr(torch, "empty", empty)
    s._buffers(2)
    assert len(made) == (6 if tree else 2) and all(m == [s.stream] for m in made)


@pytest.mark.parametrize("tree", [True, False])
def test_another_batch_size_waits_for_the_copies_in_flight(monkeypatch, tree):
    """The pinned staging buffers of the old size are let go of, and their memory
    may be written by the next owner: not before the copies out of them are done."""
    s, pkv = _step(monkeypatch, tree)
    prepare = lambda **kw: s.prepare(*([[1, 3, 5, 9]] if tree else []), **kw)  # noqa: E731
    prepare()
    waited = []

    class Event:
        def __init__(self, name):
            self.name = name

        def synchronize(self):
            waited.append(self.name)
    s._host[0].done, s._host[1].done = Event(0), Event(1)
    prepare(seqs=[1])
    assert sorted(waited[:2]) == [0, 1] and s.h_lens.numel() == 1
