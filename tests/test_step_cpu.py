"""CPU checks of the step objects' host side: what they refuse, what they keep and
which stream their memory belongs to.  Nothing is launched."""
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
