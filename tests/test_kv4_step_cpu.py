"""Host side of Kv4Step and of steps with rotary positions: what they refuse when they are made, and the memory that they
take.  Nothing is launched."""
import contextlib

import pytest
import torch

from test_tree_cpu import _gpu, _pkv

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


class Rope:     # (a RopeTable, as far as a step looks at it)
    rot_dim = 64


@pytest.mark.parametrize("shape", [(8, 2, 18 * 96), (8, 2, 18 * 64 + 1), (8, 2, 64), (8, 2, 0), (8, 2 * 18 * 64), (8, 2, 16, 64)])
def test_a_cache_of_another_shape_is_refused(shape):
    _pkv()
    from paged_kv_gqa_03_gb300.step import Kv4Step
    with pytest.raises(ValueError, match="4-bit cache"):
        Kv4Step(_gpu(torch.zeros(shape, dtype=torch.uint8)), 4, BF16, 8, stream=object())


def test_a_cache_of_another_type_is_refused():
    _pkv()
    from paged_kv_gqa_03_gb300.step import Kv4Step
    with pytest.raises(TypeError, match="uint8"):
        Kv4Step(_gpu(torch.zeros(8, 2, 18 * 64, dtype=torch.int8)), 4, BF16, 8, stream=object())


def test_a_cache_in_host_memory_is_refused():
    _pkv()
    from paged_kv_gqa_03_gb300.step import Kv4Step
    with pytest.raises(ValueError, match="CUDA tensor"):
        Kv4Step(torch.zeros(8, 2, 18 * 64, dtype=torch.uint8), 4, BF16, 8, stream=object())


def test_a_cache_of_its_shape():
    _pkv()
    from paged_kv_gqa_03_gb300.step import Kv4Step
    for D in (64, 128):
        s = Kv4Step(_gpu(torch.zeros(8, 2, 18 * D, dtype=torch.uint8)), 4, BF16, 8, stream=object())
        assert (s.num_blocks, s.Hkv, s.D) == (8, 2, D)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "kv4"])
def test_rotated_keys_have_a_buffer_only_where_they_are_appended_apart(monkeypatch, kind):
    """FP8 caches: the rotation is a call of its own.  The fused appends write rotated keys to the cache."""
    _pkv()
    from paged_kv_gqa_03_gb300 import step as mod
    if kind == "kv4":
        s = mod.Kv4Step(_gpu(torch.zeros(32, 2, 18 * 64, dtype=torch.uint8)), 4, BF16, 8, stream=object(), rope=Rope())
    else:
        kc, vc = (_gpu(torch.zeros(32, 2, 16, 64, dtype=E4M3 if kind == "fp8" else BF16)) for _ in range(2))
        s = mod.DecodeStep(kc, vc, 4, BF16, 8, stream=object(), rope=Rope())
    monkeypatch.setattr(type(s), "_workspace_bytes", lambda self, B: 256)
    monkeypatch.setattr(torch.cuda, "stream", lambda st: contextlib.nullcontext())
    for seq in range(3):
        assert s.bm.allocate(seq, 20)
    s.seqs = [0, 1, 2]
    s.prepare()
    assert s._q_rot.shape == (3, 4, 64)
    held = [n for n, t in vars(s).items() if isinstance(t, torch.Tensor) and t.shape == (3, 2, 64)
            and t.data_ptr() not in [x.data_ptr() for x in (s.d_k_new, s.d_v_new, s.h_k_new, s.h_v_new)]]
    assert held == (["_k_rot"] if kind == "fp8" else [])
