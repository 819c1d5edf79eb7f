"""Workspaces that the binding allocates itself, for calls on another stream than
the current one."""
import pytest
import torch

from tree_reference import Inputs, check_attention

pytestmark = pytest.mark.gpu


def _args(x):
    dev = "cuda"
    return (x.q.to(dev), x.kc.to(dev), x.vc.to(dev), torch.from_numpy(x.table).to(dev),
            torch.tensor(x.ctx, dtype=torch.int32, device=dev))


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("tree", [True, False])
def test_a_dropped_workspace_is_handed_out_behind_the_call(tree, raw):
    """The workspace of a call on a side stream is that stream's memory: after it
    is dropped the current stream gets other memory while the call may run."""
    import paged_kv_gqa_03_gb300 as pkv
    x = Inputs(5, [3000, 700], 5, 8, 2, 128, "bf16", kind="chain")
    q, kc, vc, table, lens = _args(x)
    mask, st = x.mask.cuda(), torch.cuda.Stream()
    outs = [torch.empty_like(q) for _ in range(4)]
    torch.cuda.synchronize()
    where = st.cuda_stream if raw else st
    for out in outs:
        if tree:
            ws = pkv.paged_tree_attention(out, q, kc, vc, table, lens, mask, x.scale, stream=where)
        else:
            ws = pkv.paged_decode_attention(out, q, kc, vc, table, lens, x.scale, stream=where)
        at, n = ws.data_ptr(), ws.numel()
        del ws
        other = torch.empty(n, dtype=torch.uint8, device="cuda")
        assert not at <= other.data_ptr() < at + n
        other.fill_(255)                        # (on the current stream, while the call runs)
    torch.cuda.synchronize()
    for out in outs:
        check_attention(out, x)


def test_default_streams():
    """No stream, and the default stream's handle (0)."""
    import paged_kv_gqa_03_gb300 as pkv
    x = Inputs(6, [300, 70], 5, 8, 2, 128, "bf16", kind="chain")
    q, kc, vc, table, lens = _args(x)
    for stream in (None, 0, torch.cuda.default_stream()):
        out = torch.empty_like(q)
        ws = pkv.paged_tree_attention(out, q, kc, vc, table, lens, x.mask.cuda(), x.scale, stream=stream)
        assert pkv.paged_decode_status(ws) == (0, 0)
        check_attention(out, x)


@pytest.mark.parametrize("tree", [True, False])
def test_a_steps_buffers_belong_to_its_stream(tree):
    """By torch's own record of which stream a segment was allocated for."""
    from paged_kv_gqa_03_gb300.step import DecodeStep, TreeStep
    st = torch.cuda.Stream()
    kc, vc = (torch.zeros(16, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    step = TreeStep(kc, vc, 4, torch.bfloat16, 8, 4, stream=st) if tree else DecodeStep(kc, vc, 4, torch.bfloat16, 8, stream=st)
    for seq in (0, 1):
        assert step.bm.allocate(seq, 20)
    step.seqs = [0, 1]
    step.prepare(*([[1, 3, 5, 9]] if tree else []))
    segments = torch.cuda.memory_snapshot()
    mine = [step._dev.buf, step.workspace] + ([step.d_path, step.d_path_len, step.d_new_lens, step.d_next_token] if tree else [])
    for t in mine:
        at = [s for s in segments if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]]
        assert len(at) == 1 and at[0]["stream"] == st.cuda_stream
