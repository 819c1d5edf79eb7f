"""Whole steps: Kv4Step, and DecodeStep with rotary positions, against a mirror of every sequence in 64 bits."""
import math

import pytest
import torch

import kv4_reference as ref

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_gqa_03_gb300 as m
    return m


class Mirror:
    """Each sequence's cached keys and values as the cache holds them, and its step's expected output."""

    def __init__(self, D, table, held):
        self.D, self.table, self.held = D, table, held
        self.k, self.v = {}, {}

    def rotated(self, x, first):
        if self.table is None:
            return x.cpu().double()
        pos = torch.arange(first, first + x.shape[0])
        return ref.rotated(x, pos, self.table.frequencies, self.table.magnitude, self.table.interleaved)

    def append(self, seq, k, v, dtype):
        first = len(self.k[seq]) if seq in self.k else 0
        k = self.rotated(k, first).to(dtype)     # rounded to the rows' type, then held by the cache
        for d, x in ((self.k, self.held(k)), (self.v, self.held(v.cpu()))):
            d[seq] = torch.cat((d[seq], x)) if seq in d else x

    def check(self, seq, q, out, scale, window):
        n = q.shape[0]
        k, v = self.k[seq], self.v[seq]
        rq = self.rotated(q, len(k) - n).to(q.dtype)
        want = ref.attention(rq, k, v, scale, window)
        tol = ref.tolerance(want, rq, k, v, scale, out.dtype)
        # A rotated element may round the other way: a step of 2^-8 (bf16) of one element of q or of a key moves a score by
        # less than 2^-8 of one of its D terms; where a key's element stands on a border between two codes the term moves by a
        # third of itself.  A weight then is off by the few such elements' share of its score: 2^-7 of the largest value.
        turn = 0.0 if self.table is None else 0.5
        err = (out.cpu().double() - want).abs()
        assert (err <= tol + turn * float(v.abs().max()) * 2.0 ** -6).all(), (seq, float((err - tol).max()))


def held4(x):
    return ref.quantised(x)


def make(pkv, kind, q_len, window, rope, dtype, Hq=8, Hkv=2, D=128, blocks=96):
    from paged_kv_gqa_03_gb300.step import DecodeStep, Kv4Step
    table = pkv.RopeTable(D, base=10000.0, interleaved=q_len > 1) if rope else None
    stream = torch.cuda.Stream()
    if kind == "kv4":
        cache = torch.zeros(blocks, Hkv, 18 * D, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        return Kv4Step(cache, Hq, dtype, 24, stream=stream, q_len=q_len, window=window, rope=table), Mirror(D, table, held4)
    kc, vc = (torch.zeros(blocks, Hkv, 16, D, dtype=dtype, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    return (DecodeStep(kc, vc, Hq, dtype, 24, stream=stream, q_len=q_len, window=window, rope=table),
            Mirror(D, table, lambda x: x.to(dtype).double()))


@pytest.mark.parametrize("kind", ["kv4", "16"])
@pytest.mark.parametrize("q_len,window,rope,dtype", [(1, 0, False, BF16), (1, 0, True, BF16), (3, 0, True, F16), (2, 40, True, BF16)])
def test_steps(pkv, kind, q_len, window, rope, dtype):
    """Several steps from device tensors and from pinned host memory (a graph per staging buffer), a fork with
    copy-on-write in between."""
    step, mirror = make(pkv, kind, q_len, window, rope, dtype)
    g = torch.Generator().manual_seed(q_len + window)
    B, Hq, Hkv, D = 3, step.Hq, step.Hkv, step.D
    scale = 1.0 / math.sqrt(D)
    for seq in range(B):
        step.bm.allocate(seq, 0)
    step.seqs = list(range(B))
    shape = (B,) if q_len == 1 else (B, q_len)
    h_out = torch.zeros(*shape, Hq, D, dtype=dtype, pin_memory=True)
    for it in range(30):
        if it == 20:      # sequence 9 shares sequence 0's blocks and goes on by itself
            step.stream.synchronize()
            assert step.bm.fork(0, 9)
            mirror.k[9], mirror.v[9] = mirror.k[0].clone(), mirror.v[0].clone()
            step.seqs = [9, 1, 2]
        q, k, v = (torch.randn(*shape, h, D, generator=g).to(dtype) for h in (Hq, Hkv, Hkv))
        step.prepare()
        if it % 2:
            step.stage_inputs(q, k, v)
            step.run(h_out)
            step.stream.synchronize()
            out = h_out.clone()
        else:
            step.upload()
            dq, dk, dv = (x.cuda() for x in (q, k, v))
            out = torch.zeros_like(dq)
            torch.cuda.synchronize()
            step.launch(dq, dk, dv, out)
            step.stream.synchronize()
            assert torch.equal(dq.cpu(), q)
        for b, seq in enumerate(step.seqs):
            rows = lambda x: x[b].view(q_len, -1, D)  # noqa: E731
            mirror.append(seq, rows(k), rows(v), dtype)
            if it % 3 == 0 or it > 26:
                mirror.check(seq, rows(q), rows(out), scale, window)


@pytest.mark.parametrize("calibrated", [False, True])
def test_fp8_step_with_rope(pkv, calibrated):
    """FP8 caches: the step's bytes are those of a rotation and an append, call by call."""
    from paged_kv_gqa_03_gb300.step import DecodeStep
    B, Hq, Hkv, D = 2, 4, 2, 128
    g = torch.Generator().manual_seed(1)

    def caches():
        return [torch.zeros(8, Hkv, 16, D, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)] + \
            [torch.zeros(8, Hkv, device="cuda") for _ in range(2)]
    a, b = caches(), caches()
    table = pkv.RopeTable(64)
    step = DecodeStep(a[0], a[1], Hq, BF16, 4, a[2], a[3], stream=torch.cuda.Stream(), calibrated=calibrated, rope=table)
    for seq in range(B):
        step.bm.allocate(seq, 0)
    step.seqs = list(range(B))
    for it in range(5):
        q, k, v = (torch.randn(B, h, D, generator=g).to(BF16).cuda() for h in (Hq, Hkv, Hkv))
        out = torch.empty_like(q)
        step.prepare()
        step.upload()
        torch.cuda.synchronize()
        step.launch(q, k, v, out)
        step.stream.synchronize()
        pos = torch.full((B,), it, device="cuda")
        qr, kr = torch.empty_like(q), torch.empty_like(k)
        pkv.paged_rope(q, k, pos, table, q_out=qr, k_out=kr)
        pkv.paged_kv_append(kr, v, b[0], b[1], step.d_slots, b[2], b[3], calibrated=calibrated)
        want = torch.empty_like(q)
        pkv.paged_decode_attention(want, qr, b[0], b[1], step.d_table, step.d_lens, 1.0 / math.sqrt(D), b[2], b[3])
        assert torch.equal(out, want)
        assert all(torch.equal(x.view(torch.uint8) if x.dtype == E4M3 else x, y.view(torch.uint8) if y.dtype == E4M3 else y)
                   for x, y in zip(a, b))


def test_prompt_through_16_bits(pkv):
    """A prompt prefilled on 16-bit pages, packed, continued in 4 bits, its prefix expanded for the next chunk: the
    calls in the order of a server."""
    Hq, Hkv, D, n, m = 8, 2, 128, 200, 70
    g = torch.Generator().manual_seed(3)
    scale = 1.0 / math.sqrt(D)
    table = pkv.RopeTable(D, base=500000.0)
    rows = [torch.randn(n + m, h, D, generator=g).to(BF16) for h in (Hq, Hkv, Hkv)]
    dq, dk, dv = (x.cuda() for x in rows)
    blocks = (n + m + 15) // 16
    kc, vc = (torch.zeros(blocks, Hkv, 16, D, dtype=BF16, device="cuda") for _ in range(2))
    cache = torch.zeros(blocks, Hkv, 18 * D, dtype=torch.uint8, device="cuda")
    ids = torch.randperm(blocks, generator=g)
    slot = lambda a, b: (ids[torch.arange(a, b) // 16] * 16 + torch.arange(a, b) % 16).cuda()  # noqa: E731
    bt = ids.to(torch.int32).view(1, -1).cuda()
    pos = torch.arange(n + m, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q1 = torch.empty_like(dq[:n])
    pkv.paged_rope_append(dq[:n], dk[:n], dv[:n], pos[:n], table, kc, vc, slot(0, n), q_out=q1)
    out1 = torch.empty_like(q1)
    pkv.paged_prefill_attention(out1, q1, kc, vc, bt, i32(n), i32(0, n), n, scale)
    used = (n + 15) // 16
    pairs = torch.stack((ids[:used], ids[:used]), -1).to(torch.int32).contiguous().cuda()
    pkv.paged_kv4_pack_blocks(cache, kc, vc, pairs)
    # the next chunk: quantised like the rest, attended over the expanded pages
    q2 = torch.empty_like(dq[n:])
    pkv.paged_kv4_rope_append(dq[n:], dk[n:], dv[n:], pos[n:], table, cache, slot(n, n + m), q_out=q2)
    every = torch.stack((ids, ids), -1).to(torch.int32).contiguous().cuda()
    pkv.paged_kv4_expand_blocks(kc, vc, cache, every)
    out2 = torch.empty_like(q2)
    pkv.paged_prefill_attention(out2, q2, kc, vc, bt, i32(n + m), i32(0, m), m, scale)
    # and its last rows on the 4-bit pages
    few = 4
    out3 = torch.empty(1, few, Hq, D, dtype=BF16, device="cuda")
    pkv.paged_kv4_decode_attention(out3, q2[-few:].unsqueeze(0).contiguous(), cache, bt, i32(n + m), scale)
    k4, v4 = ref.quantised(ref.rotated(rows[1], pos, table.frequencies).to(BF16)), ref.quantised(rows[2])
    want = ref.attention(q2[-few:].cpu(), k4, v4, scale)
    tol = ref.tolerance(want, q2[-few:].cpu(), k4, v4, scale, BF16) + 2.0 ** -7 * float(v4.abs().max())
    assert ((out3[0].cpu().double() - want).abs() <= tol).all()
    # expanded values are exact in bf16 (E2M1 times E4M3: 6 bits), so prefill and decode see the same keys
    assert ((out2[-few:].cpu().double() - out3[0].cpu().double()).abs() <= 2 * tol).all()
