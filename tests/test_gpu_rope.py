"""Rotary positions on the GPU against the rotation in 64 bits, and the fused appends against the two calls."""
import math

import pytest
import torch

import kv4_reference as ref

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_gqa_03_gb300 as m
    return m


def close(got, want, x, magnitude):
    """An angle is off by less than 2^-21 radians (the float of its turn 2^-25 half turns, the sine and cosine 2 units in
    the last place), three fp32 roundings, one rounding to the type: of the pair's largest element twice."""
    reach = x.detach().cpu().double().abs().amax(-1, keepdim=True) * abs(magnitude)
    tol = 2 * reach * (2.0 ** -21 + 3 * 2.0 ** -24) + torch.finfo(got.dtype).eps / 2 * want.abs() + torch.finfo(got.dtype).tiny
    err = (got.detach().cpu().double() - want).abs()
    assert (err <= tol).all(), float((err - tol).max())


FAR = [0, 1, 2, 77, 8191, 131071, 999_999, (1 << 31) + 5, (1 << 40) + 3, -1, -4097]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (128, 16), (128, 48), (64, 64), (64, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation(pkv, dtype, D, rot, interleaved):
    T, Hq, Hkv = len(FAR), 7, 2
    g = torch.Generator().manual_seed(D + rot)
    q, k = (torch.randn(T, h, D, generator=g).to(dtype).cuda() for h in (Hq, Hkv))
    # frequencies with few bits: position * f is exact in 64 bits, however far the position
    f = torch.tensor([round(2.0 ** 20 * 10000.0 ** (-2 * i / rot)) / 2.0 ** 20 for i in range(rot // 2)], dtype=torch.float64)
    pos = torch.tensor(FAR)
    table = pkv.RopeTable(rot, frequencies=f.numpy(), magnitude=1.25, interleaved=interleaved)
    near = pos.abs() < 1 << 32       # (a frequency's own 2^-53 is 2^-13 radians at 2^40)
    q0, k0 = q.clone(), k.clone()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pkv.paged_rope(q, k, pos.cuda(), table, q_out=qo, k_out=ko)
    assert torch.equal(q, q0) and torch.equal(k, k0)
    for got, x in ((qo, q), (ko, k)):
        want = ref.rotated(x, pos, f, 1.25, interleaved)
        close(got[near.cuda()], want[near], x[near.cuda()], 1.25)
        assert torch.isfinite(got.float()).all()
    pkv.paged_rope(q, k, pos.cuda(), table)     # in place
    assert torch.equal(q, qo) and torch.equal(k, ko)
    pkv.paged_rope(q0, None, pos.cuda(), table)
    pkv.paged_rope(None, k0, pos.cuda(), table)
    assert torch.equal(q0, qo) and torch.equal(k0, ko)


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "parts"])
def test_scalings(pkv, scaling):
    T, D = 33, 128
    g = torch.Generator().manual_seed(1)
    q = torch.randn(T, 3, D, generator=g).to(F32).cuda()
    pos = torch.randint(0, 1_000_000, (T,), generator=g)
    table = pkv.RopeTable(D, base=500000.0, scaling=scaling, factor=8.0, original_positions=8192, slow=1.0, fast=4.0)
    i = torch.arange(0, D, 2, dtype=torch.float64)
    f = 500000.0 ** (-i / D)
    if scaling == "linear":
        f = f / 8
    elif scaling == "base":
        f = (500000.0 * 8 ** (D / (D - 2))) ** (-i / D)
    elif scaling == "parts":
        r = 8192 * f / (2 * math.pi)
        f = torch.where(r >= 4, f, torch.where(r <= 1, f / 8, f * (r - 1) / 3 + f / 8 * (4 - r) / 3))
    assert torch.allclose(torch.as_tensor(table.frequencies), f, rtol=1e-13, atol=0)
    out = torch.empty_like(q)
    pkv.paged_rope(q, None, pos.cuda(), table, q_out=out)
    close(out, ref.rotated(q, pos, table.frequencies), q, 1.0)


def projection(T, Hq, Hkv, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(dtype).cuda()
    return qkv, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,interleaved", [(1, 1, 1, 64, 16, True), (5, 64, 8, 128, 128, False),
                                                        (300, 9, 3, 128, 48, False), (700, 32, 32, 64, 64, True),
                                                        (260, 200, 8, 128, 64, True), (2, 300, 20, 128, 128, False)])
def test_appends_equal_the_two_calls(pkv, dtype, T, Hq, Hkv, D, rot, interleaved):
    """Rows of one projection; skipped tokens' queries are rotated, their keys go nowhere; the rest of the caches stays."""
    qkv, q, k, v = projection(T, Hq, Hkv, D, dtype, T)
    nb = (T + 15) // 16 + 2
    g = torch.Generator().manual_seed(2)
    slots = torch.randperm(nb * 16, generator=g)[:T]
    if T > 3:
        slots[1], slots[3] = -1, nb * 16 + 4
    slots, pos = slots.cuda(), torch.randint(0, 200_000, (T,), generator=g).cuda()
    table = pkv.RopeTable(rot, base=500000.0, magnitude=1.1, interleaved=interleaved)
    qo, ko = torch.empty(T, Hq, D, dtype=dtype, device="cuda"), torch.empty(T, Hkv, D, dtype=dtype, device="cuda")
    pkv.paged_rope(q, k, pos, table, q_out=qo, k_out=ko)
    caches = [torch.full((nb, Hkv, 16, D), 3.0, dtype=dtype, device="cuda") for _ in range(4)]
    pkv.paged_kv_append(ko, v.contiguous(), caches[0], caches[1], slots)
    before = qkv.clone()
    out = torch.empty_like(qo)
    pkv.paged_rope_append(q, k, v, pos, table, caches[2], caches[3], slots, q_out=out)
    assert torch.equal(out, qo) and torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    four = [torch.full((nb, Hkv, 18 * D), 5, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pkv.paged_kv4_append(ko, v, four[0], slots, k_unit=0.7, v_unit=1.3)
    out.zero_()
    pkv.paged_kv4_rope_append(q, k, v, pos, table, four[1], slots, k_unit=0.7, v_unit=1.3, q_out=out)
    assert torch.equal(out, qo) and torch.equal(four[0], four[1])
    assert torch.equal(qkv, before)
    pkv.paged_rope_append(q, k, v, pos, table, caches[2], caches[3], slots)     # q in place, in the projection
    assert torch.equal(q, qo) and torch.equal(k, before[:, Hq:Hq + Hkv]) and torch.equal(caches[0], caches[2])


def test_stream_and_graph(pkv):
    T, Hq, Hkv, D = 40, 16, 2, 128
    _, q, k, v = projection(T, Hq, Hkv, D, BF16, 3)
    pos, slots = torch.arange(100, 100 + T, device="cuda"), torch.arange(T, device="cuda")
    table = pkv.RopeTable(D)
    kc, vc = (torch.zeros(3, Hkv, 16, D, dtype=BF16, device="cuda") for _ in range(2))
    want = torch.empty(T, Hq, D, dtype=BF16, device="cuda")
    pkv.paged_rope_append(q, k, v, pos, table, kc, vc, slots, q_out=want)
    torch.cuda.synchronize()
    for other in (False, True):
        out, kc2, vc2 = torch.zeros_like(want), torch.zeros_like(kc), torch.zeros_like(vc)
        torch.cuda.synchronize()
        if other:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                pkv.paged_rope_append(q, k, v, pos, table, kc2, vc2, slots, q_out=out)
            out.zero_()
            graph.replay()
        else:
            pkv.paged_rope_append(q, k, v, pos, table, kc2, vc2, slots, q_out=out, stream=torch.cuda.Stream())
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_columns_of_one_buffer(pkv):
    """Outputs side by side in one buffer, and both turned in place in the projection that holds them."""
    T, Hq, Hkv, D = 70, 6, 2, 64
    qkv, q, k, v = projection(T, Hq, Hkv, D, F16, 4)
    pos, table = torch.arange(T, device="cuda") * 1000, pkv.RopeTable(D, interleaved=True)
    apart = [torch.empty(T, h, D, dtype=F16, device="cuda") for h in (Hq, Hkv)]
    pkv.paged_rope(q, k, pos, table, q_out=apart[0], k_out=apart[1])
    both = torch.zeros(T, Hq + Hkv, D, dtype=F16, device="cuda")
    pkv.paged_rope(q, k, pos, table, q_out=both[:, Hkv:], k_out=both[:, :Hkv])
    assert torch.equal(both[:, Hkv:], apart[0]) and torch.equal(both[:, :Hkv], apart[1])
    values = v.clone()
    pkv.paged_rope(q, k, pos, table)
    assert torch.equal(q, apart[0]) and torch.equal(k, apart[1]) and torch.equal(v, values)
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_rope(q, qkv[:, 1:1 + Hkv], pos, table)


def test_no_tokens(pkv):
    e = torch.empty(0, 2, 64, dtype=F16, device="cuda")
    i = torch.empty(0, dtype=torch.int64, device="cuda")
    c = torch.zeros(1, 2, 16, 64, dtype=F16, device="cuda")
    pkv.paged_rope(e, e, i, pkv.RopeTable(64))
    pkv.paged_rope_append(e, e, e, i, pkv.RopeTable(64), c, c.clone(), i)
    assert not c.any()
