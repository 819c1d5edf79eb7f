"""paged_kv4_rope_append leaves the bytes that paged_rope and then paged_kv4_append leave, whatever the units: also of
zeros of either sign, of elements far below their group's scale, and of groups that the format holds as zeros."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_gqa_03_gb300 as m
    return m


def rows(T, heads, D, dtype, g):
    """Ordinary groups, groups below 6 * 2^-10 (a scale of 0), and groups with zeros and tiny elements of both signs."""
    x = torch.randn(T, heads, D // 16, 16, generator=g)
    kind = torch.randint(0, 4, (T, heads, D // 16, 1), generator=g)
    sign = 1 - 2.0 * torch.randint(0, 2, x.shape, generator=g)
    tiny = x * 2.0 ** -12
    some = torch.where(torch.rand(x.shape, generator=g) < 0.4, sign * 0.0, x)
    spread = x * 2.0 ** -torch.randint(0, 24, x.shape, generator=g)
    x = torch.where(kind == 0, x, torch.where(kind == 1, tiny, torch.where(kind == 2, some, spread)))
    return x.flatten(-2).to(dtype)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 48), (64, 64)])
@pytest.mark.parametrize("units", [(1.0, 1.0), (0.7, 1.3), (1.0, 2.0 ** -4), (2.0 ** 5, 1.0)])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_same_bytes(pkv, dtype, D, rot, units, T):
    Hq, Hkv = 4, 2
    g = torch.Generator().manual_seed(T + rot)
    q, k, v = (rows(T, h, D, dtype, g).cuda() for h in (Hq, Hkv, Hkv))
    nb = (T + 15) // 16 + 1
    slots = torch.randperm(nb * 16, generator=g)[:T].cuda() if T < 300 else torch.arange(T, device="cuda")
    pos = torch.randint(0, 100_000, (T,), generator=g).cuda()
    pos[::2] = 0        # (these turn by nothing: signs of zero stay)
    table = pkv.RopeTable(rot, base=500000.0)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pkv.paged_rope(q, k, pos, table, q_out=qo, k_out=ko)
    u = dict(k_unit=units[0], v_unit=units[1])
    two, one = (torch.full((nb, Hkv, 18 * D), 0xa5, dtype=torch.uint8, device="cuda") for _ in range(2))
    pkv.paged_kv4_append(ko, v, two, slots, **u)
    out = torch.empty_like(q)
    pkv.paged_kv4_rope_append(q, k, v, pos, table, one, slots, q_out=out, **u)
    assert torch.equal(out, qo)
    assert torch.equal(one, two)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
def test_pages_and_rows_alike(pkv, dtype, D):
    """Packed pages hold the bytes of rows appended one by one."""
    Hkv, nb = 2, 5
    g = torch.Generator().manual_seed(D)
    k, v = (rows(nb * 16, Hkv, D, dtype, g) for _ in range(2))
    a, b = (torch.zeros(nb, Hkv, 18 * D, dtype=torch.uint8, device="cuda") for _ in range(2))
    pkv.paged_kv4_append(k.cuda(), v.cuda(), a, torch.arange(nb * 16, device="cuda"))
    pages = [x.view(nb, 16, Hkv, D).transpose(1, 2).contiguous().cuda() for x in (k, v)]
    pairs = torch.arange(nb, dtype=torch.int32, device="cuda").repeat_interleave(2).view(-1, 2).contiguous()
    pkv.paged_kv4_pack_blocks(b, *pages, pairs)
    assert torch.equal(a, b)
