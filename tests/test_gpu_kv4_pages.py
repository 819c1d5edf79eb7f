"""The 4-bit cache's pages on the GPU: append, pack, expand and copy against the format's definition, bit for bit."""
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


def rows(shape, dtype, seed, reach=1.0):
    """Rows that hold what is hard about the format: empty groups, borders between two codes, groups beyond both
    ends of the scales, elements that are not finite."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * torch.exp(torch.randn(*shape[:-1], 1, generator=g)) * reach
    flat = x.view(-1, 16)
    n = flat.shape[0]
    flat[0::11] = 0.0
    flat[3::11, 5] = 1.75 * reach                                     # with 6 as the largest: borders
    borders = torch.tensor([6.0, 0.25, -0.25, 0.75, -0.75, 1.25, -1.25, 1.75, -1.75, 2.5, -2.5, 3.5, -3.5, 5.0, -5.0, 0.125])
    flat[1::13] = borders * 2.0 ** torch.randint(-3, 4, (flat[1::13].shape[0], 1), generator=g) * reach
    flat[5::17] *= 2.0 ** -10
    flat[6::17] *= 2.0 ** 12
    if n > 40:
        flat[17, 3], flat[23, 0], flat[31, 15] = math.inf, math.nan, -math.inf
    return x.to(dtype).cuda()


def same(got, want):
    got, want = got.detach().cpu().double(), want.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


def expanded(pkv, cache, D, dtype=F32, **units):
    n, Hkv = cache.shape[:2]
    k = torch.full((n, Hkv, 16, D), 7.0, dtype=dtype, device="cuda")
    v = torch.full_like(k, 7.0)
    pairs = torch.arange(n, dtype=torch.int32, device="cuda").repeat_interleave(2).view(-1, 2).contiguous()
    pkv.paged_kv4_expand_blocks(k, v, cache, pairs, **units)
    return k, v


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("units", [(1.0, 1.0), (0.03, 1.7)])
@pytest.mark.parametrize("T,Hkv", [(1, 1), (37, 3), (200, 8)])
def test_append(pkv, D, dtype, units, T, Hkv):
    nb = T // 3 + 3
    k, v = rows((T, Hkv, D), dtype, 1, units[0]), rows((T, Hkv, D), dtype, 2, units[1])
    g = torch.Generator().manual_seed(3)
    slots = torch.randperm(nb * 16, generator=g)[:T]
    if T > 4:
        slots[1], slots[2], slots[4] = -1, nb * 16, 1 << 40     # skipped
    cache = torch.randint(0, 0x77, (nb, Hkv, 18 * D), dtype=torch.uint8, device="cuda")
    before = [x.clone() for x in expanded(pkv, cache, D, k_unit=units[0], v_unit=units[1])]
    pkv.paged_kv4_append(k, v, cache, slots.cuda(), k_unit=units[0], v_unit=units[1])
    got = expanded(pkv, cache, D, k_unit=units[0], v_unit=units[1])
    keep = (slots >= 0) & (slots < nb * 16)
    for x, old, now, unit in ((k, before[0], got[0], units[0]), (v, before[1], got[1], units[1])):
        want = old.cpu().double()
        want[slots[keep] // 16, :, slots[keep] % 16] = ref.quantised(x, unit)[keep]
        same(now, want)


def test_append_rows_of_a_projection(pkv):
    """k and v as columns of one wider row, and one token whose stride plays no part."""
    T, Hq, Hkv, D = 19, 4, 2, 128
    qkv = rows((T, Hq + 2 * Hkv, D), BF16, 5)
    cache, dense = (torch.zeros(2, Hkv, 18 * D, dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = torch.arange(T, device="cuda")
    k, v = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    pkv.paged_kv4_append(k, v, cache, slots)
    pkv.paged_kv4_append(k.contiguous(), v.contiguous(), dense, slots)
    assert torch.equal(cache, dense)
    pkv.paged_kv4_append(k[3:4], v[3:4], cache, slots[3:4])
    assert torch.equal(cache, dense)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("n,Hkv", [(1, 1), (7, 3), (40, 8)])
def test_pack_and_expand(pkv, D, dtype, n, Hkv):
    unit = (0.5, 3.0)
    k, v = rows((n, Hkv, 16, D), dtype, 7, unit[0]), rows((n, Hkv, 16, D), dtype, 8, unit[1])
    g = torch.Generator().manual_seed(9)
    dst = torch.randperm(n + 2, generator=g)[:n]
    pairs = torch.stack((torch.arange(n), dst), -1).to(torch.int32)
    bad = torch.tensor([[-1, 0], [n, 1], [0, -3], [0, n + 2], [1 << 30, 0]], dtype=torch.int32)   # skipped
    both = torch.cat((pairs, bad)).cuda()
    cache = torch.zeros(n + 2, Hkv, 18 * D, dtype=torch.uint8, device="cuda")
    pkv.paged_kv4_pack_blocks(cache, k, v, both, k_unit=unit[0], v_unit=unit[1])
    want_k, want_v = ref.quantised(k, unit[0]), ref.quantised(v, unit[1])
    got_k, got_v = expanded(pkv, cache, D, k_unit=unit[0], v_unit=unit[1])
    same(got_k[dst], want_k)
    same(got_v[dst], want_v)
    rest = [i for i in range(n + 2) if i not in dst.tolist()]
    assert not cache[rest].any()
    # into the rows' type, one rounding, into other blocks; others stay
    back_k, back_v = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    few = pairs.flip(-1)[: (n + 1) // 2].contiguous().cuda()
    pkv.paged_kv4_expand_blocks(back_k, back_v, cache, torch.cat((few, bad.flip(-1).cuda())), k_unit=unit[0], v_unit=unit[1])
    at = few[:, 1].long().cpu()
    same(back_k[at], want_k[at].float().to(dtype))
    same(back_v[at], want_v[at].float().to(dtype))
    stay = [i for i in range(n) if i not in at.tolist()]
    assert (back_k[stay] == 7).all() and (back_v[stay] == 7).all()


def test_append_equals_pack(pkv):
    Hkv, D = 2, 64
    k, v = rows((3, Hkv, 16, D), F16, 10), rows((3, Hkv, 16, D), F16, 11)
    packed, appended = (torch.zeros(3, Hkv, 18 * D, dtype=torch.uint8, device="cuda") for _ in range(2))
    pkv.paged_kv4_pack_blocks(packed, k, v, torch.arange(3, dtype=torch.int32, device="cuda").repeat_interleave(2).view(3, 2).contiguous())
    tokens = [x.transpose(1, 2).reshape(48, Hkv, D).contiguous() for x in (k, v)]
    order = torch.randperm(48, generator=torch.Generator().manual_seed(1))
    pkv.paged_kv4_append(tokens[0][order].contiguous(), tokens[1][order].contiguous(), appended, order.cuda())
    assert torch.equal(packed, appended)


@pytest.mark.parametrize("D", [64, 128])
def test_copy_blocks(pkv, D):
    cache = torch.randint(0, 256, (9, 3, 18 * D), dtype=torch.uint8, device="cuda")
    want = cache.clone()
    pairs = torch.tensor([[0, 4], [1, 5], [8, 2], [7, 7], [-1, 3], [3, 9], [9, 3]], dtype=torch.int32, device="cuda")
    for s, d in ((0, 4), (1, 5), (8, 2)):
        want[d] = want[s]
    pkv.paged_kv4_copy_blocks(cache, pairs)
    assert torch.equal(cache, want)


def test_blocks_beyond_32_bit_offsets(pkv):
    Hkv, D = 8, 128
    n = (1 << 32) // (Hkv * 18 * D) + 40
    cache = torch.empty(n, Hkv, 18 * D, dtype=torch.uint8, device="cuda")
    k, v = rows((2, Hkv, 16, D), BF16, 12), rows((2, Hkv, 16, D), BF16, 13)
    pkv.paged_kv4_pack_blocks(cache, k, v, torch.tensor([[0, n - 1], [1, 5]], dtype=torch.int32, device="cuda"))
    pkv.paged_kv4_copy_blocks(cache, torch.tensor([[n - 1, n - 3]], dtype=torch.int32, device="cuda"))
    pkv.paged_kv4_append(k[1, :, :1].transpose(0, 1).contiguous(), v[1, :, :1].transpose(0, 1).contiguous(), cache,
                         torch.tensor([(n - 3) * 16 + 2], device="cuda"))
    got_k, got_v = torch.zeros_like(k), torch.zeros_like(v)
    pkv.paged_kv4_expand_blocks(got_k, got_v, cache, torch.tensor([[n - 3, 1], [5, 0]], dtype=torch.int32, device="cuda"))
    for got, x in ((got_k, k), (got_v, v)):
        want = ref.quantised(x)
        first = want[0].clone()
        first[:, 2] = want[1][:, 0]
        same(got[1], first)
        same(got[0], want[1])


def test_neighbours_appended_at_once(pkv):
    """Even tokens on one stream, their odd neighbours, whose values share bytes, on another."""
    n, Hkv, D = 4096, 4, 128
    k, v = rows((n, Hkv, D), BF16, 12), rows((n, Hkv, D), BF16, 13)
    slots = torch.arange(n, device="cuda")
    want = torch.zeros(n // 16, Hkv, 18 * D, dtype=torch.uint8, device="cuda")
    pkv.paged_kv4_append(k, v, want, slots)
    parts = [(k[i::2].contiguous(), v[i::2].contiguous(), slots[i::2].contiguous()) for i in range(2)]
    got, streams = torch.zeros_like(want), [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for (a, b, s), stream in zip(parts, streams):
            pkv.paged_kv4_append(a, b, got, s, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_nothing_to_do(pkv):
    cache = torch.full((1, 1, 18 * 64), 3, dtype=torch.uint8, device="cuda")
    e = torch.empty(0, 1, 64, dtype=F16, device="cuda")
    page = torch.ones(1, 1, 16, 64, dtype=F16, device="cuda")
    none = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    pkv.paged_kv4_append(e, e, cache, torch.empty(0, dtype=torch.int64, device="cuda"))
    pkv.paged_kv4_pack_blocks(cache, page, page, none)
    pkv.paged_kv4_expand_blocks(page, page, cache, none)
    pkv.paged_kv4_copy_blocks(cache, none)
    assert (cache == 3).all() and (page == 1).all()
