"""What the Python calls on the 4-bit cache and of the rotary positions refuse before anything runs, and prepared calls."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
I32, I64 = torch.int32, torch.int64


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_gqa_03_gb300 as m
    return m


def dev(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def test_append(pkv):
    cache, slots = dev(3, 2, 18 * 64, dtype=torch.uint8), dev(5, dtype=I64)
    k = dev(5, 2, 64)
    for a in ((dev(5, 3, 64), k), (k, dev(4, 2, 64)), (k, dev(5, 2, 128)), (k.cpu(), k), (k, k.cpu()),
              (dev(5, 64, 2).transpose(1, 2), k), (dev(5, 2, 128)[..., ::2], k), (dev(5, 4, 64)[:, ::2], k)):
        with pytest.raises(ValueError):
            pkv.paged_kv4_append(*a, cache, slots)
    with pytest.raises(TypeError):
        pkv.paged_kv4_append(k, k.to(F16), cache, slots)
    with pytest.raises(TypeError):
        pkv.paged_kv4_append(k, k, cache, slots.to(I32))
    with pytest.raises(TypeError):
        pkv.paged_kv4_append(k, k, cache.view(torch.int8), slots)
    for c in (cache[..., :1000], cache.view(3, 1, -1), cache.view(-1), cache.cpu(), dev(6, 2, 18 * 64, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            pkv.paged_kv4_append(k, k, c, slots)
    for rows in (k.expand(5, 2, 64)[:1].expand(5, 2, 64), dev(5 * 132 + 8)[:5 * 132].view(5, 132)[:, 2:130].view(5, 2, 64)):
        with pytest.raises(pkv.PagedKVError):      # the same row for all; rows off a 16-byte border
            pkv.paged_kv4_append(rows, k, cache, slots)
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_kv4_append(k, k, cache, slots, k_unit=0.0)
    with pytest.raises(TypeError):
        pkv.paged_kv4_append(k.to(torch.int16), k.to(torch.int16), cache, slots)
    torch.cuda.synchronize()
    assert not cache.any()


def test_pages(pkv):
    cache, k, pairs = dev(3, 2, 18 * 64, dtype=torch.uint8), dev(4, 2, 16, 64), dev(2, 2, dtype=I32)
    for call in (lambda *a: pkv.paged_kv4_pack_blocks(a[2], a[0], a[1], a[3]), pkv.paged_kv4_expand_blocks):
        for a in ((dev(4, 2, 16, 128), k, cache, pairs), (k, k[:3], cache, pairs), (k, k.cpu(), cache, pairs),
                  (k, k, cache, dev(4, dtype=I32)[None].expand(2, 4)), (k.transpose(1, 2).contiguous(), k, cache, pairs)):
            with pytest.raises(ValueError):
                call(*a)
        with pytest.raises(TypeError):
            call(k, k.to(F16), cache, pairs)
        with pytest.raises(TypeError):
            call(k, k, cache, pairs.long())
        with pytest.raises(pkv.PagedKVError):      # fp8 pages have scales of their own
            call(k.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn), cache, pairs)
    with pytest.raises(TypeError):
        pkv.paged_kv4_copy_blocks(cache, pairs.long())


def test_attention(pkv):
    q, cache = dev(2, 4, 64), dev(3, 2, 18 * 64, dtype=torch.uint8)
    table, lens = dev(2, 3, dtype=I32), dev(2, dtype=I32)
    out = torch.empty_like(q)

    def call(out=out, q=q, cache=cache, table=table, lens=lens, **kw):
        return pkv.paged_kv4_decode_attention(out, q, cache, table, lens, 0.1, **kw)
    for kw in (dict(q=q[0], out=out[0]), dict(out=out[:1]), dict(out=out.to(F16)), dict(cache=dev(3, 2, 18 * 128, dtype=torch.uint8)),
               dict(table=table[:1]), dict(table=table[0]), dict(lens=lens[:1]), dict(q=dev(2, 64, 4).transpose(1, 2)),
               dict(out=torch.zeros(2, 4, 64, dtype=BF16)), dict(q=q.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(table=table.long()), dict(lens=lens.long())):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(q=q.float(), out=out.float()), dict(window=-1), dict(k_unit=-1.0), dict(workspace=dev(64, dtype=torch.uint8)),
               dict(q=dev(2, 3, 64), out=dev(2, 3, 64)), dict(num_splits=-1)):
        with pytest.raises(pkv.PagedKVError):
            call(**kw)


def test_rope(pkv):
    T, Hq, Hkv, D = 3, 4, 2, 64
    q, k, pos, slots, table = dev(T, Hq, D), dev(T, Hkv, D), dev(T, dtype=I64), dev(T, dtype=I64), pkv.RopeTable(D)
    kc, cache = dev(2, Hkv, 16, D), dev(2, Hkv, 18 * D, dtype=torch.uint8)
    for a in ((None, None), (q, dev(2, Hkv, D)), (q, dev(T, Hkv, 128)), (q.cpu(), k)):
        with pytest.raises(ValueError):
            pkv.paged_rope(*a, pos, table)
    with pytest.raises(ValueError):
        pkv.paged_rope(q, None, pos, table, k_out=k)
    with pytest.raises(ValueError):
        pkv.paged_rope(q, k, pos[:2], table)
    with pytest.raises(ValueError):
        pkv.paged_rope(q, k, pos, pkv.RopeTable(D, device="cpu"))
    with pytest.raises(TypeError):
        pkv.paged_rope(q, k.float(), pos, table)
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_rope(q, k, pos, pkv.RopeTable(128))          # more than the head
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_rope(q, k, pos, pkv.RopeTable(24))
    for append, caches in ((pkv.paged_rope_append, (kc, kc.clone())), (pkv.paged_kv4_rope_append, (cache,))):
        for a in ((q, k, k[:2], pos, table), (q, dev(T, 1, D), k, pos, table), (q, k, k, pos.cpu(), table)):
            with pytest.raises(ValueError):
                append(*a, *caches, slots)
        with pytest.raises(ValueError):
            append(q, k, k, pos, table, *caches, slots[:1])
        with pytest.raises(pkv.PagedKVError):      # the queries' rows in place of the keys'
            append(q, q[:, :Hkv], k, pos, table, *caches, slots)
    with pytest.raises(TypeError):
        pkv.paged_rope_append(q, k, k, pos, table, kc.to(F16), kc.to(F16), slots)


def test_prepared_calls(pkv):
    """The same calls marshalled once, issued twice, against the plain calls."""
    T, Hq, Hkv, D = 20, 4, 2, 64
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(T, h, D, generator=g).to(BF16).cuda() for h in (Hq, Hkv, Hkv))
    pos, slots, table = torch.arange(T, device="cuda"), torch.arange(T, device="cuda"), pkv.RopeTable(D)
    got = []
    for prepare in (False, True):
        q_out, k_out, cache = torch.zeros_like(q), torch.zeros_like(k), dev(4, Hkv, 18 * D, dtype=torch.uint8)
        kc, vc, k16, v16 = (dev(4, Hkv, 16, D) for _ in range(4))
        pairs = torch.tensor([[0, 2], [1, 3]], dtype=I32, device="cuda")
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        kw = dict(prepare=True, stream=stream) if prepare else dict(stream=stream)
        done = [lambda **kw: pkv.paged_rope(q, k, pos, table, q_out=q_out, k_out=k_out, **kw),
                lambda **kw: pkv.paged_rope_append(q, k, v, pos, table, kc, vc, slots, q_out=q_out, **kw),
                lambda **kw: pkv.paged_kv4_append(k, v, cache, slots, **kw),
                lambda **kw: pkv.paged_kv4_rope_append(q, k, v, pos, table, cache, slots, q_out=q_out, **kw),
                lambda **kw: pkv.paged_kv4_pack_blocks(cache, kc, vc, pairs, **kw),
                lambda **kw: pkv.paged_kv4_copy_blocks(cache, pairs[:1], **kw),
                lambda **kw: pkv.paged_kv4_expand_blocks(k16, v16, cache, pairs, **kw)]
        for call in done:
            r = call(**kw)
            if prepare:
                r()
                r()
        torch.cuda.synchronize()
        got.append([x.clone() for x in (q_out, k_out, cache, kc, vc, k16, v16)])
    assert all(torch.equal(a, b) for a, b in zip(*got)) and got[0][5].any()
