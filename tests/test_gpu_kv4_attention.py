"""paged_kv4_decode_attention against the definition in 64 bits on the cache's own values."""
import math

import pytest
import torch

import kv4_reference as ref

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_gqa_03_gb300 as m
    return m


class Case:
    def __init__(self, pkv, lens, q_len, Hq, Hkv, D, dtype, seed=0, extra=3, unit=(1.0, 1.0), keys=1.0):
        g = torch.Generator().manual_seed(seed)
        self.pkv, self.lens, self.n, self.D, self.Hkv, self.unit = pkv, lens, q_len, D, Hkv, unit
        need = [(max(c, 0) + 15) // 16 for c in lens]
        total = sum(need)
        ids = torch.randperm(total + extra, generator=g)[:total].to(torch.int32)
        self.table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = ids[at:at + m]
            at += m
        chan = torch.exp(0.5 * torch.randn(Hkv, 1, D, generator=g))
        shape = (total + extra, Hkv, 16, D)
        self.k = (torch.randn(*shape, generator=g) * chan * keys * unit[0]).to(BF16)
        self.v = (torch.randn(*shape, generator=g) * unit[1]).to(BF16)
        shape = (len(lens), q_len, Hq, D)
        self.q = torch.randn(*shape, generator=g).to(dtype)
        self.scale = 1.0 / math.sqrt(D)

    def call(self, q=None, **kw):
        pkv, dev = self.pkv, "cuda"
        n = self.k.shape[0]
        cache = torch.zeros(n, self.Hkv, 18 * self.D, dtype=torch.uint8, device=dev)
        pairs = torch.arange(n, dtype=torch.int32, device=dev).repeat_interleave(2).view(-1, 2).contiguous()
        u = dict(k_unit=self.unit[0], v_unit=self.unit[1])
        pkv.paged_kv4_pack_blocks(cache, self.k.to(dev), self.v.to(dev), pairs, **u)
        q = (self.q if q is None else q).to(dev)
        if not kw.pop("four", False) and q.shape[1] == 1:
            q = q[:, 0]
        out = torch.full_like(q, 9.0)
        ws = pkv.paged_kv4_decode_attention(out, q.contiguous(), cache, self.table.to(dev),
                                            torch.tensor(self.lens, dtype=torch.int32, device=dev),
                                            kw.pop("scale", self.scale), **u, **kw)
        self.status = pkv.paged_decode_status(ws)
        return out.view(len(self.lens), self.n, *q.shape[-2:]).cpu()

    def check(self, window=0, q=None, k=None, v=None, **kw):
        out = self.call(window=window, q=q, **kw)
        q = self.q if q is None else q
        scale = kw.get("scale", self.scale)
        kq = ref.quantised(self.k, self.unit[0]) if k is None else k
        vq = ref.quantised(self.v, self.unit[1]) if v is None else v
        for b, ctx in enumerate(self.lens):
            ids = self.table[b, :(ctx + 15) // 16].long()
            kb, vb = (x[ids].transpose(1, 2).reshape(-1, self.Hkv, self.D)[:ctx] for x in (kq, vq))
            want = ref.attention(q[b], kb, vb, scale, window)
            got = out[b].double()
            assert torch.equal(torch.isnan(got), torch.isnan(want)), (b, ctx)
            tol = ref.tolerance(torch.nan_to_num(want), q[b], kb, vb, scale, out.dtype)
            err = (torch.nan_to_num(got) - torch.nan_to_num(want)).abs()
            assert (err <= tol).all(), (b, ctx, float((err - tol).max()), float(err.max()))
        return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (8, 1), (6, 2), (14, 2), (32, 2), (21, 1), (12, 4),
                                    (9, 3), (24, 12)])
def test_single_token(pkv, D, dtype, Hq, Hkv):
    c = Case(pkv, [1, 15, 16, 17, 0, 63, 64, 65, 300, 1111], 1, Hq, Hkv, D, dtype, seed=Hq + D)
    c.check()
    assert c.status == (0, 0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_len,Hq,Hkv", [(2, 4, 2), (3, 8, 1), (4, 32, 8), (8, 8, 8), (7, 14, 2), (64, 4, 1), (1, 4, 4)])
@pytest.mark.parametrize("window", [0, 1, 16, 17, 100])
def test_new_tokens_and_windows(pkv, D, q_len, Hq, Hkv, window):
    """Contexts shorter than the new tokens too: their first rows see nothing and give 0."""
    lens = [0, 1, q_len, q_len + 1, 16, 129, 333, 700]
    c = Case(pkv, lens, q_len, Hq, Hkv, D, BF16, seed=q_len + window)
    out = c.check(window=window, four=True)
    assert (out[0] == 0).all()
    if q_len > 1:
        assert (out[1, :q_len - 1] == 0).all()


@pytest.mark.parametrize("splits", [1, 2, 5, 64, 1000])
def test_split_counts(pkv, splits):
    c = Case(pkv, [5, 1000, 0, 77, 2049], 2, 16, 2, 128, F16, seed=3)
    c.check(num_splits=splits)


@pytest.mark.parametrize("Hq,Hkv,q_len,D", [(8, 1, 1, 128), (16, 4, 1, 128), (4, 2, 2, 64), (32, 8, 3, 128), (8, 8, 1, 64)])
def test_long_contexts(pkv, Hq, Hkv, q_len, D):
    """Units cut between many CTAs, of one, two and four heads."""
    c = Case(pkv, [12000, 3, 4001], q_len, Hq, Hkv, D, BF16, seed=4, keys=2.0)
    c.check()


def test_one_long_context(pkv):
    c = Case(pkv, [40000], 1, 8, 1, 128, BF16, seed=4, keys=2.0)
    c.check()


@pytest.mark.parametrize("B", [33, 100, 128, 129, 300, 510, 511, 512, 2500])
def test_many_sequences(pkv, B):
    """Planned in registers, in shared memory and (511 and more) by a kernel of its own; many are empty."""
    g = torch.Generator().manual_seed(5)
    lens = (torch.randint(0, 90, (B,), generator=g) - 20).clamp(min=0).tolist()
    c = Case(pkv, lens, 1, 4, 2, 64, F16, seed=5)
    c.check()
    assert c.status == (0, 0)


@pytest.mark.parametrize("lens", [[768] * 9, [769] * 9, [16] * 700, [190, 200] * 40])
def test_units_whole_or_cut(pkv, lens):
    """Tables at the border up to which units are not cut between CTAs, and more units than CTAs."""
    c = Case(pkv, lens, 1, 8, 4, 128, BF16, seed=15)
    c.check()


@pytest.mark.parametrize("D,whole", [(64, 96), (128, 48)])
@pytest.mark.parametrize("q_len", [1, 3])
@pytest.mark.parametrize("over", [0, 1])
def test_windows_whole_or_cut(pkv, D, whole, q_len, over):
    """Windows that reach into `whole` blocks at most, and one position more, at every offset within a block."""
    lens = [4096 + i for i in range(17)] + [whole * 16, 20, 0]
    c = Case(pkv, lens, q_len, 4, 4, D, BF16, seed=16)
    c.check(window=16 * whole - 15 - q_len + over)


@pytest.mark.parametrize("lens", [[1536] * 9, [1537] * 9, [700, 1500] * 10])
def test_units_whole_or_cut_64(pkv, lens):
    c = Case(pkv, lens, 1, 8, 4, 64, F16, seed=17)
    c.check()


@pytest.mark.parametrize("unit", [(1e-6, 3e-5), (1e6, 2e3), (0.37, 5.0), (2.0 ** -64, 2.0 ** 64), (2.0 ** 64, 2.0 ** -64)])
def test_units(pkv, unit):
    """Keys and values far from 1, held by their units."""
    c = Case(pkv, [100, 31, 500], 2, 8, 2, 128, BF16, seed=6, unit=unit)
    c.scale = 1.0 / math.sqrt(128) / unit[0]
    c.check()


@pytest.mark.parametrize("reach", [2.0 ** 70, 2.0 ** 20, 2.0 ** -20, 2.0 ** -100])
def test_queries_beyond_f16(pkv, reach):
    c = Case(pkv, [100, 31], 1, 8, 2, 128, BF16, seed=7)
    q = (c.q.float() * reach).to(BF16)
    c.check(q=q, scale=c.scale / reach)


@pytest.mark.parametrize("scale", [0.0, -0.07, 3.0])
def test_any_scale(pkv, scale):
    c = Case(pkv, [100, 31, 260], 2, 8, 2, 64, F16, seed=8)
    c.check(scale=scale)


def poke(case, which, b, pos, h, d, value):
    x = getattr(case, which)
    x[int(case.table[b, pos // 16]), h, pos % 16, d] = value


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_len,Hq", [(1, 2), (5, 2), (5, 12)])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_not_finite(pkv, D, q_len, Hq, value):
    """A group that holds what is not finite reads as NaN where a row sees it, and nowhere else: beyond the context,
    newer tokens, before the window."""
    lens, window = [70, 130, 40, 200, 333], 60
    for w in (0, window):
        c = Case(pkv, lens, q_len, Hq, 2, D, BF16, seed=9)
        for b, ctx in enumerate(lens):
            for pos in range(ctx, (ctx + 15) // 16 * 16):       # stale
                poke(c, "k", b, pos, 0, 3, value)
                poke(c, "v", b, pos, 1, 20, value)
        poke(c, "v", 0, 69, 0, 17, value)                       # the newest token
        poke(c, "k", 1, 129, 1, 40, value)
        poke(c, "v", 2, 3, 1, 63, value)                        # (windowless) every row sees it
        poke(c, "v", 3, 200 - window - q_len // 2, 0, 5, value)  # at the windows' edge: some rows
        poke(c, "k", 3, 200 - window - q_len // 2, 1, 5, value)
        poke(c, "k", 4, 10, 0, 1, value)                        # far before the window
        poke(c, "v", 4, 12, 1, 1, value)
        c.check(window=w, four=True)


def test_queries_not_finite(pkv):
    c = Case(pkv, [70, 2000], 1, 8, 2, 128, BF16, seed=10)
    clean = c.check()
    q = c.q.clone()
    q[1, 0, 5, 9] = math.nan
    out = c.call(q=q)
    assert torch.isnan(out[1, 0, 5]).all()
    keep = torch.ones(2, 1, 8, dtype=torch.bool)
    keep[1, 0, 5] = False
    assert torch.equal(out[keep], clean[keep])


def test_bad_blocks_and_lengths(pkv):
    """An id outside the cache reads as zeros and is flagged; lengths are clamped and flagged."""
    c = Case(pkv, [64, 100, 40], 1, 4, 2, 128, BF16, seed=11)
    c.call()
    assert c.status == (0, 0)
    kq, vq = ref.quantised(c.k), ref.quantised(c.v)
    good = c.table.clone()
    n = c.k.shape[0]
    for bad in (-1, n, 1 << 30):
        c.table[1, 2] = bad
        out = c.call()
        assert c.status[1] == pkv.PKV_FLAG_BAD_BLOCK
        ids = good[1].long()
        kb, vb = (x[ids].transpose(1, 2).reshape(-1, 2, 128)[:100].clone() for x in (kq, vq))
        kb[32:48], vb[32:48] = 0, 0
        want = ref.attention(c.q[1], kb, vb, c.scale)
        assert ((out[1].double() - want).abs() <= ref.tolerance(want, c.q[1], kb, vb, c.scale, BF16)).all()
    c.table = good
    full = c.table.shape[1] * 16
    c.lens = [64, full + 5, -7]
    out = c.call()
    assert c.status[1] == pkv.PKV_FLAG_BAD_LEN
    assert (out[2] == 0).all()


def test_blocks_beyond_32_bit_offsets(pkv):
    Hkv, D = 8, 128
    n = (1 << 32) // (Hkv * 18 * D) + 64
    cache = torch.empty(n, Hkv, 18 * D, dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(12)
    k, v = (torch.randn(8, Hkv, 16, D, generator=g).to(BF16) for _ in range(2))
    dst = torch.arange(n - 8, n, dtype=torch.int32)
    pkv.paged_kv4_pack_blocks(cache, k.cuda(), v.cuda(), torch.stack((torch.arange(8, dtype=torch.int32), dst), -1).contiguous().cuda())
    q = torch.randn(1, 16, D, generator=g).to(BF16)
    out = torch.empty_like(q, device="cuda")
    pkv.paged_kv4_decode_attention(out, q.cuda(), cache, dst.view(1, 8).cuda(),
                                   torch.tensor([125], dtype=torch.int32, device="cuda"), 0.09)
    kb, vb = (ref.quantised(x).transpose(1, 2).reshape(-1, Hkv, D)[:125] for x in (k, v))
    want = ref.attention(q, kb, vb, 0.09)
    assert ((out.cpu().double() - want).abs() <= ref.tolerance(want, q, kb, vb, 0.09, BF16)).all()


def test_same_bits_streams_and_graphs(pkv):
    """The same call gives the same bits: on another stream, two at once with workspaces of their own, replayed
    from a graph, into pinned host memory."""
    c = Case(pkv, [3000, 17, 900], 2, 16, 2, 128, BF16, seed=13)
    want = c.call()
    n = c.k.shape[0]
    cache = torch.zeros(n, 2, 18 * 128, dtype=torch.uint8, device="cuda")
    pairs = torch.arange(n, dtype=torch.int32, device="cuda").repeat_interleave(2).view(-1, 2).contiguous()
    pkv.paged_kv4_pack_blocks(cache, c.k.cuda(), c.v.cuda(), pairs)
    q, table, lens = c.q.cuda(), c.table.cuda(), torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    outs, streams = [torch.zeros_like(q) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for o, s in zip(outs, streams):
            pkv.paged_kv4_decode_attention(o, q, cache, table, lens, c.scale, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o.cpu(), want) for o in outs)
    host = torch.zeros(*q.shape, dtype=BF16, pin_memory=True)
    graph, out = torch.cuda.CUDAGraph(), torch.zeros_like(q)
    ws = torch.empty(pkv.paged_kv4_decode_workspace_bytes(3, 16, 2, 128, BF16, q_len=2), dtype=torch.uint8, device="cuda")
    with torch.cuda.graph(graph):
        pkv.paged_kv4_decode_attention(out, q, cache, table, lens, c.scale, workspace=ws)
        pkv.paged_kv4_decode_attention(host, q, cache, table, lens, c.scale, workspace=ws)
    for _ in range(3):
        out.zero_()
        host.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want) and torch.equal(host, want)
    call = pkv.paged_kv4_decode_attention(out.zero_(), q, cache, table, lens, c.scale, prepare=True)
    call()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want)


def test_timeout_is_reported(pkv):
    c = Case(pkv, [300, 40], 1, 8, 2, 128, BF16, seed=14)
    want = c.call()
    pkv.pkv_test_stall_next("decode", 2_000_000)
    c.call()
    assert c.status == (pkv.PKV_ETIMEOUT, pkv.PKV_FLAG_TIMEOUT)
    assert torch.equal(c.call(), want) and c.status == (0, 0)
