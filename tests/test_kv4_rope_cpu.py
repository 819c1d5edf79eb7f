"""Refusals of the 4-bit cache's and the rotary calls, and the rotary frequencies; no GPU."""
import ctypes
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_gqa_03_gb300 as m
    return m


P = 1 << 20     # an aligned address that no refused call reads


def append(L, **kw):
    a = dict(k=P, ldk=256, v=P, ldv=256, dt=2, c=P, s=P, T=2, Hkv=2, D=128, nb=4, ku=1.0, vu=1.0)
    a.update(kw)
    return L.paged_kv4_append(a["k"], a["ldk"], a["v"], a["ldv"], a["dt"], a["c"], a["s"], a["T"], a["Hkv"], a["D"],
                              a["nb"], a["ku"], a["vu"], None)


def test_append_refusals(pkv):
    L, bad, un = pkv.lib(), pkv.PKV_EINVAL, pkv.PKV_EUNSUPPORTED
    assert append(L, T=0) == pkv.PKV_OK
    for kw in (dict(T=-1), dict(Hkv=0), dict(nb=0), dict(k=None), dict(v=None), dict(c=None), dict(s=None), dict(dt=9),
               dict(ldk=255), dict(ldv=252), dict(k=P + 2), dict(v=P + 8), dict(c=P + 8), dict(ku=0.0), dict(vu=-1.0),
               dict(ku=math.inf), dict(vu=math.nan), dict(ldk=260)):
        assert append(L, **kw) == bad, kw
    for kw in (dict(D=96), dict(D=256), dict(dt=3), dict(T=(1 << 31) - 1, Hkv=1 << 20, ldk=1 << 40, ldv=1 << 40)):
        assert append(L, **kw) == un, kw


def test_page_refusals(pkv):
    L, bad, un = pkv.lib(), pkv.PKV_EINVAL, pkv.PKV_EUNSUPPORTED

    def pack(**kw):
        a = dict(c=P, nb=4, k=P, v=P, dt=1, ns=4, p=P, n=1, Hkv=2, D=64, ku=1.0, vu=1.0)
        a.update(kw)
        one = L.paged_kv4_pack_blocks(a["c"], a["nb"], a["k"], a["v"], a["dt"], a["ns"], a["p"], a["n"], a["Hkv"], a["D"],
                                      a["ku"], a["vu"], None)
        two = L.paged_kv4_expand_blocks(a["k"], a["v"], a["dt"], a["ns"], a["c"], a["nb"], a["p"], a["n"], a["Hkv"],
                                        a["D"], a["ku"], a["vu"], None)
        assert one == two
        return one
    assert pack(n=0) == pkv.PKV_OK
    for kw in (dict(n=-1), dict(ns=0), dict(nb=0), dict(Hkv=0), dict(c=None), dict(k=None), dict(v=None), dict(p=None),
               dict(c=P + 4), dict(k=P + 2), dict(v=P + 8), dict(dt=7), dict(ku=0.0), dict(vu=math.nan)):
        assert pack(**kw) == bad, kw
    for kw in (dict(D=32), dict(dt=3), dict(n=(1 << 31) - 1, Hkv=1 << 20)):
        assert pack(**kw) == un, kw

    def copy(**kw):
        a = dict(c=P, p=P, n=1, Hkv=2, D=64, nb=4)
        a.update(kw)
        return L.paged_kv4_copy_blocks(a["c"], a["p"], a["n"], a["Hkv"], a["D"], a["nb"], None)
    assert copy(n=0) == pkv.PKV_OK
    for kw in (dict(n=-1), dict(Hkv=0), dict(nb=0), dict(c=None), dict(p=None), dict(c=P + 8)):
        assert copy(**kw) == bad, kw
    assert copy(D=80) == un
    assert [L.paged_kv4_tile_bytes(d) for d in (64, 128, 96)] == [1152, 2304, 0]


def test_attention_refusals(pkv):
    L, bad, un, ws = pkv.lib(), pkv.PKV_EINVAL, pkv.PKV_EUNSUPPORTED, pkv.PKV_EWORKSPACE

    def attend(**kw):
        a = dict(o=P, q=P, dt=2, c=P, t=P, mb=4, l=P, B=2, n=1, w=0, Hq=8, Hkv=2, D=128, nb=10, s=0.1, ku=1.0, vu=1.0, ns=3,
                 ws=P, wsb=1 << 30)
        a.update(kw)
        return L.paged_kv4_decode_attention(a["o"], a["q"], a["dt"], a["c"], a["t"], a["mb"], a["l"], a["B"], a["n"], a["w"],
                                            a["Hq"], a["Hkv"], a["D"], a["nb"], a["s"], a["ku"], a["vu"], a["ns"], a["ws"],
                                            a["wsb"], None)
    assert attend(B=0) == pkv.PKV_OK
    for kw in (dict(o=None), dict(q=None), dict(c=None), dict(t=None), dict(l=None), dict(q=P + 2), dict(o=P + 8),
               dict(c=P + 8), dict(B=-1), dict(n=0), dict(n=65), dict(w=-1), dict(Hq=7), dict(nb=0), dict(mb=0), dict(dt=3),
               dict(s=math.nan), dict(s=math.inf), dict(s=3e38, ku=3e38), dict(ku=0.0), dict(vu=math.inf), dict(ns=-1)):
        assert attend(**kw) == bad, kw
    for kw in (dict(dt=0), dict(D=96), dict(mb=1 << 27), dict(B=1 << 20, mb=1 << 20)):
        assert attend(**kw) == un, kw
    for kw in (dict(ws=None), dict(ws=P + 128), dict(wsb=100)):
        assert attend(**kw) == ws, kw
    n = ctypes.c_size_t(0)
    assert L.paged_kv4_decode_workspace_bytes(2, 1, 8, 2, 128, 2, 3, ctypes.byref(n)) == pkv.PKV_OK and n.value > 0
    assert L.paged_kv4_decode_workspace_bytes(2, 1, 8, 2, 128, 0, 3, ctypes.byref(n)) == un
    assert L.paged_kv4_decode_workspace_bytes(2, 1, 8, 2, 128, 2, 3, None) == bad


def rope(L, which, **kw):
    a = dict(qo=8 * P, ldqo=512, q=P, ldq=512, ko=9 * P, ldko=256, k=2 * P, ldk=256, v=3 * P, ldv=256, dt=2, p=P, t=P, rot=64,
             il=0, m=1.0, c=5 * P, c2=6 * P, s=P, T=2, Hq=4, Hkv=2, D=128, nb=4, ku=1.0, vu=1.0)
    a.update(kw)
    head = (a["qo"], a["ldqo"], a["q"], a["ldq"])
    pos = (a["dt"], a["p"], a["t"], a["rot"], a["il"], a["m"])
    if which == "rope":
        return L.paged_rope(*head, a["ko"], a["ldko"], a["k"], a["ldk"], *pos, a["T"], a["Hq"], a["Hkv"], a["D"], None)
    rows = (a["k"], a["ldk"], a["v"], a["ldv"])
    if which == "append":
        return L.paged_rope_append(*head, *rows, *pos, a["c"], a["c2"], a["s"], a["T"], a["Hq"], a["Hkv"], a["D"], a["nb"], None)
    return L.paged_kv4_rope_append(*head, *rows, *pos, a["c"], a["s"], a["T"], a["Hq"], a["Hkv"], a["D"], a["nb"], a["ku"],
                                   a["vu"], None)


@pytest.mark.parametrize("which", ["rope", "append", "kv4"])
def test_rope_refusals(pkv, which):
    L, bad, un = pkv.lib(), pkv.PKV_EINVAL, pkv.PKV_EUNSUPPORTED
    assert rope(L, which, T=0) == pkv.PKV_OK
    for kw in (dict(T=-1), dict(Hq=-1), dict(rot=0), dict(rot=144), dict(il=2), dict(m=math.nan), dict(dt=8), dict(p=None),
               dict(t=None), dict(q=None), dict(qo=None), dict(k=None), dict(q=P + 2), dict(ldq=511), dict(ldq=516),
               dict(ldk=255), dict(qo=P, ldqo=1024), dict(qo=P + 64), dict(qo=2 * P)):
        assert rope(L, which, **kw) == bad, kw
    for kw in (dict(rot=24), dict(rot=8), dict(D=96, rot=32), dict(dt=3), dict(T=(1 << 31) - 1, Hq=1 << 20, ldq=1 << 40, ldqo=1 << 40)):
        assert rope(L, which, **kw) == un, kw
    if which == "rope":
        for kw in (dict(ko=2 * P, ldko=512), dict(ko=2 * P + 64), dict(ko=P), dict(ko=8 * P), dict(Hq=0, Hkv=0)):
            assert rope(L, which, **kw) == bad, kw
    else:
        for kw in (dict(c=None), dict(c=5 * P + 8), dict(s=None), dict(v=None), dict(ldv=10), dict(qo=3 * P), dict(nb=0),
                   dict(Hkv=0), dict(Hq=0)):
            assert rope(L, which, **kw) == bad, kw
    if which == "kv4":
        for kw in (dict(ku=0.0), dict(vu=math.inf)):
            assert rope(L, which, **kw) == bad, kw
    elif which == "append":
        assert rope(L, which, c2=None) == bad


@pytest.mark.parametrize("which", ["rope", "append", "kv4"])
def test_rope_in_place_over_other_inputs(pkv, which):
    """Queries that are turned in place must not be the keys (or the values), not even in part."""
    for kw in (dict(qo=P, ldqo=512, k=P, ldk=512), dict(qo=P, ldqo=512, k=P + 1008, ldk=512),
               dict(qo=P, ldqo=512, k=P - 512 + 16, ldk=512), dict(qo=P, ldqo=512, k=P + 16 * 1024, ldk=256, T=40)):
        assert rope(L := pkv.lib(), which, **kw) == pkv.PKV_EINVAL, kw
    if which == "rope":
        assert rope(L, which, ko=2 * P, q=2 * P + 512, ldq=512, ldk=512, ldko=512) == pkv.PKV_EINVAL
    else:
        assert rope(L, which, qo=P, ldqo=512, v=P + 16, ldv=512) == pkv.PKV_EINVAL


def test_units_range(pkv):
    L = pkv.lib()
    for unit, rc in ((2.0 ** -64, pkv.PKV_OK), (2.0 ** 64, pkv.PKV_OK), (2.0 ** -65, pkv.PKV_EINVAL), (2.0 ** 65, pkv.PKV_EINVAL)):
        assert append(L, ku=unit, T=0) == rc and append(L, vu=unit, T=0) == rc


def test_turns(pkv):
    """The fraction of a turn a position, in 2^-64, to the frequency's own 53 bits."""
    f = np.array([1.0, 0.5, 2 * math.pi, 3e-9, 0.0, 100.0, 2 * math.pi * 0.999999])
    out = np.empty(len(f), dtype=np.uint64)
    assert pkv.lib().pkv_rope_turns(out.ctypes.data, f.ctypes.data, len(f)) == 0
    for t, x in zip(out, f):
        want = x / (2 * math.pi) % 1.0
        assert abs(int(t) / 2.0 ** 64 - want) <= 2.0 ** -52 * max(1.0, x / (2 * math.pi))
    L = pkv.lib()
    for x in (math.nan, math.inf, -1.0):
        f[2] = x
        assert L.pkv_rope_turns(out.ctypes.data, f.ctypes.data, len(f)) == pkv.PKV_EINVAL
    assert L.pkv_rope_turns(None, f.ctypes.data, 2) == pkv.PKV_EINVAL
    assert L.pkv_rope_turns(out.ctypes.data, None, 2) == pkv.PKV_EINVAL
    assert L.pkv_rope_turns(out.ctypes.data, f.ctypes.data, 0) == pkv.PKV_EINVAL


def test_table_refusals(pkv):
    for kw in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=64, scaling="cubic"), dict(rot_dim=64, base=0.0),
               dict(rot_dim=64, scaling="linear", factor=0.0), dict(rot_dim=2, scaling="base", factor=2.0),
               dict(rot_dim=64, scaling="parts", factor=2.0), dict(rot_dim=64, scaling="parts", original_positions=8, slow=3, fast=3),
               dict(rot_dim=64, frequencies=[1.0] * 31)):
        with pytest.raises(ValueError):
            pkv.RopeTable(device="cpu", **kw)
    with pytest.raises(pkv.PagedKVError):
        pkv.RopeTable(4, frequencies=[1.0, math.nan], device="cpu")
    t = pkv.RopeTable(64, base=500000.0, device="cpu")
    assert np.allclose(t.frequencies, 500000.0 ** (-np.arange(0, 64, 2) / 64), rtol=1e-14)
