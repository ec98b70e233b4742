"""The paged-cache operators on the host: the oracle's hand-made values, the
workspace query, and every refusal of the C entry points and of the binding
before anything is launched."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import paged_oracle as O
from synth import f32_to_bf16_bits


@pytest.fixture(scope="module")
def L():
    import __graft_entry__ as g
    g.build()
    import sparse_kv_verify_gb300 as dk
    return dk


def bits(x):
    return f32_to_bf16_bits(np.asarray(x, dtype=np.float32))


# ------------------------------------------------------------------ oracle


def test_oracle_page_map_by_hand():
    # request 0 grows from 2 pages to 3, request 1 gives back 2 of 3, request 2 is new
    table = np.array([[4, 7, 0, 0], [1, 2, 9, 0], [0, 0, 0, 0]])
    r = O.page_map([7, 3, 0], [2, 1, 5], table, [2, 3, 0], [5, 6, 0, 0, 0, 0, 0, 0, 0, 0], 2, 4, 10, 5)
    # pushed: 2, 9 -> stack 5 6 2 9; request 0 pops 9, request 2 pops 2 and 6
    assert r["free_list"].tolist()[:4] == [5, 6, 2, 9] and r["n_free"].tolist() == [1]
    assert r["table"].tolist() == [[4, 7, 9, 0], [1, 2, 9, 0], [2, 6, 0, 0]]
    assert r["held"].tolist() == [3, 1, 2] and r["kv_len"].tolist() == [9, 4, 5] and r["cu"].tolist() == [0, 2, 3, 8]
    assert r["slot"].tolist() == [31, 36, 7, 8, 9, 10, 11, 24, -1, -1]
    assert r["pos"].tolist() == [7, 8, 3, 0, 1, 2, 3, 4, 0, 0] and r["flags"] == 0


def test_oracle_page_map_shortage_is_first_come_first_served():
    table = np.zeros((4, 4), int)
    # three free pages: 0 takes two, 1 wants two and stops the rest, 3 needs none
    r = O.page_map([0, 0, 0, 5], [8, 8, 4, 2], np.array([[0] * 4, [0] * 4, [0] * 4, [6, 7, 0, 0]]), [0, 0, 0, 2],
                   [1, 2, 3, 0, 0, 0, 0, 0], 3, 4, 40, 8)
    assert r["kv_len"].tolist() == [8, 0, 0, 7] and r["held"].tolist() == [2, 0, 0, 2] and r["flags"] == O.PAGES
    assert r["slot"][8:20].tolist() == [-1] * 12 and r["slot"][20:22].tolist() == [29, 30]
    assert r["pos"][8:16].tolist() == list(range(8)) and r["n_free"].tolist() == [1]
    # nobody's pages move while the pool's count is wrong
    for n_free in (-1, 9, 8):
        r = O.page_map([0, 9], [8, 0], table[:2], [0, 4], [0] * 8, n_free, 4, 8, 8)
        assert r["held"].tolist() == [0, 4] and r["kv_len"].tolist() == [0, 9] and r["flags"] == O.PAGES, n_free


def test_oracle_page_map_inconsistent_requests():
    t = np.zeros((5, 2), int)
    r = O.page_map([-1, 0, 0, 7, 0], [1, -3, 9, 2, 4], t, [0] * 5, [0, 1, 2, 3], 4, 4, 20, 8)
    assert r["flags"] == O.SEQLEN and r["kv_len"].tolist() == [0, 0, 0, 0, 4] and r["held"].tolist() == [0, 0, 0, 0, 1]
    assert r["cu"].tolist() == [0, 1, 1, 10, 12, 16]
    # tokens past row N: the request whose last one does not fit is not served
    r = O.page_map([0, 0], [4, 4], t[:2], [0, 0], [0, 1], 2, 4, 7, 4)
    assert r["cu"].tolist() == [0, 4, 7] and r["kv_len"].tolist() == [4, 0] and r["flags"] == O.SEQLEN


def test_oracle_norm_rope_by_hand():
    x = np.zeros((2, 1, 64), np.float32)
    x[:, 0, 0], x[:, 0, 1], x[:, 0, 32] = 3.0, 4.0, 1.0
    quarter = np.full(32, math.pi / 2)
    y, _ = O.norm_rope(bits(x), None, 0.0, quarter, [0, 1], 64, False)
    assert np.allclose(y[0, 0], x[0, 0]) and np.allclose(y[1, 0, [0, 1, 32, 33]], [-1, 0, 3, 4])
    y, _ = O.norm_rope(bits(x), None, 0.0, quarter, [0, 1], 2, True)
    assert np.allclose(y[1, 0, [0, 1, 32]], [-4, 3, 1])
    # the norm: unit mean square, a rotation keeps it
    y, _ = O.norm_rope(bits(x), bits(np.ones(64)), 0.0, quarter, [5, 7], 64, True)
    assert np.allclose((y * y).mean(axis=-1), 1)


def test_oracle_paged_attn_by_hand():
    """Zero queries weigh every visible row alike."""
    kc = np.zeros((3, 1, 2, 64), np.float32)
    vc = np.arange(6, dtype=np.float32).reshape(3, 1, 2, 1) * np.ones(64, np.float32)
    q = np.zeros((4, 1, 64), np.float32)
    # request 0: rows 4, 5, 0 (pages 2, 0), two new; request 1: one row for two queries
    o, lse, _ = O.paged_attn(bits(q), bits(kc), bits(vc), [[2, 0], [1, -1]], [0, 2, 4], [3, 1])
    assert np.allclose(o[:, 0, 0], [4.5, 3, 0, 2])
    assert np.allclose(lse[:, 0], [math.log(2), math.log(3), -math.inf, 0])
    # a page outside the pool: rows of zeros
    o, _, _ = O.paged_attn(bits(q), bits(kc), bits(vc), [[2, 9], [1, -1]], [0, 2, 4], [3, 1])
    assert np.allclose(o[:, 0, 0], [4.5, 3, 0, 2])


# --------------------------------------------------------------- workspace


def _batch(bd, **o):
    a = dict(B=2, N=8, max_new=4, max_pages=8)
    a.update(o)
    return bd.CBatch(*a.values())


BAD_BATCH = [dict(B=0), dict(N=0), dict(max_new=0), dict(max_pages=0)]
BIG_BATCH = [dict(B=8193), dict(N=(1 << 20) + 1), dict(max_new=(1 << 20) + 1)]


def test_paged_workspace_query(L):
    bd, lib = L.binding, L.lib()
    size = lambda b, *a: lib.dustin_paged_workspace_bytes(ctypes.byref(b), *a)
    base = 256 + 65536
    assert size(_batch(bd), 0, 0, 0) >= base and size(_batch(bd), 64, 8, 128) >= size(_batch(bd), 0, 0, 0)
    for o in BAD_BATCH + BIG_BATCH:
        assert size(_batch(bd, **o), 0, 0, 0) == 0, o
    for bad in [(60, 8, 128), (64, 8, 96), (64, 0, 128), (-8, 8, 128), (129, 1, 64)]:
        assert size(_batch(bd), *bad) == 0, bad
    assert lib.dustin_paged_workspace_bytes(None, 0, 0, 0) == 0
    with pytest.raises(L.DustinError):
        L.paged_workspace_bytes(L.Batch(2, 8, 4, 8), 60, 8, 128)


# ---------------------------------------------------------------- refusals


def _pool(bd, **o):
    a = dict(ptr=0x10000, hkv=8, d=128, n_pages=64, page=16, sp=8 * 16 * 128, sh=16 * 128, sl=128)
    a.update(o)
    return bd.CPagedKV(*a.values())


BAD_POOL = [dict(ptr=None), dict(ptr=0x10008), dict(d=96), dict(hkv=0), dict(n_pages=0), dict(page=0), dict(page=-16),
            dict(sl=64), dict(sl=132), dict(sp=0), dict(sh=-128), dict(sh=2052), dict(n_pages=1 << 27), dict(sp=1 << 35)]


def test_page_map_refusals(L):
    bd, lib = L.binding, L.lib()

    def call(bt=None, ws=0x100000, nbytes=1 << 20, **o):
        a = dict(page=16, n_pages=64, seq=0x1000, new=0x2000, table=0x3000, held=0x4000, free=0x5000, n_free=0x6000,
                 cu=0x7000, kv=0x8000, slot=0x9000, pos=0xA000)
        a.update(o)
        return lib.dustin_page_map(ctypes.byref(bt or _batch(bd)), *a.values(), ws, nbytes, None)
    names = ["seq", "new", "table", "held", "free", "n_free", "cu", "kv", "slot", "pos"]
    for n in names:
        assert call(**{n: None}) == -1 and call(**{n: 0x1002}) == -1, n
    for i, n in enumerate(names):
        for m in names[:i]:
            assert call(**{n: 0xB000, m: 0xB000}) == -1, (n, m)
    assert call(page=0) == -1 and call(n_pages=0) == -1 and call(page=-4) == -1
    for o in BAD_BATCH:
        assert call(_batch(bd, **o)) == -1, o
    for o in BIG_BATCH + [dict(max_pages=(1 << 16) + 1)]:
        assert call(_batch(bd, **o)) == -2, o
    assert call(n_pages=1 << 27) == -2
    assert call(_batch(bd, B=2048, max_pages=1 << 20), page=1) == -2   # a table of 2^31 entries
    assert call(ws=None) == -5 and call(ws=0x100008) == -5 and call(nbytes=1000) == -5
    assert lib.dustin_page_map(None, 16, 64, *range(0x1000, 0xB000, 0x1000), 0x100000, 1 << 20, None) == -1


def test_norm_rope_refusals(L):
    bd, lib = L.binding, L.lib()
    shape = dict(N=8, hq=64, rot=128, inter=0, eps=1e-6)

    def call(r=None, ws=0x100000, nbytes=1 << 20, **o):
        a = dict(q=0x1000, qs=8192, k=0x2000, ks=1024, v=0x3000, vs=1024, qw=0x4000, kw=0x5000, f=0x6000, pos=0x7000,
                 slot=0x8000, out=0x9000, os=8192, kc=_pool(bd), vc=_pool(bd, ptr=0x20000))
        a.update(o)
        s = dict(shape)
        s.update(r or {})
        return lib.dustin_norm_rope(ctypes.byref(bd.CRope(*s.values())), *a.values(), ws, nbytes, None)
    for r in [dict(N=0), dict(hq=0), dict(rot=-16), dict(rot=8), dict(rot=144), dict(inter=2), dict(eps=-1.0),
              dict(eps=math.nan), dict(eps=math.inf)]:
        assert call(r) == -1, r
    assert call(dict(N=(1 << 20) + 1)) == -2
    assert call(dict(hq=65537), qs=1 << 24, os=1 << 24) == -2
    assert call(ks=1 << 24, vs=1 << 24, kc=_pool(bd, hkv=65537), vc=_pool(bd, ptr=0x20000, hkv=65537)) == -2
    for o in [dict(q=None), dict(q=0x1008), dict(qs=8184), dict(qs=8196), dict(k=None), dict(ks=1016), dict(v=0x3004),
              dict(vs=0), dict(qw=0x4008), dict(kw=0x5002), dict(f=None), dict(f=0x6002), dict(pos=None), dict(slot=None),
              dict(slot=0x8001), dict(out=None), dict(os=8), dict(out=0x1000, os=8200), dict(out=0x2000), dict(out=0x3000),
              dict(out=0x4000), dict(out=0x10000), dict(k=0x10000), dict(v=0x20000), dict(q=0x10000),
              dict(vc=_pool(bd)), dict(vc=_pool(bd, ptr=0x20000, page=32)), dict(vc=_pool(bd, ptr=0x20000, hkv=4)),
              dict(vc=_pool(bd, ptr=0x20000, n_pages=63))]:
        assert call(**o) == -1, o
    for bad in BAD_POOL:
        assert call(kc=_pool(bd, **bad)) == -1, bad
        assert call(vc=_pool(bd, **dict(dict(ptr=0x20000), **bad))) == -1, bad
    assert call(ws=None) == -5 and call(nbytes=1000) == -5


def test_paged_attn_refusals(L):
    bd, lib = L.binding, L.lib()

    def call(bt=None, ws=0x100000, nbytes=1 << 30, **o):
        a = dict(hq=64, q=0x1000, kc=_pool(bd), vc=_pool(bd, ptr=0x20000), table=0x2000, cu=0x3000, kv=0x4000, o=0x5000,
                 lse=0x6000)
        a.update(o)
        return lib.dustin_paged_attn(ctypes.byref(bt or _batch(bd)), *a.values(), ws, nbytes, None)
    for o in [dict(hq=0), dict(hq=60), dict(q=None), dict(q=0x1008), dict(table=None), dict(table=0x2002), dict(cu=None),
              dict(kv=None), dict(o=None), dict(o=0x5008), dict(o=0x5010), dict(lse=0x6002), dict(lse=0x5000), dict(o=0x1000),
              dict(o=0x10000), dict(o=0x20000), dict(o=0x2000), dict(lse=0x2000), dict(lse=0x3000), dict(lse=0x4000),
              dict(vc=_pool(bd, ptr=0x20000, d=64, sl=64)), dict(vc=_pool(bd, ptr=0x20000, n_pages=3))]:
        assert call(**o) == -1, o
    for bad in BAD_POOL:
        assert call(kc=_pool(bd, **bad)) == -1, bad
        assert call(vc=_pool(bd, **dict(dict(ptr=0x20000), **bad))) == -1, bad
    for page in (1, 8, 24, 48, 96, 192):
        assert call(kc=_pool(bd, page=page), vc=_pool(bd, ptr=0x20000, page=page)) == -1, page
    for o in BAD_BATCH:
        assert call(_batch(bd, **o)) == -1, o
    for o in BIG_BATCH + [dict(max_pages=(1 << 16) + 1)]:
        assert call(_batch(bd, **o)) == -2, o
    assert call(hq=8 * 129) == -2
    assert call(hq=65537, kc=_pool(bd, hkv=65537), vc=_pool(bd, ptr=0x20000, hkv=65537)) == -2
    assert call(ws=None) == -5 and call(nbytes=1000) == -5


def test_binding_refuses_wrong_tensors(L):
    """Shapes, types and devices are checked before the library is called."""
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    bt = L.Batch(2, 8, 4, 3)
    good = [i(2), i(2), i(2, 3), i(2), i(9), i(1)]
    with pytest.raises(ValueError, match="CUDA"):
        L.PageMapCall(bt, 16, *good)
    for n, bad in enumerate([i(3), i(1), i(2, 4), i(3), i(3, 3), i(2)]):
        with pytest.raises(ValueError):
            L.PageMapCall(bt, 16, *good[:n], bad, *good[n + 1:])
    with pytest.raises(ValueError):
        L.PageMapCall(bt, 16, *good, slot=i(7))
    r = L.Rope(64)
    f, kc = torch.zeros(32), bf(3, 2, 16, 64)
    good = [bf(8, 4, 64), bf(8, 2, 64), bf(8, 2, 64), bf(64), bf(64), f, i(8), i(8), kc, kc.clone()]
    with pytest.raises(ValueError, match="CUDA"):
        L.NormRopeCall(r, *good)
    for n, bad in enumerate([bf(8, 4, 64, 1), bf(7, 2, 64), bf(8, 3, 64), bf(32), bf(128), f[:31], i(7), i(9),
                             bf(3, 2, 16, 128), bf(4, 2, 16, 64)]):
        with pytest.raises(ValueError):
            L.NormRopeCall(r, *good[:n], bad, *good[n + 1:])
    with pytest.raises(ValueError, match="packed"):
        L.NormRopeCall(r, bf(8, 4, 128)[..., ::2], *good[1:])
    with pytest.raises(TypeError):
        L.NormRopeCall(r, *good[:5], None, *good[6:])
    good = [bf(8, 4, 64), kc, kc.clone(), i(2, 3), i(3), i(2)]
    with pytest.raises(ValueError, match="CUDA"):
        L.PagedAttnCall(bt, *good)
    for n, bad in enumerate([bf(7, 4, 64), bf(3, 2, 16, 128), bf(3, 2, 32, 64), i(3, 3), i(2), i(3)]):
        with pytest.raises(ValueError):
            L.PagedAttnCall(bt, *good[:n], bad, *good[n + 1:])
    with pytest.raises(ValueError):
        L.PagedAttnCall(bt, *good, o=bf(8, 4, 128))
    with pytest.raises(ValueError):
        L.paged_view(bf(3, 2, 16, 128)[..., ::2])
