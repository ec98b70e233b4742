"""The cache operators on the host: the oracle's hand-made values, the
workspace query, and every refusal of the C entry points and of the binding
before anything is launched."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import cache_oracle as O
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


def test_oracle_window_by_hand():
    """Zero queries weigh every visible key alike, so outputs are means of
    values and the log-sum-exp is the log of their number."""
    Lc, T = 6, 3
    V = np.arange(1, Lc + 1, dtype=np.float32)[None, None, :, None] * np.ones((1, 1, 1, 64), np.float32)
    Vb = 100.0 * np.arange(1, T + 1, dtype=np.float32)[None, None, :, None] * np.ones((1, 1, 1, 64), np.float32)
    K, Kb = np.zeros_like(V), np.zeros_like(Vb)
    Q = np.zeros((1, T, 1, 64), np.float32)
    run = lambda s, w, n=Lc: O.window_attn(bits(Q), bits(K), bits(V), bits(Kb), bits(Vb), [n], s, w)
    # window 2, one sink: query 0 (position 6) sees positions 0, 5 and itself
    o, lse = run(1, 2)
    assert np.allclose(o[0, :, 0, 0], [(1 + 6 + 100) / 3, (1 + 100 + 200) / 3, (1 + 200 + 300) / 3])
    assert np.allclose(lse, math.log(3))
    # no window: the sinks alone; no sinks either: nothing
    o, lse = run(2, 0)
    assert np.allclose(o[0, :, 0, 0], 1.5) and np.allclose(lse, math.log(2))
    o, lse = run(0, 0)
    assert np.all(o == 0) and np.all(np.isneginf(lse))
    # an empty cache: block rows are the sinks and the window
    o, lse = run(1, 1, 0)
    assert np.allclose(o[0, :, 0, 0], [100, 150, 200])
    # a window past everything: the causal block over the whole cache
    o, _ = run(0, 99)
    assert np.allclose(o[0, 2, 0, 0], (21 + 600) / 9)


def test_oracle_prefix_is_dense_over_the_joined_rows():
    rng = np.random.default_rng(3)
    mk = lambda *s: bits(rng.standard_normal(s))
    Q, PK, PV, K, V, Kb, Vb = (mk(2, 2, 4, 64), mk(1, 2, 9, 64), mk(1, 2, 9, 64), mk(2, 2, 6, 64),
                               mk(2, 2, 6, 64), mk(2, 2, 2, 64), mk(2, 2, 2, 64))
    o, lse = O.prefix_attn(Q, PK, PV, 7, K, V, Kb, Vb, [5, 0])
    join = lambda a, b, n: np.concatenate([a[:, :, :7], b[:, :, :n]], axis=2)
    for b, n in ((0, 5), (1, 0)):
        o1, l1 = O.window_attn(Q[b:b + 1], join(PK, K[b:b + 1], n), join(PV, V[b:b + 1], n), Kb[b:b + 1],
                               Vb[b:b + 1], [7 + n], 0, 10 ** 6)
        assert np.allclose(o[b], o1[0], atol=1e-12) and np.allclose(lse[b], l1[0], atol=1e-12)


def test_oracle_accumulate_rows_sum_to_the_query_rows():
    """With the log-sum-exp of the same keys every accepted row adds one in
    all; rows that the causal rule hides from a query get nothing of it."""
    rng = np.random.default_rng(4)
    Q, K = bits(rng.standard_normal((1, 3, 2, 64))), bits(rng.standard_normal((1, 1, 9, 64)))
    lse = np.full((1, 3, 2), -math.inf)
    from oracle.dustin_oracle import bf16
    for t in range(3):
        for h in range(2):
            z = bf16(K[0, 0, :5 + t]) @ bf16(Q[0, t, h]) / 8.0
            lse[0, t, h] = np.log(np.exp(z).sum())
    w0 = np.ones((1, 1, 12))
    w, pos = O.accumulate(Q, lse, K, [2], [6], [106], w0, np.zeros((1, 1, 12), np.int32))
    # rows 4 and 5 are new: they start from 0; rows 0..3 had 1 each
    assert np.isclose(w[0, 0, :6].sum() - 4, 2 * 2)
    assert np.all(w[0, 0, 6:] == 1) and pos[0, 0].tolist() == [0, 0, 0, 0, 104, 105] + [0] * 6


def test_oracle_evict_by_hand():
    w = np.array([5, 1, 9, 1, 7, 1, 0, 0], np.float32)
    pos = np.arange(8, dtype=np.int32)
    # k = 5 of 8, one sink, two recent: rows 0, 6, 7 and then 2 and 4 stay
    dst, src = O.evict_rows(w, pos, 8, 5, 1, 2, 8)
    assert dst.tolist() == [1, 3] and src.tolist() == [6, 7]
    # equal weights: the lower rows stay
    dst, src = O.evict_rows(np.ones(8), pos, 8, 5, 0, 0, 8)
    assert dst.size == 0 and src.size == 0
    assert O.evict_rows(w, pos, 5, 5, 0, 0, 8)[0].size == 0
    # more protected rows than the budget: the lower ones stay
    dst, src = O.evict_rows(w, np.full(8, 7), 8, 3, 0, 1, 8)
    assert dst.size == 0 and src.size == 0


# --------------------------------------------------------------- workspace


def test_cache_workspace_query(L):
    bd = L.binding
    lib = L.lib()
    size = lambda p, *a: lib.dustin_cache_workspace_bytes(ctypes.byref(bd.CParams(*p)), *a)
    good = (2, 1024, 4, 4, 32, 32, 128)
    base = 256 + 65536
    assert size(good, 0, 1, 0, 0, 0) >= base
    # eviction lists: two int32 lists of k rows per layer and unit at most
    assert size(good, 0, 8, 128, 3, 0) >= size(good, 0, 8, 128, 1, 0) >= base
    assert size(good, 64, 8, 128, 0, 4096) >= size(good, 64, 8, 128, 0, 0) >= base
    for bad in [(64, 0, 128, 0, 0), (60, 8, 128, 0, 0), (64, 8, 96, 0, 0), (64, 8, 128, 17, 0),
                (64, 8, 128, -1, 0), (64, 8, 128, 0, -1), (64, 8, 128, 0, (1 << 20) + 1)]:
        assert size(good, *bad) == 0, bad
    assert size((0,) + good[1:], 64, 8, 128, 0, 0) == 0
    assert size((2, 1024, 64, 4, 32, 32, 128), 8, 8, 128, 0, 0) == 0      # 65 block rows
    assert size((2, 1024, 16, 4, 32, 32, 128), 64, 8, 128, 0, 0) == 0     # 17 x 8 query rows
    assert size((16385, 1024, 0, 4, 32, 32, 128), 1, 1, 64, 0, 0) == 0    # units
    with pytest.raises(L.DustinError):
        L.cache_workspace_bytes(L.Params(2, 1024, 4, 4, 32, 32, 128), 60, 8, 128)


# ---------------------------------------------------------------- refusals


def _kv(bd, **o):
    a = dict(ptr=0x10000, hkv=8, d=128, sb=8 * 1024 * 128, sh=1024 * 128, sl=128)
    a.update(o)
    return bd.CKV(a["ptr"], a["hkv"], a["d"], a["sb"], a["sh"], a["sl"])


def _params(bd, **o):
    a = dict(B=2, Lcap=1024, gamma=4, sinks=4, window=32, m=32, k=128)
    a.update(o)
    return bd.CParams(*a.values())


BAD_KV = [dict(ptr=None), dict(ptr=0x10008), dict(d=96), dict(sl=64), dict(sb=0), dict(sh=-128),
          dict(sh=1024 * 128 + 4), dict(hkv=0)]


def test_window_refusals(L):
    bd, lib = L.binding, L.lib()

    def call(p=None, ws=0x100000, nbytes=1 << 30, **o):
        a = dict(hq=64, q=0x1000, k=_kv(bd), v=_kv(bd), kb=0x2000, vb=0x3000, sl=0x5000, o=0x6000, lse=0x7000)
        a.update(o)
        return lib.dustin_window_attn(ctypes.byref(p or _params(bd)), *a.values(), ws, nbytes, None)
    for o in [dict(q=None), dict(q=0x1008), dict(kb=None), dict(vb=0x3004), dict(sl=None), dict(o=None),
              dict(o=0x6008), dict(o=0x1000), dict(lse=0x6000), dict(lse=0x7002), dict(hq=60), dict(hq=0)]:
        assert call(**o) == -1, o
    for bad in BAD_KV:
        assert call(k=_kv(bd, **bad)) == -1, bad
        assert call(v=_kv(bd, **bad)) == -1, bad
    assert call(v=_kv(bd, hkv=4)) == -1 and call(v=_kv(bd, d=64)) == -1
    for o in [dict(B=0), dict(Lcap=0), dict(Lcap=(1 << 20) + 1), dict(gamma=-1), dict(k=0), dict(window=200)]:
        assert call(_params(bd, **o)) == -1, o
    assert call(_params(bd, gamma=16)) == -2               # 17 x 8 query rows
    assert call(_params(bd, gamma=64), hq=8) == -2         # 65 block rows
    assert call(_params(bd, B=2049)) == -2                 # 16392 units
    assert call(ws=None) == -5 and call(ws=0x100008) == -5 and call(nbytes=1000) == -5


def test_prefix_refusals(L):
    bd, lib = L.binding, L.lib()

    def call(p=None, ws=0x100000, nbytes=1 << 30, **o):
        a = dict(hq=64, q=0x1000, pk=_kv(bd), pv=_kv(bd), cap=1024, n=0x8000, k=_kv(bd), v=_kv(bd), kb=0x2000,
                 vb=0x3000, sl=0x5000, o=0x6000, lse=None)
        a.update(o)
        return lib.dustin_prefix_attn(ctypes.byref(p or _params(bd)), *a.values(), ws, nbytes, None)
    for o in [dict(q=None), dict(n=None), dict(cap=0), dict(cap=-1), dict(sl=None), dict(o=0x1000),
              dict(pk=_kv(bd, hkv=4)), dict(pv=_kv(bd, d=64)), dict(v=_kv(bd, hkv=4))]:
        assert call(**o) == -1, o
    for bad in BAD_KV:
        assert call(pk=_kv(bd, **bad)) == -1, bad
        assert call(pv=_kv(bd, **bad)) == -1, bad
    assert call(cap=(1 << 20) + 1) == -2
    assert call(_params(bd, gamma=16)) == -2
    assert call(ws=None) == -5 and call(nbytes=1000) == -5


def test_accumulate_refusals(L):
    bd, lib = L.binding, L.lib()

    def call(p=None, ws=0x100000, nbytes=1 << 20, **o):
        a = dict(hq=64, q=0x1000, lse=0x2000, k=_kv(bd), n=0x3000, sl=0x4000, seen=0x5000, w=0x6000, pos=0x7000)
        a.update(o)
        return lib.dustin_accumulate(ctypes.byref(p or _params(bd)), *a.values(), ws, nbytes, None)
    for o in [dict(q=None), dict(q=0x1004), dict(lse=None), dict(lse=0x2001), dict(n=None), dict(sl=None),
              dict(seen=None), dict(w=None), dict(w=0x6002), dict(pos=None), dict(pos=0x6000), dict(w=0x2000),
              dict(hq=63)]:
        assert call(**o) == -1, o
    for bad in BAD_KV:
        assert call(k=_kv(bd, **bad)) == -1, bad
    assert call(_params(bd, gamma=16)) == -2
    assert call(ws=None) == -5 and call(nbytes=1000) == -5


def test_evict_refusals(L):
    bd, lib = L.binding, L.lib()
    ptrs = lambda *x: (ctypes.c_void_p * len(x))(*x)

    def call(p=None, n=2, ws=0x100000, nbytes=1 << 30, **o):
        a = dict(k=[_kv(bd), _kv(bd, ptr=0x20000)], v=[_kv(bd, ptr=0x30000), _kv(bd, ptr=0x40000)],
                 w=[0x1000, 0x2000], pos=[0x3000, 0x4000], seen=0x5000, sl=0x6000)
        a.update(o)
        return lib.dustin_evict(ctypes.byref(p or _params(bd)), n, (bd.CKV * 2)(*a["k"]), (bd.CKV * 2)(*a["v"]),
                                ptrs(*a["w"]), ptrs(*a["pos"]), a["seen"], a["sl"], ws, nbytes, None)
    for o in [dict(n=0), dict(w=[0x1000, None]), dict(pos=[None, 0x4000]), dict(w=[0x1000, 0x2001]),
              dict(seen=None), dict(sl=None), dict(sl=0x5000), dict(w=[0x1000, 0x1000]),
              dict(pos=[0x3000, 0x3000]), dict(pos=[0x3000, 0x2000]), dict(v=[_kv(bd)] * 2),
              dict(k=[_kv(bd), _kv(bd, ptr=0x20000, hkv=4)]), dict(v=[_kv(bd, ptr=0x30000, d=64)] * 2)]:
        assert call(**o) == -1, o
    for bad in BAD_KV:
        assert call(k=[_kv(bd), _kv(bd, **bad)]) == -1, bad
    assert call(n=17) == -2
    assert call(_params(bd, B=2049)) == -2
    assert call(ws=None) == -5 and call(nbytes=1000) == -5


def test_binding_refuses_wrong_tensors(L):
    """Shapes, types and devices are checked before the library is called."""
    p = L.Params(2, 64, 1, 2, 8, 0, 16)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    q, k, kb, sl = bf(2, 2, 4, 64), bf(2, 2, 64, 64), bf(2, 2, 2, 64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        L.dustin_window_attn(p, q, k, k, kb, kb, sl)
    for a in [(bf(2, 3, 4, 64), k, k, kb, kb, sl), (q, bf(2, 2, 65, 64), k, kb, kb, sl), (q, k, bf(2, 1, 64, 64), kb, kb, sl),
              (q, k, k, bf(2, 2, 3, 64), kb, sl), (q, k, k, kb, kb, sl[:1]), (q[0], k, k, kb, kb, sl)]:
        with pytest.raises(ValueError):
            L.dustin_window_attn(p, *a)
    with pytest.raises(ValueError):
        L.dustin_window_attn(p, q, k, k, kb, kb, sl, o=bf(2, 2, 4, 128))
    with pytest.raises(ValueError):
        L.dustin_prefix_attn(p, q, bf(2, 2, 9, 64), bf(2, 2, 9, 64), sl[:1], k, k, kb, kb, sl)
    w, pos, lse = torch.zeros(2, 2, 64), torch.zeros(2, 2, 64, dtype=torch.int32), torch.zeros(2, 2, 4)
    with pytest.raises(ValueError):
        L.dustin_accumulate(p, q, lse, k, sl, sl, sl, w[:, :, :60], pos)
    with pytest.raises(ValueError):
        L.dustin_accumulate(p, q, lse[:, :1], k, sl, sl, sl, w, pos)
    with pytest.raises(ValueError):
        L.dustin_evict(p, [k], [k, k], [w], [pos], sl, sl)
    with pytest.raises(ValueError):
        L.dustin_evict(p, [], [], [], [], sl, sl)


def test_evict_call_refuses_caches_of_other_ranks(L):
    p = L.Params(1, 8, 0, 0, 0, 0, 4)
    flat, w, i = torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 8), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        L.EvictCall(p, [flat], [flat], [w], [w.int()], i, i)
    with pytest.raises(ValueError):
        L.EvictCall(p, [flat[0]], [flat[0]], [w], [w.int()], i, i)


def test_outputs_that_are_inputs_are_refused(L):
    """Units write their rows while others still read: no input can be an output."""
    bd, lib = L.binding, L.lib()
    k, v = _kv(bd, ptr=0x10000), _kv(bd, ptr=0x20000)
    pk, pv = _kv(bd, ptr=0x30000), _kv(bd, ptr=0x40000)
    ws = (0x100000, 1 << 30, None)
    p = ctypes.byref(_params(bd))
    for out in (0x1000, 0x2000, 0x3000, 0x5000, 0x10000, 0x20000):
        assert lib.dustin_window_attn(p, 64, 0x1000, k, v, 0x2000, 0x3000, 0x5000, out, 0x7000, *ws) == -1, hex(out)
        assert lib.dustin_window_attn(p, 64, 0x1000, k, v, 0x2000, 0x3000, 0x5000, 0x6000, out, *ws) == -1, hex(out)
    for out in (0x1000, 0x2000, 0x3000, 0x5000, 0x8000, 0x10000, 0x20000, 0x30000, 0x40000):
        for o, lse in ((out, 0x7000), (0x6000, out)):
            assert lib.dustin_prefix_attn(p, 64, 0x1000, pk, pv, 1024, 0x8000, k, v, 0x2000, 0x3000, 0x5000, o, lse,
                                          *ws) == -1, hex(out)
    for out in (0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x10000):
        for w, pos in ((out, 0x7000), (0x6000, out)):
            assert lib.dustin_accumulate(p, 64, 0x1000, 0x2000, k, 0x3000, 0x4000, 0x5000, w, pos, *ws) == -1, hex(out)
