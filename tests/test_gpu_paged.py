"""The paged-cache operators against float64 (whole numbers: exactly): block
tables and slots, head norms with the rotation and the cache write, attention of
ragged new tokens, and a serving loop of them together."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU too
    pytest.skip("needs a GPU", allow_module_level=True)

import sparse_kv_verify_gb300 as dk  # noqa: E402
from oracle import paged_oracle as O  # noqa: E402
from synth import to_bits  # noqa: E402

from _cache_cases import assert_attended, attend64, i32, logit_error, normal  # noqa: E402
from _paged_cases import NAN, Paged, assert_rotated, pages_of  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def workspace(bt, hq=0, hkv=1, d=128):
    return dk.binding.Workspace(dk.paged_workspace_bytes(bt, hq, hkv, d))


# ---------------------------------------------------------------- page map


def check_map(seq_len, n_new, table, held, free_list, n_free, page, N, max_new):
    """One call against the oracle, every output and every entry left alone."""
    bt = dk.Batch(len(seq_len), N, max_new, table.shape[1])
    ws = workspace(bt)
    dev = [i32(x) for x in (seq_len, n_new, table, held, free_list, [n_free])]
    out = [torch.full((n,), -99, dtype=torch.int32, device="cuda") for n in (bt.B + 1, bt.B, N, N)]
    got = dk.dustin_page_map(bt, page, *dev, *out, ws=ws)
    flags = dk.check(ws)
    ref = O.page_map(seq_len, n_new, table, held, free_list, n_free, page, N, max_new)
    names = ("table", "held", "free_list", "n_free")
    for name, t in list(zip(names, dev[2:])) + list(zip(("cu", "kv_len", "slot", "pos"), got)):
        assert np.array_equal(t.cpu().numpy(), ref[name]), name
    assert flags == ref["flags"]
    return ref


def random_pool(rng, B, page, width, top_new, spare):
    """A consistent state: requests that hold pages for about what they have."""
    seq = rng.integers(0, width * page // 2 + 1, B)
    new = np.minimum(rng.integers(0, top_new + 1, B), width * page - seq)
    held = np.clip(-(-(seq + rng.integers(-page, 3 * page, B)) // page), 0, width)
    extra = int(spare * np.maximum(0, -(-(seq + new) // page) - held).sum())
    n_pages = int(held.sum()) + extra + 2
    order = rng.permutation(n_pages)
    table, at = rng.integers(-5, 5, (B, width)), 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    return seq, new, table, held, np.concatenate([order[at:at + extra], np.full(n_pages - extra, -3)]), extra


@pytest.mark.parametrize("B,page,width,top_new,spare,pad", [
    (1, 16, 4, 1, 1, 0), (1, 1, 9, 5, 1, 2), (3, 7, 6, 9, 1, 0), (33, 16, 40, 1, 1, 5), (64, 64, 9, 200, 1, 0),
    (200, 16, 30, 50, 0.5, 1), (200, 256, 3, 300, 0, 0), (1023, 16, 8, 3, 1, 0), (1025, 3, 20, 8, 0.9, 7),
    (8192, 16, 5, 2, 1, 0), (2, 16, 4000, 30000, 1, 0), (40, 128, 60, 2000, 1, 100)])
def test_map_parity(B, page, width, top_new, spare, pad):
    rng = np.random.default_rng(B + page)
    for _ in range(2):
        seq, new, table, held, free, n_free = random_pool(rng, B, page, width, top_new, spare)
        check_map(seq, new, table, held, free, n_free, page, max(1, int(new.sum()) + pad), max(1, top_new))


def test_map_flags():
    rng = np.random.default_rng(1)
    seq, new, table, held, free, n_free = random_pool(rng, 12, 16, 8, 20, 1)
    N = int(new.sum())
    # inconsistent requests among good ones
    for b, (s, n, h) in enumerate([(-1, 2, 0), (5, -1, 1), (5, 21, 2), (127, 5, 8), (8, 8, -1), (8, 8, 9),
                                   (2 ** 31 - 1, 1, 0), (3, 2 ** 31 - 1, 0)]):
        s2, n2, h2 = seq.copy(), new.copy(), held.copy()
        s2[3], n2[3], h2[3] = s, n, h
        if s < 2 ** 31 - 1:
            r = check_map(s2, n2, table, h2, free, n_free, 16, N + 100, 20)
            assert r["flags"] & O.SEQLEN
    # tokens past row N
    r = check_map(seq, new, table, held, free, n_free, 16, N - 3, 20)
    assert r["flags"] == O.SEQLEN
    # a pool whose count is wrong
    for bad in (-1, len(free) + 1, len(free)):
        r = check_map(seq, new, table, held, free, bad, 16, N, 20)
        assert r["flags"] == O.PAGES
    # a table that holds what is no page
    t2 = table.copy()
    t2[:, 0] = 10 ** 6
    r = check_map(seq, new, t2, held, free, n_free, 16, N, 20)
    assert r["flags"] == O.INDEX


@pytest.mark.parametrize("n_pages", [150, 50])
def test_map_passes_never_share_a_page(n_pages):
    """Passes of a server: requests come, decode, lose rejected tokens and end;
    pages are conserved and no two requests hold the same one."""
    rng = np.random.default_rng(7)
    B, page, width, N, top = 24, 16, 20, 600, 40
    seq, table, held = np.zeros(B, int), i32(np.zeros((B, width))), i32(np.zeros(B))
    free, n_free = i32(rng.permutation(n_pages)), i32([n_pages])
    bt = dk.Batch(B, N, top, width)
    ws = workspace(bt)
    dseq, dnew = i32(seq), i32(seq)
    call = dk.PageMapCall(bt, page, dseq, dnew, table, held, free, n_free, ws=ws)
    short = 0
    for step in range(40):
        new = np.where(seq == 0, rng.integers(0, top + 1, B), rng.integers(0, 7, B))
        ended = (seq + new > width * page - 8) | (rng.random(B) < 0.05)
        seq, new = np.where(ended, 0, seq), np.where(ended, 0, new)
        dseq.copy_(i32(seq))
        dnew.copy_(i32(new))
        before = [x.cpu().numpy() for x in (table, held, free, n_free)]
        cu, kv, slot, pos = [t.cpu().numpy() for t in call()]
        ref = O.page_map(seq, new, before[0], before[1], before[2], before[3][0], page, N, top)
        for name, t in (("table", table), ("held", held), ("free_list", free), ("n_free", n_free)):
            assert np.array_equal(t.cpu().numpy(), ref[name]), (step, name)
        assert np.array_equal(slot, ref["slot"]) and np.array_equal(kv, ref["kv_len"])
        assert dk.check(ws) == ref["flags"]
        short += ref["flags"] != 0
        h = held.cpu().numpy()
        owned = np.concatenate([table.cpu().numpy()[b, :h[b]] for b in range(B)])
        pool = free.cpu().numpy()[:int(n_free)]
        assert sorted(np.concatenate([owned, pool]).tolist()) == list(range(n_pages))
        used = slot[slot >= 0]
        assert len(set(used.tolist())) == used.size
        kept = np.where(kv > 0, rng.integers(0, 1 + np.maximum(new, 0)), 0)     # some tokens are rejected
        seq = np.where(kv > 0, seq + kept, seq)
    assert short < 40 and (short > 0) == (n_pages < 100)


# --------------------------------------------------------------- norm, rope


def rope_case(N, hq, hkv, d, page, rot, seed, far=1 << 20, layout="head", fused=True):
    rng = np.random.default_rng(seed)
    n_pages = pages_of(N, page) + 3
    x = Paged([1], [0], 1, hkv, d, page=page, spare=n_pages - 1, layout=layout)
    x.kc.copy_(normal(seed, *x.kc.shape))
    x.vc.copy_(normal(seed + 1, *x.vc.shape))
    if fused:
        t = normal(seed + 2, N, hq + 2 * hkv, d)
        q, k, v = t[:, :hq], t[:, hq:hq + hkv], t[:, hq + hkv:]
    else:
        q, k, v = normal(seed + 2, N, hq, d), normal(seed + 3, N, hkv, d), normal(seed + 4, N, hkv, d)
    pos = rng.integers(0, far, N)
    pos[0] = far - 1
    slot = rng.permutation(n_pages * page)[:N]
    w = [(1 + normal(seed + 5 + i, d, scale=0.3).float()).to(torch.bfloat16) for i in range(2)]
    inv = np.float32([1e6 ** (-2 * j / max(rot, 1)) for j in range(rot // 2)])
    return x, q, k, v, w, pos, slot, inv


def check_rope(x, q, k, v, w, pos, slot, inv, rot, interleaved=False, eps=1e-6, norm=True, flags=0, q_out=None):
    page = x.kc.shape[2]
    kc, vc = to_bits(x.kc).copy(), to_bits(x.vc).copy()
    qb, kb, vb = to_bits(q).copy(), to_bits(k).copy(), to_bits(v).copy()
    ws = workspace(dk.Batch(1, 1, 1, 1))
    qw, kw = (w if norm else (None, None))
    got = dk.dustin_norm_rope(dk.Rope(rot, interleaved, eps), q, k, v, qw, kw,
                              torch.as_tensor(inv, device="cuda") if rot else None, i32(pos), i32(slot), x.kc, x.vc, q_out,
                              ws=ws)
    assert dk.check(ws) == flags
    bits = lambda t: None if t is None else to_bits(t)
    ref, size = O.norm_rope(qb, bits(qw), eps, inv, pos, rot, interleaved)
    assert_rotated(got, ref, size)
    rows, ksize = O.norm_rope(kb, bits(kw), eps, inv, pos, rot, interleaved)
    ok = (slot >= 0) & (slot < x.n_pages * page)
    at, r = slot[ok] // page, slot[ok] % page
    assert_rotated(x.kc[at, :, r], rows[ok], ksize[ok])
    assert np.array_equal(to_bits(x.vc)[at, :, r], vb[ok])
    # every other row as it was
    gk, gv = to_bits(x.kc).copy(), to_bits(x.vc).copy()
    gk[at, :, r], gv[at, :, r] = kc[at, :, r], vc[at, :, r]
    assert np.array_equal(gk, kc) and np.array_equal(gv, vc)
    return got


@pytest.mark.parametrize("N,hq,hkv,d,page,rot,interleaved,layout,fused", [
    (1, 64, 8, 128, 16, 128, False, "head", True), (1, 1, 1, 64, 16, 64, False, "head", False),
    (7, 14, 2, 64, 16, 64, False, "token", True), (5, 14, 2, 64, 32, 32, True, "head", False),
    (96, 64, 8, 128, 64, 128, False, "padded", True), (33, 8, 8, 128, 128, 64, False, "token", True),
    (130, 3, 1, 128, 1, 16, True, "head", True), (61, 5, 5, 64, 24, 48, False, "head", False),
    (9, 128, 1, 64, 100, 16, False, "padded", False), (1001, 16, 4, 128, 256, 112, True, "head", True),
    (4, 2, 1, 64, 16, 0, False, "head", True), (300, 40, 2, 64, 16, 64, True, "token", True)])
def test_rope_parity(N, hq, hkv, d, page, rot, interleaved, layout, fused):
    for norm in (True, False):
        c = rope_case(N, hq, hkv, d, page, rot, N + hq, layout=layout, fused=fused)
        check_rope(*c, rot, interleaved, norm=norm)


def test_rope_in_place_and_strided_output():
    x, q, k, v, w, pos, slot, inv = rope_case(50, 14, 2, 64, 16, 64, 3)
    ref = check_rope(x, q, k, v, w, pos, slot, inv, 64)
    wide = torch.full((50, 15, 64), NAN, dtype=torch.bfloat16, device="cuda")
    got = check_rope(x, q, k, v, w, pos, slot, inv, 64, q_out=wide[:, :14])
    assert torch.equal(got, ref) and bool(wide[:, 14].isnan().all())
    kv = torch.cat([k, v], dim=1).clone()
    got = check_rope(x, q, k, v, w, pos, slot, inv, 64, q_out=q)
    assert torch.equal(got, ref) and torch.equal(torch.cat([k, v], dim=1), kv)


def test_rope_padding_rows_and_bad_slots():
    x, q, k, v, w, pos, slot, inv = rope_case(40, 8, 2, 128, 16, 128, 4)
    slot[[0, 7, 39]] = -1
    check_rope(x, q, k, v, w, pos, slot, inv, 128)
    slot[5], slot[6], slot[8] = x.n_pages * 16, -2, 2 ** 31 - 1
    check_rope(x, q, k, v, w, pos, slot, inv, 128, flags=dk.DEV_INDEX)


def test_rope_extremes():
    """Rows of zeros, huge and tiny rows, infinities and NaN: these stay in their head."""
    x, q, k, v, w, pos, slot, inv = rope_case(12, 4, 2, 64, 16, 64, 5)
    q[0], q[1], q[2] = 0, 1e-30, 2.0 ** 60
    k[0] = 0
    check_rope(x, q, k, v, w, pos, slot, inv, 64)
    q2 = q.clone()
    q2[3, 1, 5], q2[4, 2, 40] = math.inf, NAN
    k2, v2 = k.clone(), v.clone()
    k2[5, 0, 0], v2[6, 1, 3] = NAN, math.inf
    ws = workspace(dk.Batch(1, 1, 1, 1))
    args = (w[0], w[1], torch.as_tensor(inv, device="cuda"), i32(pos), i32(slot))
    a = dk.dustin_norm_rope(dk.Rope(64), q.contiguous(), k.contiguous(), v.contiguous(), *args, x.kc, x.vc, ws=ws)
    ka, va = x.kc.clone(), x.vc.clone()
    b = dk.dustin_norm_rope(dk.Rope(64), q2, k2, v2, *args, x.kc, x.vc, ws=ws)
    same = torch.ones(12, 4, dtype=torch.bool, device="cuda")
    same[3, 1] = same[4, 2] = False
    assert torch.equal(a[same], b[same]) and bool(b[4, 2].isnan().all())
    at, r = slot // 16, slot % 16
    assert bool(x.kc[at[5], 0, r[5]].isnan().all()) and torch.equal(x.kc[at[5], 1, r[5]], ka[at[5], 1, r[5]])
    assert x.vc[at[6], 1, r[6], 3] == math.inf
    assert torch.equal(x.kc[at[6], :, r[6]], ka[at[6], :, r[6]])


def test_rope_into_a_contiguous_cache():
    """A contiguous cache is a pool of one page a sequence: slot = b * Lcap + position."""
    B, hkv, Lcap, d = 3, 2, 70, 64
    kc, vc = normal(1, B, hkv, Lcap, d), normal(2, B, hkv, Lcap, d)
    q, k, v = normal(3, 6, 4, d), normal(4, 6, hkv, d), normal(5, 6, hkv, d)
    b, pos = np.array([0, 0, 1, 1, 2, 2]), np.array([0, 1, 68, 69, 5, 6])
    inv = np.float32([1e4 ** (-2 * j / d) for j in range(d // 2)])
    dk.dustin_norm_rope(dk.Rope(d), q, k, v, None, None, torch.as_tensor(inv, device="cuda"), i32(pos),
                        i32(b * Lcap + pos), kc, vc)
    ref, size = O.norm_rope(to_bits(k), None, 0, inv, pos, d, False)
    assert_rotated(kc[b, :, pos], ref, size)
    assert torch.equal(vc[b, :, pos], v)


# --------------------------------------------------------------- attention


ATTN = [
    # ctx, new, hq, hkv, d, page
    ([0], [1], 1, 1, 64, 16),
    ([1000], [1], 8, 1, 128, 16),                      # single tokens
    ([300, 70, 0], [1, 1, 1], 8, 2, 64, 32),
    ([127, 128, 129, 255, 256], [1] * 5, 4, 2, 128, 64),
    ([15, 16, 17, 31], [1, 2, 1, 2], 2, 2, 64, 16),    # pages that end inside tiles
    ([200, 0, 1], [5, 5, 5], 8, 2, 64, 16),
    ([500, 40, 333, 90], [6, 6, 6, 6], 16, 2, 128, 64),
    ([90, 250, 0], [6, 0, 3], 14, 2, 64, 16),          # G = 7, an idle request
    ([0], [130], 8, 2, 128, 16),                       # a prompt from its first token on
    ([0, 0, 0], [1, 200, 17], 2, 1, 64, 128),
    ([100], [150], 16, 1, 128, 256),                   # G = 16
    ([130], [300], 2, 2, 128, 32),                     # G = 1: chunks of whole row tiles
    ([260, 3, 700, 64], [1, 70, 1, 33], 8, 1, 128, 16),   # single tokens among chunks
    ([40], [19], 3, 1, 64, 384),
    ([150, 20], [1, 2], 128, 1, 64, 16),               # 128 query heads on one KV head
    ([150], [3], 65, 1, 128, 64),
    ([10], [40], 12, 1, 64, 16),
    ([5000], [2], 4, 1, 64, 16),
]


def check_attn(x, **kw):
    bt = x.batch(dk, **kw.pop("batch", {}))
    ws = workspace(bt, x.hq, x.hkv, x.d)
    o = torch.full((x.N, x.hq, x.d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((x.N, x.hq), 7.0, device="cuda")
    dk.dustin_paged_attn(bt, x.q, x.kc, x.vc, x.table, x.cu, x.kv_len, o, lse, ws=ws)
    assert dk.check(ws) == 0
    ro, rl, ra = O.paged_attn(to_bits(x.q), to_bits(x.kc), to_bits(x.vc), x.table_host, x.cu_host, x.kv)
    n = int(x.cu_host[-1])
    keys = [x.rows(b, g, x.kc) for b in range(x.B) for g in range(x.hkv) if x.kv[b]]
    assert_attended(o[:n], lse[:n], ro[:n], rl[:n], ra[:n], logit_error(x.q[:n], *keys), max(x.kv))
    assert bool((o[n:] == 7).all()) and bool((lse[n:] == 7).all())
    return o, lse


@pytest.mark.parametrize("ctx,new,hq,hkv,d,page", ATTN)
def test_attn_parity(ctx, new, hq, hkv, d, page):
    check_attn(Paged(ctx, new, hq, hkv, d, page, seed=sum(ctx) + hq, pad=sum(new) % 3))


@pytest.mark.parametrize("layout", ["token", "padded"])
def test_attn_strided_pools(layout):
    ref = check_attn(Paged([300, 97, 64], [4, 30, 1], 8, 2, 128, 32, seed=5))
    got = check_attn(Paged([300, 97, 64], [4, 30, 1], 8, 2, 128, 32, seed=5, layout=layout))
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])


@pytest.mark.parametrize("d,kl,vl", [(128, "head", "token"), (64, "token", "token"), (64, "padded", "head"), (128, "token", "padded")])
def test_attn_pools_of_different_layouts(d, kl, vl):
    x = Paged([300, 97, 64, 700], [4, 30, 1, 150], 8, 2, d, 32, seed=6)
    ref = check_attn(x)
    for name, layout in (("kc", kl), ("vc", vl)):
        pool = x._pool(layout)
        pool.copy_(getattr(x, name))
        setattr(x, name, pool)
    got = check_attn(x)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])


def test_attn_over_a_contiguous_cache():
    """A contiguous cache is a pool of one page a sequence."""
    B, hq, hkv, d, Lcap, kv, n = 3, 8, 2, 128, 384, [300, 7, 129], [1, 7, 60]
    kc, vc = (torch.full((B, hkv, Lcap, d), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for b in range(B):
        for t, s in ((kc, 1), (vc, 2)):
            t[b, :, :kv[b]] = normal(10 * b + s, hkv, kv[b], d)
    q, cu = normal(5, sum(n), hq, d, scale=2.0), np.concatenate([[0], np.cumsum(n)])
    o, lse = dk.dustin_paged_attn(dk.Batch(B, sum(n), max(n), 1), q, kc, vc, i32([[0], [1], [2]]), i32(cu), i32(kv))
    ro, rl, ra = O.paged_attn(to_bits(q), to_bits(kc), to_bits(vc), [[0], [1], [2]], cu, kv)
    assert_attended(o, lse, ro, rl, ra, logit_error(q, *[kc[b, :, :kv[b]] for b in range(B)]), max(kv))


@pytest.mark.parametrize("max_new", [1, 64])
def test_attn_without_any_token(max_new):
    """A captured batch with nothing in it: rows and flags are left alone."""
    x = Paged([0, 0, 0], [0, 0, 0], 8, 2, 128, 16, pad=5)
    for kv in ([0, 0, 0], [16, 0, 32]):
        ws = workspace(x.batch(dk, max_new=max_new), 8, 2, 128)
        o, lse = torch.full((5, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((5, 8), 7.0, device="cuda")
        dk.dustin_paged_attn(x.batch(dk, max_new=max_new), x.q, x.kc, x.vc, x.table, x.cu, i32(kv), o, lse, ws=ws)
        assert dk.check(ws) == 0 and bool((o == 7).all()) and bool((lse == 7).all())


def test_attn_without_lse():
    import ctypes
    x = Paged([100, 3000], [40, 2], 8, 2, 64, 32, seed=13)
    ref = dk.dustin_paged_attn(x.batch(dk), x.q, x.kc, x.vc, x.table, x.cu, x.kv_len)
    ws, o = workspace(x.batch(dk), 8, 2, 64), torch.empty_like(x.q)
    bt, bd = x.batch(dk).c(), dk.binding
    st = dk.lib().dustin_paged_attn(ctypes.byref(bt), 8, x.q.data_ptr(), bd.paged_view(x.kc), bd.paged_view(x.vc),
                                    x.table.data_ptr(), x.cu.data_ptr(), x.kv_len.data_ptr(), o.data_ptr(), None, ws.ptr,
                                    ws.nbytes, torch.cuda.current_stream().cuda_stream)
    assert st == 0 and dk.check(ws) == 0 and torch.equal(o, ref[0])


def test_attn_scores_that_rise_and_fall():
    """The largest scores come late, early, in steps far over the first ones', and
    in one row of a warp only: the reference maximum has to follow."""
    for d, new, page in ((64, 1, 16), (128, 6, 64), (128, 200, 128), (64, 90, 16)):
        x = Paged([1500], [new], 8, 1, d, page, seed=31)
        for at, f in ((40, 9.0), (300, 30.0), (301, 60.0), (900, 120.0), (1400, 3.0)):
            j = int(x.table_host[0, at // page])
            x.kc[j, 0, at % page] = (x.q[0, 3].float() * f / x.q[0, 3].float().norm()).to(torch.bfloat16)
        check_attn(x)
        x.q.mul_(0)          # and none at all
        check_attn(x)


def test_attn_many_requests_and_extreme_scores():
    """Ragged lengths over a large batch; scores far apart (up to about 150),
    so that the running maximum moves and most weights underflow."""
    rng = np.random.default_rng(0)
    x = Paged(rng.integers(0, 300, 90).tolist(), rng.integers(0, 6, 90).tolist(), 4, 2, 64, seed=9)
    x.q.mul_(8)
    check_attn(x)


@pytest.mark.parametrize("d", [64, 128])
def test_attn_many_short_units(d):
    rng = np.random.default_rng(d)
    x = Paged(rng.integers(0, 40, 260).tolist(), rng.integers(0, 3, 260).tolist(), 8, 8, d, seed=d)
    for _ in range(3):
        check_attn(x)


def test_attn_rows_before_the_first_position():
    """More query rows than cache rows: those before position 0 see nothing."""
    x = Paged([0, 0, 60], [3, 40, 5], 8, 2, 128, 16, seed=3)
    x.kv = [2, 25, 0]
    x.kv_len = i32(x.kv)
    o, lse = check_attn(x)
    assert bool((o[0] == 0).all()) and bool((o[3:18] == 0).all()) and bool((o[43:] == 0).all())
    assert bool(lse[43:].isneginf().all()) and not bool(lse[18:43].isinf().any())


def test_attn_flags():
    x = Paged([100, 50, 200], [3, 2, 40], 8, 2, 64, 16, seed=6)
    ref = check_attn(x)
    ws = workspace(x.batch(dk), 8, 2, 64)

    def run(bt=None, **o):
        a = dict(table=x.table, cu=x.cu, kv=x.kv_len)
        a.update(o)
        out = (torch.full_like(ref[0], 7.0), torch.full_like(ref[1], 7.0))
        dk.dustin_paged_attn(bt or x.batch(dk), x.q, x.kc, x.vc, a["table"], a["cu"], a["kv"], *out, ws=ws)
        return out, dk.check(ws)
    rows = [slice(0, 3), slice(3, 5), slice(5, 45)]

    ro, rl, ra = O.paged_attn(to_bits(x.q), to_bits(x.kc), to_bits(x.vc), x.table_host, x.cu_host, x.kv)
    keys = [x.rows(b, g, x.kc) for b in range(3) for g in range(2)]
    zerr = logit_error(x.q, *keys)

    def same(out, left):
        """The other requests within their bounds: where a request's tiles are cut,
        and so the order of its fp32 sums, depends on the whole batch."""
        for b, r in enumerate(rows):
            if b in left:
                assert all(bool((a[r] == 7).all()) for a in out), b
            else:
                assert_attended(out[0][r], out[1][r], ro[r], rl[r], ra[r], zerr, max(x.kv))
    for kv in (-1, x.width * 16 + 1, 2 ** 31 - 1):
        out, flags = run(kv=i32([x.kv[0], kv, x.kv[2]]))
        assert flags == dk.DEV_SEQLEN
        same(out, {1})
    out, flags = run(x.batch(dk, max_new=39))
    assert flags == dk.DEV_SEQLEN
    same(out, {2})
    for cu, left in (([0, 3, 2, 45], None), ([0, 3, 5, 46], {2}), ([-1, 3, 5, 45], {0}), ([0, 2 ** 31 - 1, 5, 45], {0, 1})):
        out, flags = run(cu=i32(cu))
        assert flags == dk.DEV_SEQLEN
        if left is not None:
            same(out, left)
    # table entries outside the pool: rows of zeros, in every needed position
    t = x.table_host.copy()
    t[0, 1], t[2, 0], t[2, pages_of(x.kv[2], 16) - 1] = x.n_pages, -1, 2 ** 31 - 1
    out, flags = run(table=i32(t))
    assert flags == dk.DEV_INDEX
    ro, rl, ra = O.paged_attn(to_bits(x.q), to_bits(x.kc), to_bits(x.vc), t, x.cu_host, x.kv)
    assert_attended(*out, ro, rl, ra, zerr, max(x.kv))


def test_attn_query_rows_that_are_not_finite():
    x = Paged([100, 300], [20, 3], 8, 2, 64, 32, seed=8)
    ref = check_attn(x)
    x.q[3, 2, 5], x.q[21, 7, 63], x.q[10, 0, 0] = NAN, math.inf, -math.inf
    o, lse = dk.dustin_paged_attn(x.batch(dk), x.q, x.kc, x.vc, x.table, x.cu, x.kv_len)
    bad = torch.zeros((x.N, 8), dtype=torch.bool, device="cuda")
    bad[3, 2] = bad[21, 7] = bad[10, 0] = True
    assert bool(o[bad].isnan().all()) and bool(lse[bad].isnan().all())
    assert torch.equal(o[~bad], ref[0][~bad]) and torch.equal(lse[~bad], ref[1][~bad])


def big_reference(x, b, g, t0, t1):
    """float64 (o, lse, sum p |v|) of rows t0..t1-1 of request b, KV head g."""
    G, n, kv = x.hq // x.hkv, x.new[b], x.kv[b]
    q = x.q[int(x.cu_host[b]) + t0:int(x.cu_host[b]) + t1, g * G:(g + 1) * G].reshape(-1, x.d)
    p = (kv - n + torch.arange(t0, t1, device="cuda")).repeat_interleave(G).view(-1, 1)
    k, v = x.rows(b, g, x.kc), x.rows(b, g, x.vc)
    return q, k, attend64(q, k, v, torch.arange(kv, device="cuda") <= p)


@pytest.mark.parametrize("ctx,new,hq,hkv,d,page", [
    ([6000], [1100], 16, 2, 128, 128), ([0], [3001], 8, 1, 64, 64), ([3000, 9000, 12000], [900, 1, 6], 8, 1, 128, 16),
    ([20000], [6], 64, 8, 128, 64), ([0, 500], [1500, 700], 4, 4, 128, 32), ([2000], [700], 14, 2, 64, 16)])
def test_attn_long(ctx, new, hq, hkv, d, page):
    """Requests whose tiles are shared among many CTAs, and chunks of many row tiles."""
    x = Paged(ctx, new, hq, hkv, d, page, seed=11)
    ws = workspace(x.batch(dk), hq, hkv, d)
    o, lse = dk.dustin_paged_attn(x.batch(dk), x.q, x.kc, x.vc, x.table, x.cu, x.kv_len, ws=ws)
    assert dk.check(ws) == 0
    G = hq // hkv
    for b in range(x.B):
        for g in range(hkv):
            for t0 in range(0, new[b], 512):
                t1 = min(new[b], t0 + 512)
                q, k, (ro, rl, ra) = big_reference(x, b, g, t0, t1)
                rows = slice(int(x.cu_host[b]) + t0, int(x.cu_host[b]) + t1)
                got_o, got_l = o[rows, g * G:(g + 1) * G].reshape(-1, d), lse[rows, g * G:(g + 1) * G].reshape(-1)
                assert_attended(got_o, got_l, ro.cpu().numpy(), rl.cpu().numpy(), ra.cpu().numpy(), logit_error(q, k),
                                x.kv[b])


def test_attn_pool_offsets_past_32_bits():
    """Pages whose elements lie past 2^31 (and 2^32) in the pool."""
    page, hkv, d = 256, 8, 128
    far = (1 << 32) // (page * hkv * d) + 5
    x = Paged([700], [3], 16, hkv, d, page, seed=12, far=far)
    assert int(x.table_host[0, :3].min()) * page * hkv * d > 1 << 32
    y = Paged([700], [3], 16, hkv, d, page, seed=12)
    a = dk.dustin_paged_attn(x.batch(dk), x.q, x.kc, x.vc, x.table, x.cu, x.kv_len)
    b = dk.dustin_paged_attn(y.batch(dk), y.q, y.kc, y.vc, y.table, y.cu, y.kv_len)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # and written there
    q, k, v = normal(1, 2, 16, d), normal(2, 2, hkv, d), normal(3, 2, hkv, d)
    last = x.n_pages * page - 1
    dk.dustin_norm_rope(dk.Rope(0), q, k, v, None, None, None, i32([0, 0]), i32([last, last - 1]), x.kc, x.vc)
    assert torch.equal(x.kc[-1, :, -1], k[0]) and torch.equal(x.vc[-1, :, -2], v[1])


def test_attn_matches_the_contiguous_operators():
    """The same rows in a contiguous cache, through windowed attention without a
    limit, give the same attention (each within its own bounds of float64)."""
    from _cache_cases import Block
    y = Block([250, 77], 5, 8, 2, 128, seed=4)
    x = Paged([250, 77], [5, 5], 8, 2, 128, 64, seed=4)
    x.q = y.q.reshape(x.N, 8, 128).contiguous()
    for b, L in enumerate(y.lens):
        for g in range(2):
            for pool, cache, block in ((x.kc, y.k, y.kb), (x.vc, y.v, y.vb)):
                rows = torch.cat([cache[b, g, :L], block[b, g]])
                for j in range(pages_of(L + 5, 64)):
                    part = rows[64 * j:64 * (j + 1)]
                    pool[int(x.table_host[b, j]), g, :part.shape[0]] = part
    p = dk.Params(2, y.cap, 4, 0, y.cap + 5, 0, y.cap + 5)
    o, lse = dk.dustin_window_attn(p, y.q, y.k, y.v, y.kb, y.vb, y.seq)
    got = check_attn(x)
    assert torch.allclose(lse.reshape(x.N, 8), got[1], atol=1e-4, rtol=0)
    assert torch.allclose(o.reshape(x.N, 8, 128).float(), got[0].float(), atol=2.0 ** -6, rtol=2.0 ** -6)


# ---------------------------------------------------------------- together


def test_large_batches_of_single_tokens():
    """More requests than CTAs, and every length from 0 on."""
    lens = list(range(0, 320))
    x = Paged(lens, [1] * 320, 4, 2, 64, 16, seed=40)
    ws = workspace(x.batch(dk), 4, 2, 64)
    o, lse = dk.dustin_paged_attn(x.batch(dk), x.q, x.kc, x.vc, x.table, x.cu, x.kv_len, ws=ws)
    assert dk.check(ws) == 0
    for b in range(0, 320, 7):
        for g in range(2):
            q, k, (ro, rl, ra) = big_reference(x, b, g, 0, 1)
            assert_attended(o[b, 2 * g:2 * g + 2], lse[b, 2 * g:2 * g + 2], ro.cpu().numpy(), rl.cpu().numpy(),
                            ra.cpu().numpy(), logit_error(q, k), x.kv[b])


def test_a_single_token_in_a_batch_that_allows_chunks():
    """The same requests in both shapes of the kernel (the batch's max_new chooses)."""
    x = Paged([0, 1, 500, 127, 128, 4000], [1] * 6, 16, 2, 128, 16, seed=41)
    for max_new in (1, 16, 17, 4096):
        check_attn(x, batch=dict(max_new=max_new)) if max_new > 1 else check_attn(x)


def test_deterministic():
    x = Paged([3000, 30, 0, 1000], [5, 1, 200, 64], 8, 2, 128, 16, seed=21)
    call = dk.PagedAttnCall(x.batch(dk), x.q, x.kc, x.vc, x.table, x.cu, x.kv_len)
    a = [t.clone() for t in call()]
    for _ in range(10):
        assert all(torch.equal(s, t) for s, t in zip(a, call()))


def test_graphs_follow_lengths_and_share_a_workspace():
    """One capture of map, rope and attention serves batches of other lengths; a
    second graph on the same workspace runs in turn with it."""
    B, hq, hkv, d, page, width, N, top = 3, 8, 2, 64, 16, 12, 64, 40
    n_pages = 30
    seq, new = i32([0, 0, 0]), i32([0, 0, 0])
    table, held, free, n_free = i32(np.zeros((B, width))), i32([0] * B), i32(range(n_pages)), i32([n_pages])
    kc, vc = (torch.full((n_pages, hkv, page, d), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, k, v = normal(1, N, hq, d, scale=2.0), normal(2, N, hkv, d), normal(3, N, hkv, d)
    w = (1 + normal(4, d, scale=0.2).float()).to(torch.bfloat16)
    inv = torch.tensor([1e4 ** (-2 * j / d) for j in range(d // 2)], device="cuda")
    bt = dk.Batch(B, N, top, width)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        ws = workspace(bt, hq, hkv, d)
        m = dk.PageMapCall(bt, page, seq, new, table, held, free, n_free, ws=ws)
        cu, kv, slot, pos = m._result
        r = dk.NormRopeCall(dk.Rope(d), q, k, v, w, w, inv, pos, slot, kc, vc, ws=ws)
        a = dk.PagedAttnCall(bt, r._result, kc, vc, table, cu, kv, ws=ws)
        for c in (m, r, a):
            c()
        side.synchronize()
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                for c in (m, r, a):
                    c()
            graphs.append(g)
    state = (table, held, free, n_free, kc, vc)
    first = [t.clone() for t in state]
    for lens, adds in (([0, 0, 0], [40, 3, 0]), ([40, 3, 0], [1, 6, 20]), ([41, 5, 20], [6, 6, 6]), ([0, 9, 0], [0, 1, 1])):
        seq.copy_(i32(lens))
        new.copy_(i32(adds))
        before = [t.clone() for t in state]
        outs = []
        for run in (lambda: [c() for c in (m, r, a)], graphs[0].replay, graphs[1].replay):
            for t, s in zip(state, before):
                t.copy_(s)
            for t in a._result:
                t.fill_(7.0)
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                run()
            torch.cuda.synchronize()
            outs.append([t.clone() for t in (*state, *m._result, r._result, *a._result)])
        for o in outs[1:]:
            assert all(torch.equal(torch.nan_to_num(x.float()), torch.nan_to_num(y.float())) for x, y in zip(outs[0], o))
    assert dk.check(ws) == 0
    assert not torch.equal(first[1], held)


def test_calls_on_other_streams():
    """Calls for a stream that is not the current one, with buffers of their own."""
    x = Paged([900, 30, 333], [4, 90, 1], 8, 2, 128, 16, seed=23)
    ref = [t.clone() for t in dk.dustin_paged_attn(x.batch(dk), x.q, x.kc, x.vc, x.table, x.cu, x.kv_len)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(side):
            torch.cuda._sleep(200000)
        o, lse = dk.dustin_paged_attn(x.batch(dk), x.q, x.kc, x.vc, x.table, x.cu, x.kv_len, stream=side)
        junk = [torch.full((1 << 20,), 3.0e38, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        del junk
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_refusals_on_the_gpu():
    x = Paged([100], [2], 4, 2, 64, 16, seed=22)
    a = (x.kc, x.vc, x.table, x.cu, x.kv_len)
    with pytest.raises(dk.DustinError):
        dk.dustin_paged_attn(x.batch(dk), x.q, *a, o=x.q)
    with pytest.raises(TypeError):
        dk.dustin_paged_attn(x.batch(dk), x.q.half(), *a)
    with pytest.raises(TypeError):
        dk.dustin_paged_attn(x.batch(dk), x.q, x.kc, x.vc, x.table.long(), x.cu, x.kv_len)
    with pytest.raises(dk.DustinError):
        dk.dustin_paged_attn(x.batch(dk), x.q, x.kc[:, :1].expand(-1, 2, -1, -1), *a[1:])
    with pytest.raises(dk.DustinError):
        dk.dustin_paged_attn(x.batch(dk), x.q, *a, ws=dk.binding.Workspace(300))


def test_serving_loop():
    """Requests come with prompts (one of them in chunks), decode draft blocks some
    of whose tokens are rejected, end and are replaced -- against a float64 model
    that keeps each request's rows in a list."""
    B, hq, hkv, d, page, width, n_pages, N, top = 4, 8, 2, 64, 16, 10, 34, 150, 100
    rng = np.random.default_rng(3)
    G, rot = hq // hkv, 32
    kc, vc = (torch.full((n_pages, hkv, page, d), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table, held = i32(np.zeros((B, width))), i32([0] * B)
    free, n_free = i32(rng.permutation(n_pages)), i32([n_pages])
    qw, kw = ((1 + normal(s, d, scale=0.2).float()).to(torch.bfloat16) for s in (1, 2))
    inv = np.float32([1e4 ** (-2 * j / rot) for j in range(rot // 2)])
    dinv, bt = torch.as_tensor(inv, device="cuda"), dk.Batch(B, N, top, width)
    ws = workspace(bt, hq, hkv, d)
    rows = [[] for _ in range(B)]        # per request, (k, v) of each cached position as the cache should hold them
    left = [90, 30, 130, 7]              # prompt tokens still to come
    for step in range(25):
        lens = [len(r) for r in rows]
        new = [min(left[b], top // 2) if left[b] else 1 + (step + b) % 6 for b in range(B)]
        for b in range(B):
            if lens[b] + new[b] > width * page or (step and rng.random() < 0.06):
                rows[b], lens[b], left[b] = [], 0, int(rng.integers(1, 100))
                new[b] = min(left[b], top // 2)
        if step == 9:
            new[2] = 0                   # an idle request
        x = normal(100 + step, N, hq + 2 * hkv, d)
        cu, kv, slot, pos = dk.dustin_page_map(bt, page, i32(lens), i32(new), table, held, free, n_free, ws=ws)
        q = dk.dustin_norm_rope(dk.Rope(rot, True), x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], qw, kw, dinv, pos, slot,
                                kc, vc, ws=ws)
        o, lse = dk.dustin_paged_attn(bt, q, kc, vc, table, cu, kv, ws=ws)
        flags = dk.check(ws)
        served = kv.tolist()
        assert flags in (0, dk.DEV_PAGES) and (flags != 0) == any(s == 0 and n > 0 for s, n in zip(served, new))
        xb, at, c = to_bits(x), slot.cpu().numpy(), cu.tolist()
        ref_k, size = O.norm_rope(xb[:, hq:hq + hkv], to_bits(kw), 1e-6, inv, pos.cpu().numpy(), rot, True)
        ref_q, qsize = O.norm_rope(xb[:, :hq], to_bits(qw), 1e-6, inv, pos.cpu().numpy(), rot, True)
        assert_rotated(q, ref_q, qsize)
        for b in range(B):
            if not served[b]:
                assert (at[c[b]:c[b + 1]] == -1).all() and bool((o[c[b]:c[b + 1]] == 0).all())
                continue
            assert served[b] == lens[b] + new[b]
            if not new[b]:
                continue
            s = at[c[b]:c[b + 1]]
            k = kc[s // page, :, s % page]
            assert_rotated(k, ref_k[c[b]:c[b + 1]], size[c[b]:c[b + 1]])
            assert torch.equal(vc[s // page, :, s % page], x[c[b]:c[b + 1], hq + hkv:])
            have = rows[b] + [(k[t], x[c[b] + t, hq + hkv:]) for t in range(new[b])]
            keys, vals = (torch.stack([r[i] for r in have], dim=1) for i in range(2))     # [hkv, kv, d]
            seen = torch.arange(len(have), device="cuda") <= torch.arange(lens[b], len(have), device="cuda").repeat_interleave(G).view(-1, 1)
            for g in range(hkv):
                pick = lambda t: t[c[b]:c[b + 1], g * G:(g + 1) * G].reshape(new[b] * G, -1)
                ro, rl, ra = attend64(pick(q), keys[g], vals[g], seen)
                assert_attended(pick(o), pick(lse).squeeze(-1), ro.cpu().numpy(), rl.cpu().numpy(), ra.cpu().numpy(),
                                logit_error(pick(q), keys[g]), len(have))
            keep = new[b] if left[b] else 1 + int(rng.integers(0, new[b]))
            rows[b] = have[:lens[b] + keep]
            left[b] = max(0, left[b] - new[b])
