"""The cache operators against float64: windowed attention with sinks,
shared-prefix attention, accumulated weights, eviction, and a serving loop of
them together."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU too
    pytest.skip("needs a GPU", allow_module_level=True)

import sparse_kv_verify_gb300 as dk  # noqa: E402
from oracle import cache_oracle as O  # noqa: E402
from synth import to_bits  # noqa: E402

from _cache_cases import (Block, normal, i32, logit_error, assert_attended, attend64,  # noqa: E402
                          assert_weights)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def params(x, sinks=0, window=0, k=None):
    return dk.Params(x.B, x.cap, x.T - 1, sinks, window, 0, k or max(1, sinks + window))


def absolute(bits):
    return bits & np.uint16(0x7FFF)


# ------------------------------------------------------------------ window

WINDOW = [
    # lens, T, hq, hkv, d, sinks, window
    ([200, 0, 1], 5, 8, 2, 64, 4, 32),
    ([300, 70], 1, 8, 1, 128, 4, 64),          # single tokens
    ([130, 129, 128, 127], 1, 2, 2, 64, 0, 1),  # a window of the query alone
    ([90, 3], 4, 4, 2, 64, 0, 0),               # rows that see nothing
    ([90, 3, 0], 4, 4, 2, 64, 5, 0),            # sinks alone
    ([90, 3], 6, 4, 2, 64, 2, 3),               # a window shorter than the block
    ([90, 250], 6, 14, 2, 64, 3, 1000),         # a window past the cache, G = 7
    ([100, 64, 65], 3, 16, 1, 128, 100, 20),    # sinks that meet the window, G = 16
    ([190], 5, 8, 8, 128, 64, 65),              # whole tiles of sinks and window
    ([257, 131], 64, 2, 1, 64, 7, 100),         # the largest block, 128 query rows
    ([257], 16, 16, 2, 128, 130, 63),           # 128 query rows at d = 128
    ([260, 40], 19, 3, 1, 64, 1, 129),          # 57 query rows
    ([400], 7, 8, 1, 128, 16, 256),             # 56 query rows at d = 128
    ([5], 2, 1, 1, 64, 2, 2),
    ([150, 20], 1, 128, 1, 64, 3, 70),          # 128 query heads on one KV head
    ([150], 1, 65, 1, 128, 0, 200),
]


def check_window(x, sinks, window, **kw):
    p = params(x, sinks, window)
    ws = dk.binding.Workspace(dk.cache_workspace_bytes(p, x.hq, x.hkv, x.d))
    o, lse = dk.dustin_window_attn(p, x.q, x.k, x.v, x.kb, x.vb, x.seq, ws=ws, **kw)
    assert dk.check(ws) == 0
    q, k, v, kb, vb = x.bits("q", "k", "v", "kb", "vb")
    ro, rl = O.window_attn(q, k, v, kb, vb, x.lens, sinks, window)
    ra, _ = O.window_attn(q, k, absolute(v), kb, absolute(vb), x.lens, sinks, window)
    assert_attended(o, lse, ro, rl, ra, logit_error(x.q, x.k, x.kb), min(max(x.lens), sinks + window) + x.T)
    return o, lse


@pytest.mark.parametrize("lens,T,hq,hkv,d,sinks,window", WINDOW)
def test_window_parity(lens, T, hq, hkv, d, sinks, window):
    x = Block(lens, T, hq, hkv, d, seed=T * 31 + window)
    # rows that no query of the block sees hold NaN
    for b, L in enumerate(lens):
        x.k[b, :, sinks:max(sinks, L - window + 1)] = float("nan")
        x.v[b, :, sinks:max(sinks, L - window + 1)] = float("nan")
    check_window(x, sinks, window)


def test_window_many_sequences_and_extreme_scores():
    """Ragged lengths over a large batch; scores far apart (up to about 150),
    so that the running maximum moves and most weights underflow."""
    rng = np.random.default_rng(0)
    x = Block(rng.integers(0, 400, 70).tolist(), 3, 4, 2, 64, seed=9)
    x.q.mul_(8)
    check_window(x, 2, 150)


@pytest.mark.parametrize("d", [64, 128])
def test_window_many_short_units_per_cta(d):
    """Units of one to three tiles, ten of them to a CTA: the query buffer is
    handed from unit to unit faster than the ring of tiles goes round."""
    rng = np.random.default_rng(d)
    x = Block(rng.integers(0, 130, 260).tolist(), 2, 8, 8, d, seed=d)
    for _ in range(3):
        check_window(x, 1, 60)
    pk, pv = prefix_of(40, 8, d)
    check_prefix(x, pk, pv, 40)


@pytest.mark.parametrize("layout", ["padded", "token_major"])
def test_window_strided_caches(layout):
    x = Block([300, 97, 64], 4, 8, 2, 128, seed=5)
    ref = check_window(x, 4, 100)
    if layout == "padded":
        big = torch.full((x.B, x.hkv + 1, x.cap + 3, x.d + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
        kv = []
        for t in (x.k, x.v):
            c = big.clone()
            c[:, :x.hkv, :x.cap, :x.d] = t
            kv.append(c[:, :x.hkv, :x.cap, :x.d])
    else:
        kv = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (x.k, x.v)]
    p = params(x, 4, 100)
    o, lse = dk.dustin_window_attn(p, x.q, kv[0], kv[1], x.kb, x.vb, x.seq)
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    # the two caches need not share a layout
    o, lse = dk.dustin_window_attn(p, x.q, x.k, kv[1], x.kb, x.vb, x.seq)
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_window_bad_length_flagged_and_taken_as_empty():
    x = Block([100, 0, 60], 2, 4, 2, 64, seed=6)
    ref = check_window(x, 2, 30)
    p = params(x, 2, 30)
    ws = dk.binding.Workspace(dk.cache_workspace_bytes(p, x.hq, x.hkv, x.d))
    for bad in (-1, x.cap + 1, 2 ** 31 - 1, -2 ** 31):
        o, lse = dk.dustin_window_attn(p, x.q, x.k, x.v, x.kb, x.vb, i32([100, bad, 60]), ws=ws)
        assert dk.check(ws) == dk.DEV_SEQLEN
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_window_offsets_past_32_bits():
    """The last sequence of a batch whose caches pass 2^31 elements."""
    B, hkv, d, cap = 3, 8, 128, 1 << 20
    c = torch.zeros((B, hkv, cap, d), dtype=torch.bfloat16, device="cuda")
    L = cap - 3
    rows = normal(1, hkv, 5 + 140, d)
    c[2, :, :5], c[2, :, L - 140:L] = rows[:, :5], rows[:, 5:]
    q, kb, vb = normal(2, B, 3, 16, d, scale=2.0), normal(3, B, hkv, 3, d), normal(4, B, hkv, 3, d)
    p = dk.Params(B, cap, 2, 5, 100, 0, 105)
    o, lse = dk.dustin_window_attn(p, q, c, c, kb, vb, i32([0, 0, L]))
    at = torch.cat([torch.arange(5), torch.arange(L - 140, L + 3)]).cuda()
    i = L + torch.arange(3, device="cuda").repeat_interleave(2).view(-1, 1)
    seen = (at <= i) & ((i - at < 100) | (at < 5))
    for g in range(hkv):
        keys = torch.cat([rows[g], kb[2, g]])
        ro, rl, ra = attend64(q[2, :, 2 * g:2 * g + 2].reshape(6, d), keys, torch.cat([rows[g], vb[2, g]]), seen)
        assert_attended(o[2, :, 2 * g:2 * g + 2].reshape(6, d), lse[2, :, 2 * g:2 * g + 2].reshape(6),
                        ro.cpu().numpy(), rl.cpu().numpy(), ra.cpu().numpy(), logit_error(q, keys), 108)


# ------------------------------------------------------------------ prefix

PREFIX = [
    # P, lens, T, hq, hkv, d
    (0, [70, 0, 3], 3, 4, 2, 64),
    (1, [0, 0], 1, 2, 2, 64),
    (63, [64, 1], 1, 8, 1, 128),
    (64, [10], 5, 8, 2, 64),
    (65, [0, 130, 5], 5, 14, 2, 64),
    (127, [3, 4, 5], 4, 4, 4, 128),
    (128, [128], 16, 8, 1, 128),                  # 128 query rows in one sequence
    (129, [33] * 9, 4, 8, 2, 64),                 # 144 rows share the prefix
    (200, [0, 40, 7, 300, 64] * 3, 5, 8, 2, 64),  # 300 rows
    (300, [20, 1] * 8, 3, 16, 1, 128),            # 768 rows
    (257, [5] * 11, 3, 3, 1, 64),                 # G = 3
    (190, [30, 20], 64, 2, 1, 64),                # the largest block
    (500, [17, 0, 90], 2, 5, 1, 128),             # G = 5: tiles that whole tokens do not fill
    (140, [30, 20, 0], 1, 128, 1, 64),            # one token fills a row tile
    (140, [30, 20, 0], 1, 65, 1, 128),
]


def prefix_of(P, hkv, d, seed=77, slack=45):
    pk, pv = normal(seed, 1, hkv, P + slack, d), normal(seed + 1, 1, hkv, P + slack, d)
    pk[:, :, P:], pv[:, :, P:] = float("nan"), float("nan")
    return pk, pv


def check_prefix(x, pk, pv, P, views=None):
    p = params(x)
    ws = dk.binding.Workspace(dk.cache_workspace_bytes(p, x.hq, x.hkv, x.d, prefix_cap=pk.shape[2]))
    vk, vv = views or (pk, pv)
    o, lse = dk.dustin_prefix_attn(p, x.q, vk, vv, i32([P]), x.k, x.v, x.kb, x.vb, x.seq, ws=ws)
    assert dk.check(ws) == 0
    q, k, v, kb, vb = x.bits("q", "k", "v", "kb", "vb")
    bk, bv = to_bits(pk), to_bits(pv)
    ro, rl = O.prefix_attn(q, bk, bv, P, k, v, kb, vb, x.lens)
    ra, _ = O.prefix_attn(q, bk, absolute(bv), P, k, absolute(v), kb, absolute(vb), x.lens)
    assert_attended(o, lse, ro, rl, ra, logit_error(x.q, x.k, x.kb, pk), P + max(x.lens) + x.T)
    return o, lse


@pytest.mark.parametrize("P,lens,T,hq,hkv,d", PREFIX)
def test_prefix_parity(P, lens, T, hq, hkv, d):
    x = Block(lens, T, hq, hkv, d, seed=P)
    check_prefix(x, *prefix_of(P, hkv, d), P)


def test_prefix_extreme_scores():
    """Scores up to about 150: the running maximum moves between tiles and
    between the prefix and the sequences' own rows."""
    x = Block([100, 0, 37, 400], 4, 8, 2, 128, seed=12)
    x.q.mul_(8)
    pk, pv = prefix_of(700, 2, 128)
    check_prefix(x, pk, pv, 700)


def test_prefix_long_against_torch():
    """A prefix of many tiles over more rows than one pair of row tiles."""
    P, B, T, hq, hkv, d = 20011, 24, 4, 32, 4, 128
    x = Block([50 * b % 333 for b in range(B)], T, hq, hkv, d, seed=3)
    pk, pv = prefix_of(P, hkv, d)
    o, lse = dk.dustin_prefix_attn(params(x), x.q, pk, pv, i32([P]), x.k, x.v, x.kb, x.vb, x.seq)
    G = hq // hkv
    for b in (0, 7, 23):
        L = x.lens[b]
        for g in (0, 3):
            keys = torch.cat([pk[0, g, :P], x.k[b, g, :L], x.kb[b, g]])
            vals = torch.cat([pv[0, g, :P], x.v[b, g, :L], x.vb[b, g]])
            t = torch.arange(T, device="cuda").repeat_interleave(G).view(-1, 1)
            seen = torch.arange(P + L + T, device="cuda") <= P + L + t
            pick = lambda a: a[b, :, g * G:(g + 1) * G].reshape(T * G, -1)
            ro, rl, ra = attend64(pick(x.q), keys, vals, seen)
            assert_attended(pick(o), pick(lse).squeeze(-1), ro.cpu().numpy(), rl.cpu().numpy(),
                            ra.cpu().numpy(), logit_error(x.q, keys), P + L + T)


def test_prefix_strided_views():
    x = Block([100, 0, 37], 3, 8, 2, 64, seed=13)
    pk, pv = prefix_of(150, 2, 64)
    ref = check_prefix(x, pk, pv, 150)
    big = torch.full((1, 4, pk.shape[2] + 9, 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    views = []
    for t in (pk, pv):
        c = big.clone()
        c[:, 1:3, 9:, 8:] = t
        views.append(c[:, 1:3, 9:, 8:])
    got = check_prefix(x, pk, pv, 150, views)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    got = check_prefix(x, pk, pv, 150, (pk.transpose(1, 2).contiguous().transpose(1, 2), pv))
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_prefix_bad_length_flagged_and_taken_as_zero():
    x = Block([50, 9], 2, 4, 2, 64, seed=14)
    pk, pv = prefix_of(100, 2, 64)
    ref = check_prefix(x, pk, pv, 0)
    p = params(x)
    ws = dk.binding.Workspace(dk.cache_workspace_bytes(p, x.hq, x.hkv, x.d, prefix_cap=pk.shape[2]))
    for bad in (-1, pk.shape[2] + 1, 2 ** 31 - 1):
        o, lse = dk.dustin_prefix_attn(p, x.q, pk, pv, i32([bad]), x.k, x.v, x.kb, x.vb, x.seq, ws=ws)
        assert dk.check(ws) == dk.DEV_SEQLEN
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_attention_without_lse():
    """The C calls take a null lse."""
    import ctypes
    x = Block([100, 7], 2, 4, 2, 64, seed=15)
    p = params(x, 2, 30)
    ref, _ = check_window(x, 2, 30)
    bd = dk.binding
    ws = bd.Workspace(dk.cache_workspace_bytes(p, x.hq, x.hkv, x.d, prefix_cap=70))
    o = torch.empty_like(x.q)
    s = torch.cuda.current_stream().cuda_stream
    st = dk.lib().dustin_window_attn(ctypes.byref(p.c()), x.hq, x.q.data_ptr(), bd.kv_view(x.k), bd.kv_view(x.v),
                                     x.kb.data_ptr(), x.vb.data_ptr(), x.seq.data_ptr(), o.data_ptr(), None,
                                     ws.ptr, ws.nbytes, s)
    assert st == 0 and torch.equal(o, ref)
    pk, pv = prefix_of(70 - 45, 2, 64)
    n = i32([25])
    ref, _ = check_prefix(x, pk, pv, 25)
    st = dk.lib().dustin_prefix_attn(ctypes.byref(p.c()), x.hq, x.q.data_ptr(), bd.kv_view(pk), bd.kv_view(pv), 70,
                                     n.data_ptr(), bd.kv_view(x.k), bd.kv_view(x.v), x.kb.data_ptr(),
                                     x.vb.data_ptr(), x.seq.data_ptr(), o.data_ptr(), None, ws.ptr, ws.nbytes, s)
    assert st == 0 and torch.equal(o, ref)


# -------------------------------------------------------------- accumulate

ACCUMULATE = [
    # lens, n_new, T, hq, hkv, d
    ([1, 64, 65], [1, 1, 1], 1, 2, 2, 64),
    ([200, 130, 5, 0], [5, 0, 3, 0], 5, 8, 2, 64),
    ([127, 128, 129], [2, 4, 3], 4, 8, 1, 128),
    ([300], [16], 16, 8, 1, 128),                    # 128 query rows
    ([90, 64], [64, 33], 64, 2, 1, 64),              # the largest block
    ([140, 77], [3, 1], 3, 14, 2, 64),               # G = 7
    ([1000, 513], [2, 2], 2, 16, 1, 128),            # G = 16
    ([4, 4], [4, 2], 4, 3, 3, 128),                  # every row new
]


def lse_of(x, n_new):
    """The log-sum-exp that the block's first n_new[b] rows have over the cache
    (later rows, which must not count, get a small one)."""
    lse = torch.full((x.B, x.T, x.hq), -20.0, device="cuda")
    G = x.hq // x.hkv
    for b, (L, n) in enumerate(zip(x.lens, n_new)):
        for g in range(x.hkv):
            z = torch.einsum("thd,nd->thn", x.q[b, :n, g * G:(g + 1) * G].double(), x.k[b, g, :L].double()) / math.sqrt(x.d)
            seen = torch.arange(L, device="cuda") <= L - n + torch.arange(n, device="cuda").view(-1, 1, 1)
            lse[b, :n, g * G:(g + 1) * G] = torch.logsumexp(z.masked_fill(~seen, -math.inf), dim=-1).float()
    return lse


def check_accumulate(x, n_new, lse, k=None):
    w = torch.rand((x.B, x.hkv, x.cap), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    pos = torch.full((x.B, x.hkv, x.cap), -7, dtype=torch.int32, device="cuda")
    for b, (L, n) in enumerate(zip(x.lens, n_new)):
        w[b, :, L - n:L] = float("nan")       # new rows: what they held is not read
    w0, p0 = w.cpu().numpy(), pos.cpu().numpy()
    seen = [L + 11 * b for b, L in enumerate(x.lens)]
    p = params(x)
    ws = dk.binding.Workspace(dk.cache_workspace_bytes(p))
    dk.dustin_accumulate(p, x.q, lse, x.k if k is None else k, i32(n_new), x.seq, i32(seen), w, pos, ws=ws)
    assert dk.check(ws) == 0
    q, kb = x.bits("q", "k")
    rw, rp = O.accumulate(q, lse.cpu().numpy(), kb, n_new, x.lens, seen, w0, p0)
    assert np.array_equal(pos.cpu().numpy(), rp)
    assert_weights(w, rw, np.nan_to_num(w0), logit_error(x.q, x.k), x.T * x.hq // x.hkv)
    for b, L in enumerate(x.lens):
        assert np.array_equal(w[b, :, L:].cpu().numpy(), w0[b, :, L:])
    return w, pos


@pytest.mark.parametrize("lens,n_new,T,hq,hkv,d", ACCUMULATE)
def test_accumulate_parity(lens, n_new, T, hq, hkv, d):
    x = Block(lens, T, hq, hkv, d, seed=T, slack=5)
    check_accumulate(x, n_new, lse_of(x, n_new))


def test_accumulate_empty_rows_and_strides():
    """Rows whose lse is -inf add nothing; padded and token-major caches."""
    n_new = [3, 2]
    x = Block([150, 70], 3, 4, 2, 64, seed=4)
    lse = lse_of(x, n_new)
    lse[0, 1, :] = -math.inf
    ref = check_accumulate(x, n_new, lse)
    c = torch.full((2, 3, x.cap + 2, 80), float("nan"), dtype=torch.bfloat16, device="cuda")
    c[:, :2, :x.cap, :64] = x.k
    got = check_accumulate(x, n_new, lse, k=c[:, :2, :x.cap, :64])
    assert torch.equal(got[0], ref[0])
    got = check_accumulate(x, n_new, lse, k=x.k.transpose(1, 2).contiguous().transpose(1, 2))
    assert torch.equal(got[0], ref[0])


def test_accumulate_bad_lengths_flagged_and_untouched():
    x = Block([100, 60, 50], 2, 4, 2, 64, seed=7)
    w = torch.ones((3, 2, x.cap), device="cuda")
    pos = torch.zeros((3, 2, x.cap), dtype=torch.int32, device="cuda")
    p = params(x)
    ws = dk.binding.Workspace(dk.cache_workspace_bytes(p))
    lse = torch.zeros((3, 2, 4), device="cuda")
    for n_new, lens, seen in [([3, 0, 0], [100, 60, 50], [100, 60, 50]), ([-1, 0, 0], [100, 60, 50], [100, 60, 50]),
                              ([2, 0, 0], [1, 60, 50], [100, 60, 50]), ([1, 0, 0], [x.cap + 1, 60, 50], [2 ** 30] * 3),
                              ([1, 0, 0], [-5, 60, 50], [100, 60, 50]), ([1, 0, 0], [100, 60, 50], [99, 60, 50])]:
        dk.dustin_accumulate(p, x.q, lse, x.k, i32(n_new), i32(lens), i32(seen), w, pos, ws=ws)
        assert dk.check(ws) == dk.DEV_APPEND, (n_new, lens, seen)
        assert bool((w == 1).all()) and bool((pos == 0).all())


# ------------------------------------------------------------------- evict

EVICT = [
    # lens, k, sinks, window, hkv, d, layers
    ([130, 128, 100, 0], 128, 4, 16, 2, 64, 1),
    ([1000, 999, 65], 64, 0, 0, 2, 128, 1),
    ([700, 701], 300, 3, 65, 1, 64, 3),
    ([5000], 1023, 16, 256, 4, 128, 2),
    ([513, 512, 514, 1025], 512, 0, 512, 1, 64, 1),   # the window is the budget
    ([40, 41], 1, 0, 0, 1, 64, 1),
    ([40, 41], 1, 1, 0, 1, 64, 1),
    ([20000, 9000], 4096, 16, 100, 2, 64, 1),
    ([300] * 40, 200, 2, 30, 4, 64, 16),
    ([9000 - 7 * b for b in range(10)], 500, 4, 64, 4, 64, 1),   # two CTAs per unit
    ([410000, 7000], 5000, 16, 100, 1, 64, 1),                   # keys past a CTA's shared memory
]


def evict_inputs(lens, hkv, d, layers, seed=0, ties=False, scatter=True):
    B, cap = len(lens), max(lens) + 9
    g = torch.Generator("cuda").manual_seed(seed)
    ks = [normal(seed + 2 * l, B, hkv, cap, d) for l in range(layers)]
    vs = [normal(seed + 2 * l + 1, B, hkv, cap, d) for l in range(layers)]
    w = [torch.rand((B, hkv, cap), device="cuda", generator=g) ** 8 for _ in range(layers)]
    if ties:
        w = [torch.floor(x * 4) for x in w]
    pos = [torch.rand((B, hkv, 2 * cap), device="cuda", generator=g).argsort(-1)[..., :cap].to(torch.int32).contiguous()
           for _ in range(layers)]
    if not scatter:
        pos = [torch.arange(cap, device="cuda", dtype=torch.int32).expand(B, hkv, cap).contiguous() for _ in pos]
    seen = i32([2 * cap] * B) if scatter else i32(lens)
    return ks, vs, w, pos, seen


def check_evict(lens, k, sinks, window, ks, vs, w, pos, seen):
    p = dk.Params(len(lens), ks[0].shape[2], 0, sinks, window, 0, k)
    before = [(to_bits(a), to_bits(b), c.cpu().numpy(), e.cpu().numpy()) for a, b, c, e in zip(ks, vs, w, pos)]
    seq = i32(lens)
    ws = dk.binding.Workspace(dk.cache_workspace_bytes(p, hkv=ks[0].shape[1], n_layers=len(ks)))
    dk.dustin_evict(p, ks, vs, w, pos, seen, seq, ws=ws)
    flags = dk.check(ws)
    for l, old in enumerate(before):
        ref = O.evict(*old, seen.cpu().numpy(), np.asarray(lens), k, sinks, window)
        got = (to_bits(ks[l]), to_bits(vs[l]), w[l].cpu().numpy(), pos[l].cpu().numpy())
        for name, a, r in zip(("k", "v", "weight", "pos"), got, ref):
            assert np.array_equal(a, r, equal_nan=a.dtype.kind == "f"), (l, name)
    assert seq.tolist() == [min(n, k) for n in lens]
    return flags


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("lens,k,sinks,window,hkv,d,layers", EVICT)
def test_evict_bit_exact(lens, k, sinks, window, hkv, d, layers, ties):
    x = evict_inputs(lens, hkv, d, layers, seed=k + ties, ties=ties, scatter=layers > 1 or ties)
    assert check_evict(lens, k, sinks, window, *x) == 0


def test_evict_narrow_and_odd_weights():
    """All weights equal; weights one step apart; infinities; -0.0; NaN and
    negative weights, which rank as 0 and are flagged."""
    lens = [700, 600]
    ks, vs, w, pos, seen = evict_inputs(lens, 2, 64, 1, seed=3)
    assert check_evict(lens, 200, 2, 20, ks, vs, [torch.full_like(w[0], 0.25)], pos, seen) == 0
    step = (torch.rand_like(w[0]) * 300).to(torch.int32) + 0x3F800000
    assert check_evict(lens, 200, 2, 20, ks, vs, [step.view(torch.float32)], pos, seen) == 0
    odd = w[0].clone()
    odd[:, :, ::7], odd[:, :, 3::11] = math.inf, -0.0
    assert check_evict(lens, 200, 2, 20, ks, vs, [odd], pos, seen) == 0
    odd = w[0].clone()
    odd[0, 1, 5], odd[1, 0, 300] = math.nan, -1.0
    assert check_evict(lens, 200, 2, 20, ks, vs, [odd], pos, seen) == dk.DEV_NAN


def test_evict_more_protected_than_budget():
    """Repeated positions can protect more rows than the budget: the lower stay."""
    lens = [300, 299]
    ks, vs, w, pos, seen = evict_inputs(lens, 2, 64, 1, seed=8)
    pos[0].fill_(3)
    pos[0][:, :, ::2] = 100
    assert check_evict(lens, 70, 10, 5, ks, vs, w, pos, seen) == 0


def test_evict_strided_caches():
    lens = [400, 100, 333]
    ks, vs, w, pos, seen = evict_inputs(lens, 2, 128, 2, seed=9)
    big = torch.zeros((3, 3, ks[0].shape[2] + 2, 136), dtype=torch.bfloat16, device="cuda")
    views = []
    for t in (*ks, *vs):
        c = big.clone()
        c[:, :2, :-2, :128] = t
        views.append(c[:, :2, :-2, :128])
    assert check_evict(lens, 150, 4, 30, views[:2], views[2:], w, pos, seen) == 0
    major = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (ks[0], vs[0])]
    assert check_evict(lens, 150, 4, 30, major[:1], major[1:], w[:1], pos[:1], seen) == 0


def test_evict_bad_length_flagged_and_untouched():
    lens = [300, 200]
    ks, vs, w, pos, seen = evict_inputs(lens, 1, 64, 1, seed=10)
    p = dk.Params(2, ks[0].shape[2], 0, 2, 10, 0, 50)
    ws = dk.binding.Workspace(dk.cache_workspace_bytes(p, hkv=1, n_layers=1))
    for bad in (-1, ks[0].shape[2] + 1):
        seq, k0, w0 = i32([bad, 40]), ks[0].clone(), w[0].clone()
        dk.dustin_evict(p, ks, vs, w, pos, seen, seq, ws=ws)
        assert dk.check(ws) == dk.DEV_SEQLEN
        assert seq.tolist() == [bad, 40] and torch.equal(k0, ks[0]) and torch.equal(w0, w[0])


@pytest.mark.parametrize("lens, d", [([40, 9], 64), ([3000, 5], 128)])   # whole units; units split and merged
@pytest.mark.parametrize("prefix", [False, True])
def test_query_that_is_not_finite_shows(lens, d, prefix):
    """NaN in one query row comes out in that row, never as an empty one, and
    every other row keeps its bits."""
    x = Block(lens, 3, 8, 2, d, seed=24)
    p = params(x, 0, 0 if prefix else 2500)
    pk, pv = prefix_of(300, 2, d)
    def run():
        if prefix:
            return dk.dustin_prefix_attn(p, x.q, pk, pv, i32([300]), x.k, x.v, x.kb, x.vb, x.seq)
        return dk.dustin_window_attn(p, x.q, x.k, x.v, x.kb, x.vb, x.seq)
    o0, l0 = run()
    x.q[1, 1, 3, 5] = float("nan")
    o1, l1 = run()
    assert o1[1, 1, 3].isnan().all() and l1[1, 1, 3].isnan()
    o1[1, 1, 3], l1[1, 1, 3] = o0[1, 1, 3], l0[1, 1, 3]
    assert torch.equal(o1, o0) and torch.equal(l1, l0)


# ------------------------------------------------ streams, graphs, all together


def test_graph_replay_on_side_stream_follows_lengths():
    """All four captured into one graph on a side stream: replays read the
    lengths of their own time; a second graph shares the workspace in turn."""
    x = Block([300, 300], 3, 8, 2, 64, seed=20)
    pk, pv = prefix_of(100, 2, 64)
    n = i32([100])
    p = params(x, 4, 60, k=128)
    lse0 = lse_of(x, [1, 2])
    weight = torch.rand((2, 2, x.cap), device="cuda")
    pos = torch.arange(x.cap, dtype=torch.int32, device="cuda").expand(2, 2, x.cap).contiguous()
    seq_e, seen = i32([300, 120]), i32([300, 300])
    ke, ve = x.k.clone(), x.v.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = dk.binding.Workspace(dk.cache_workspace_bytes(p, x.hq, 2, 64, 1, pk.shape[2]))
    torch.cuda.synchronize()
    calls = [dk.WindowCall(p, x.q, x.k, x.v, x.kb, x.vb, x.seq, ws=ws),
             dk.PrefixCall(p, x.q, pk, pv, n, x.k, x.v, x.kb, x.vb, x.seq, ws=ws),
             dk.AccumulateCall(p, x.q, lse0, x.k, i32([1, 2]), x.seq, seen, weight, pos, ws=ws),
             dk.EvictCall(p, [ke], [ve], [weight], [pos], seen, seq_e, ws=ws)]
    state = [t.clone() for t in (weight, pos, ke, ve, seq_e)]

    def restore():
        for t, s in zip((weight, pos, ke, ve, seq_e), state):
            t.copy_(s)

    def snapshot():
        torch.cuda.synchronize()
        return [t.clone() for t in (*calls[0]._result, *calls[1]._result, weight, pos, ke, ve, seq_e)]

    graphs = []
    with torch.cuda.stream(side):
        for c in calls:       # first launches outside a capture
            c()
        side.synchronize()
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                for c in calls:
                    c()
            graphs.append(g)
    for lens, P in (([300, 120], 100), ([40, 2], 7), ([2, 299], 0)):
        x.seq.copy_(i32(lens))
        n.fill_(P)
        restore()
        torch.cuda.synchronize()
        for c in calls:
            c()
        want = snapshot()
        for g in graphs:
            restore()
            for t in (*calls[0]._result, *calls[1]._result):
                t.fill_(7.0)
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                g.replay()
            for a, b in zip(snapshot(), want):
                assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))
    assert dk.check(ws) == 0


def test_explicit_stream_owns_its_workspace():
    """A call on a stream that is not the current one, with a workspace of its
    own that is freed at once and other work that would take its memory."""
    x = Block([900, 30, 333], 4, 8, 2, 128, seed=23)
    p = params(x, 4, 600)
    ref = [t.clone() for t in dk.dustin_window_attn(p, x.q, x.k, x.v, x.kb, x.vb, x.seq)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(side):
            torch.cuda._sleep(200000)
        o, lse = dk.dustin_window_attn(p, x.q, x.k, x.v, x.kb, x.vb, x.seq, stream=side)
        junk = [torch.full((1 << 20,), 3.0e38, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        del junk
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("how", ["current", "explicit"])
def test_own_buffers_belong_to_the_stream_that_uses_them(how, monkeypatch):
    """What a call allocated is recorded on another stream that it runs on, the
    current one or a given one; on its own stream nothing is."""
    x = Block([70, 30], 2, 8, 2, 64, seed=25)
    p = params(x, 4, 60)
    side = torch.cuda.Stream()
    call = dk.WindowCall(p, x.q, x.k, x.v, x.kb, x.vb, x.seq)
    own = {t.data_ptr() for t in (call.ws.buf, *call._result)}
    torch.cuda.synchronize()
    seen = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.append((t.data_ptr(), s.cuda_stream)))
    ref = [t.clone() for t in call()]
    assert not seen
    side.wait_stream(torch.cuda.current_stream())
    if how == "current":
        with torch.cuda.stream(side):
            call()
    else:
        call(side)
    side.synchronize()
    assert sorted(seen) == sorted((a, side.cuda_stream) for a in own)
    assert all(torch.equal(a, b) for a, b in zip(call._result, ref))
    # built for a stream: its buffers are that stream's, and a user's are left alone
    seen.clear()
    dk.dustin_window_attn(p, x.q, x.k, x.v, x.kb, x.vb, x.seq, stream=side)
    o, lse = (torch.empty_like(t) for t in ref)
    dk.dustin_window_attn(p, x.q, x.k, x.v, x.kb, x.vb, x.seq, o, lse, ws=call.ws)
    torch.cuda.synchronize()
    assert not seen and torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_deterministic():
    x = Block([700, 30, 333], 5, 8, 2, 128, seed=21)
    pk, pv = prefix_of(900, 2, 128)
    p = params(x, 4, 200)
    for call in (dk.WindowCall(p, x.q, x.k, x.v, x.kb, x.vb, x.seq),
                 dk.PrefixCall(p, x.q, pk, pv, i32([900]), x.k, x.v, x.kb, x.vb, x.seq)):
        a = [t.clone() for t in call()]
        for _ in range(5):
            assert all(torch.equal(s, t) for s, t in zip(a, call()))


def test_call_refuses_a_wrong_workspace_and_in_place_output():
    x = Block([100], 2, 4, 2, 64, seed=22)
    p = params(x, 2, 30)
    with pytest.raises(dk.DustinError):
        dk.dustin_window_attn(p, x.q, x.k, x.v, x.kb, x.vb, x.seq, o=x.q)
    with pytest.raises(TypeError):
        dk.dustin_window_attn(p, x.q.half(), x.k, x.v, x.kb, x.vb, x.seq)
    with pytest.raises(TypeError):
        dk.dustin_window_attn(p, x.q, x.k, x.v, x.kb, x.vb, x.seq.long())
    with pytest.raises(ValueError):
        dk.dustin_window_attn(p, x.q, x.k[..., ::2], x.v, x.kb, x.vb, x.seq)
    with pytest.raises(dk.DustinError):
        dk.dustin_window_attn(p, x.q, x.k[:, :1].expand(1, 2, x.cap, 64), x.v, x.kb, x.vb, x.seq)


def test_serving_loop():
    """A batch behind a shared prompt decodes with bounded own caches: attend,
    accept, append, accumulate, evict -- against a float64 model of the whole."""
    B, T, hq, hkv, d, P, k, sinks, window = 3, 4, 8, 2, 64, 150, 48, 3, 16
    cap, G = 64, hq // hkv
    p = dk.Params(B, cap, T - 1, sinks, window, 0, k)
    pk, pv = prefix_of(P, hkv, d)
    n = i32([P])
    ks, vs = (torch.full((B, hkv, cap, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    weight = torch.full((B, hkv, cap), float("nan"), device="cuda")
    pos = torch.zeros((B, hkv, cap), dtype=torch.int32, device="cuda")
    seq, seen = i32([0] * B), i32([0] * B)
    ws = dk.binding.Workspace(max(dk.cache_workspace_bytes(p, hq, hkv, d, 1, pk.shape[2]), dk.workspace_bytes(p)))
    for step in range(30):
        s = 1000 * step
        q, kb, vb = normal(s, B, T, hq, d, scale=2.0), normal(s + 1, B, hkv, T, d), normal(s + 2, B, hkv, T, d)
        lens = seq.tolist()
        o, lse = dk.dustin_prefix_attn(p, q, pk, pv, n, ks, vs, kb, vb, seq, ws=ws)
        acc = [1 + (step + 2 * b) % T for b in range(B)]
        for b in range(B):
            L = lens[b]
            for g in range(hkv):
                keys, vals = (torch.cat([x[0, g, :P], y[b, g, :L], z[b, g]]) for x, y, z in ((pk, ks, kb), (pv, vs, vb)))
                t = torch.arange(T, device="cuda").repeat_interleave(G).view(-1, 1)
                mask = torch.arange(P + L + T, device="cuda") <= P + L + t
                pick = lambda a: a[b, :, g * G:(g + 1) * G].reshape(T * G, -1)
                ro, rl, ra = attend64(pick(q), keys, vals, mask)
                assert_attended(pick(o), pick(lse).squeeze(-1), ro.cpu().numpy(), rl.cpu().numpy(),
                                ra.cpu().numpy(), logit_error(q, keys), P + L + T)
        dk.dustin_kv_append(p, [ks], [vs], [kb], [vb], i32(acc), seq, ws=ws)
        seen += i32(acc)
        w0 = weight.cpu().numpy()
        dk.dustin_accumulate(p, q, lse, ks, i32(acc), seq, seen, weight, pos, ws=ws)
        rw, _ = O.accumulate(to_bits(q), lse.cpu().numpy(), to_bits(ks), acc, seq.tolist(), seen.tolist(), w0,
                             np.zeros((B, hkv, cap), np.int32))
        for b, L in enumerate(seq.tolist()):
            assert_weights(weight[b, :, :L], rw[b, :, :L], np.nan_to_num(w0[b, :, :L]), logit_error(q, ks), T * G)
        before = (to_bits(ks), to_bits(vs), weight.cpu().numpy(), pos.cpu().numpy())
        lens = seq.tolist()
        dk.dustin_evict(p, [ks], [vs], [weight], [pos], seen, seq, ws=ws)
        ref = O.evict(*before, seen.tolist(), np.asarray(lens), k, sinks, window)
        for a, r in zip((to_bits(ks), to_bits(vs), weight.cpu().numpy(), pos.cpu().numpy(), seq.cpu().numpy()), ref):
            assert np.array_equal(a, r, equal_nan=a.dtype.kind == "f")
        # each unit holds distinct positions, the sinks and the recent window among them
        for b, L in enumerate(seq.tolist()):
            S = int(seen[b])
            for g in range(hkv):
                held = pos[b, g, :L].tolist()
                assert len(set(held)) == L == min(S, k)
                assert set(range(min(sinks, S))) <= set(held) and set(range(max(0, S - window), S)) <= set(held)
    assert dk.check(ws) == 0
    assert seq.tolist() == [k] * B
