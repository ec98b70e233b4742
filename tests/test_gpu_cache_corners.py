"""Corners of the cache operators."""
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

from _cache_cases import Block, assert_attended, attend64, i32, logit_error, normal  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def params(x, sinks=0, window=0):
    return dk.Params(x.B, x.cap, x.T - 1, sinks, window, 0, max(1, sinks + window))


# ------------------------------------------------------- infinite queries

INFINITE = [
    # lens, T, hq, hkv, d, sinks, window
    ([40, 9], 1, 8, 2, 64, 0, 1),           # each query sees its own position alone
    ([40, 9], 1, 8, 2, 128, 0, 1),
    ([40, 9], 2, 8, 2, 64, 3, 20),
    ([3000, 5], 3, 8, 2, 128, 0, 2500),     # units split over CTAs and merged
    ([200, 90], 9, 16, 2, 64, 4, 60),       # 72 query rows
    ([40, 0], 2, 8, 2, 64, 2, 0),           # sinks alone, of the block itself in an empty cache
]


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("lens,T,hq,hkv,d,sinks,window", INFINITE)
def test_window_query_with_an_infinite_element_gives_nan(lens, T, hq, hkv, d, sinks, window, sign):
    """Every score of the row is an infinity of one sign: 0 / 0 of the softmax,
    never the 0 and -inf of a row without keys.  Other rows keep their bits."""
    x = Block(lens, T, hq, hkv, d, seed=31)
    x.k[..., 5] = x.k[..., 5].abs() + 0.125
    x.kb[..., 5] = x.kb[..., 5].abs() + 0.125
    p = params(x, sinks, window)
    o0, l0 = dk.dustin_window_attn(p, x.q, x.k, x.v, x.kb, x.vb, x.seq)
    x.q[1, T - 1, 3, 5] = sign * math.inf
    o1, l1 = dk.dustin_window_attn(p, x.q, x.k, x.v, x.kb, x.vb, x.seq)
    assert o1[1, T - 1, 3].isnan().all() and l1[1, T - 1, 3].isnan()
    o1[1, T - 1, 3], l1[1, T - 1, 3] = o0[1, T - 1, 3], l0[1, T - 1, 3]
    assert torch.equal(o1, o0) and torch.equal(l1, l0)


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("P,lens,T,hq,hkv,d", [(0, [0, 0], 1, 2, 2, 64), (300, [40, 9], 3, 8, 2, 64),
                                               (700, [900, 0], 2, 8, 2, 128)])
def test_prefix_query_with_an_infinite_element_gives_nan(P, lens, T, hq, hkv, d, sign):
    x = Block(lens, T, hq, hkv, d, seed=32)
    pk, pv = normal(7, 1, hkv, P + 5, d), normal(8, 1, hkv, P + 5, d)
    for t in (x.k, x.kb, pk):
        t[..., 5] = t[..., 5].abs() + 0.125
    p, n = params(x), i32([P])
    o0, l0 = dk.dustin_prefix_attn(p, x.q, pk, pv, n, x.k, x.v, x.kb, x.vb, x.seq)
    x.q[0, T - 1, 1, 5] = sign * math.inf
    o1, l1 = dk.dustin_prefix_attn(p, x.q, pk, pv, n, x.k, x.v, x.kb, x.vb, x.seq)
    assert o1[0, T - 1, 1].isnan().all() and l1[0, T - 1, 1].isnan()
    o1[0, T - 1, 1], l1[0, T - 1, 1] = o0[0, T - 1, 1], l0[0, T - 1, 1]
    assert torch.equal(o1, o0) and torch.equal(l1, l0)


def test_infinite_query_that_sees_nothing_is_an_empty_row():
    x = Block([40, 9], 2, 4, 2, 64, seed=33)
    x.q[0, 0, 0, 5] = -math.inf
    o, lse = dk.dustin_window_attn(params(x), x.q, x.k, x.v, x.kb, x.vb, x.seq)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())


# ------------------------------------------- block rows that nobody sees


@pytest.mark.parametrize("lens,T,hq,hkv,d,sinks", [([90, 3, 0], 4, 4, 2, 64, 5), ([90, 3, 0], 4, 4, 2, 128, 0),
                                                   ([90, 60, 1], 9, 16, 2, 64, 64)])
def test_without_a_window_unseen_block_rows_may_hold_anything(lens, T, hq, hkv, d, sinks):
    """With a window of 0 a query sees sinks alone, not even its own position:
    block rows at or beyond the sinks are no query's."""
    x = Block(lens, T, hq, hkv, d, seed=34)
    p = params(x, sinks, 0)
    o0, l0 = dk.dustin_window_attn(p, x.q, x.k, x.v, x.kb, x.vb, x.seq)
    for b, L in enumerate(lens):
        x.kb[b, :, max(0, sinks - L):] = float("nan")
        x.vb[b, :, max(0, sinks - L):] = float("nan")
    o1, l1 = dk.dustin_window_attn(p, x.q, x.k, x.v, x.kb, x.vb, x.seq)
    assert torch.equal(o1, o0) and torch.equal(l1, l0)


# ------------------------------------------------------- another stream


@pytest.mark.parametrize("how", ["current", "explicit"])
def test_call_on_another_stream_waits_for_its_own_buffers(how):
    """What a call allocates is its home stream's: the workspace is initialised
    there, and the memory may have been another tensor's that work there still
    uses.  On another stream the call comes after that."""
    x = Block([70, 30], 2, 8, 2, 64, seed=35)
    p = params(x, 4, 60)
    ref = [t.clone() for t in dk.dustin_window_attn(p, x.q, x.k, x.v, x.kb, x.vb, x.seq)]
    home, side = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(home):   # (memory of that stream, so that nothing is allocated behind the delay)
        dk.WindowCall(p, x.q, x.k, x.v, x.kb, x.vb, x.seq)
    torch.cuda.synchronize()
    with torch.cuda.stream(home):
        torch.cuda._sleep(400_000_000)
        call = dk.WindowCall(p, x.q, x.k, x.v, x.kb, x.vb, x.seq)
    assert not home.query()
    if how == "current":
        with torch.cuda.stream(side):
            call()
    else:
        call(side)
    side.synchronize()
    assert home.query()
    assert all(torch.equal(a, b) for a, b in zip(call._result, ref))
    assert dk.check(call.ws) == 0


# --------------------------------------- lengths far from what a launch is planned for


def best_us(call):
    """The shortest time of a call among others, in us."""
    times = []
    for _ in range(30):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(10):
            call()
        b.record()
        b.synchronize()
        times.append(100 * a.elapsed_time(b))
    return min(times)


@pytest.mark.parametrize("prefix", [False, True])
def test_one_long_sequence_among_short_ones_is_shared_among_the_sms(prefix):
    """As many rows in all, most of them one sequence's or spread evenly, for a
    batch with one unit per CTA: a long unit left to one CTA takes three to
    seven times as long, so a factor of 2.5 tells."""
    B = torch.cuda.get_device_properties(0).multi_processor_count * 2 // 8
    cap = 8192
    q, k, v = normal(1, B, 1, 64, 128), normal(2, B, 8, cap, 128), normal(3, B, 8, cap, 128)
    kb, vb = normal(4, B, 8, 1, 128), normal(5, B, 8, 1, 128)
    pk, pv = normal(6, 1, 8, 64, 128), normal(7, 1, 8, 64, 128)
    seq = i32([64] * B)
    p = dk.Params(B, cap, 0, 0, cap, 0, cap)
    call = (dk.PrefixCall(p, q, pk, pv, i32([64]), k, v, kb, vb, seq) if prefix
            else dk.WindowCall(p, q, k, v, kb, vb, seq))

    def best(lens):
        seq.copy_(i32(lens))
        return best_us(call)
    long = [64] * (B - 1) + [cap]
    even = best([sum(long) // B] * B)
    assert best(long) < 2.5 * even
    o, lse = (t.clone() for t in call())
    assert bool(o.isfinite().all()) and bool(lse.isfinite().all()) and dk.check(call.ws) == 0


def test_short_prefix_in_a_large_cache_does_not_wait_for_its_own_parts():
    """The launch is planned by capacities.  A large prefix cache must not leave
    the own parts so few SMs that, behind a short prefix, the call takes two and
    a half times as long as with a small cache."""
    B, rows = 4, 512
    q, k, v = normal(1, B, 1, 64, 128), normal(2, B, 8, 576, 128), normal(3, B, 8, 576, 128)
    kb, vb, seq, n = normal(4, B, 8, 1, 128), normal(5, B, 8, 1, 128), i32([rows] * B), i32([100])
    p = dk.Params(B, 576, 0, 0, 0, 0, 1)
    us, out = [], []
    for cap in (128, 65536):
        pk, pv = normal(6, 1, 8, cap, 128), normal(7, 1, 8, cap, 128)
        if out:
            pk[:, :, :100], pv[:, :, :100] = first[0][:, :, :100], first[1][:, :, :100]
        else:
            first = pk, pv
        call = dk.PrefixCall(p, q, pk, pv, n, k, v, kb, vb, seq)
        us.append(best_us(call))
        out.append([t.clone() for t in call()])
    assert us[1] < 1.8 * us[0]
    # cut among other numbers of CTAs: two sums of the same terms, off by 2^-24 a
    # term, their exponentials by 2^-21, and the logarithms' rounding
    lse = [x[1] for x in out]
    bound = 2 * ((rows + 101) * 2.0 ** -24 + 2.0 ** -21) + 2.0 ** -22 * float(lse[0].abs().max())
    assert float((lse[0] - lse[1]).abs().max()) <= bound


# ------------------------------------------------ shapes of the attention kernel

ROWS = [
    # T, hq, hkv: query rows per KV head
    (5, 12, 1),      # 60
    (8, 16, 2),      # 64
    (5, 13, 1),      # 65
    (9, 16, 2),      # 72
    (8, 32, 2),      # 128
]


def check_rows(x, o, lse, keys_of, sinks, window):
    """o and lse of every (sequence, KV head) against float64."""
    G = x.hq // x.hkv
    for b in range(x.B):
        for g in range(x.hkv):
            keys, vals = keys_of(b, g)
            n = keys.shape[0]
            i = n - x.T + torch.arange(x.T, device="cuda").repeat_interleave(G).view(-1, 1)
            j = torch.arange(n, device="cuda")
            seen = (j <= i) & ((i - j < window) | (j < sinks))
            pick = lambda a: a[b, :, g * G:(g + 1) * G].reshape(x.T * G, -1)
            ro, rl, ra = attend64(pick(x.q), keys, vals, seen)
            assert_attended(pick(o), pick(lse).squeeze(-1), ro.cpu().numpy(), rl.cpu().numpy(), ra.cpu().numpy(),
                            logit_error(x.q, keys), n)


@pytest.mark.parametrize("lens", [[60, 5], [5003, 300, 0]])   # whole units; units split and merged
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,hq,hkv", ROWS)
def test_query_rows_whole_and_split(T, hq, hkv, d, lens):
    """57 to 64 rows take one CTA per SM at d = 128, more take 128-row products;
    each over units of one CTA and of several, alone and behind a prefix."""
    x = Block(lens, T, hq, hkv, d, seed=T * hq)
    p = params(x, 7, 2900)
    o, lse = dk.dustin_window_attn(p, x.q, x.k, x.v, x.kb, x.vb, x.seq)
    own = lambda c, blk, b, g: torch.cat([c[b, g, :lens[b]], blk[b, g]])
    check_rows(x, o, lse, lambda b, g: (own(x.k, x.kb, b, g), own(x.v, x.vb, b, g)), 7, 2900)
    P = 333
    pk, pv = normal(77, 1, hkv, P, d), normal(78, 1, hkv, P, d)
    o, lse = dk.dustin_prefix_attn(p, x.q, pk, pv, i32([P]), x.k, x.v, x.kb, x.vb, x.seq)
    check_rows(x, o, lse, lambda b, g: (torch.cat([pk[0, g], own(x.k, x.kb, b, g)]),
                                        torch.cat([pv[0, g], own(x.v, x.vb, b, g)])), 0, 1 << 30)


# ------------------------------------------------ more layers than a call takes


def test_evict_in_groups_of_layers():
    """Twenty layers in two calls, the first with a copy of the lengths."""
    B, hkv, d, cap, n, k, layers = 2, 2, 64, 160, 140, 100, 20
    ks, vs = ([normal(50 + 2 * l + x, B, hkv, cap, d) for l in range(layers)] for x in (0, 1))
    g = torch.Generator("cuda").manual_seed(5)
    w = [torch.rand((B, hkv, cap), device="cuda", generator=g) for _ in range(layers)]
    pos = [torch.arange(cap, dtype=torch.int32, device="cuda").expand(B, hkv, cap).contiguous() for _ in range(layers)]
    before = [[to_bits(a), to_bits(b), c.cpu().numpy(), e.cpu().numpy()] for a, b, c, e in zip(ks, vs, w, pos)]
    lens = [n, 120]
    seq, seen = i32(lens), i32(lens)
    p = dk.Params(B, cap, 0, 2, 10, 0, k)
    first = seq.clone()
    for at, lengths in ((slice(0, 16), first), (slice(16, layers), seq)):
        dk.dustin_evict(p, ks[at], vs[at], w[at], pos[at], seen, lengths)
    assert seq.tolist() == first.tolist() == [k, k]
    for l, old in enumerate(before):
        ref = O.evict(*old, lens, np.asarray(lens), k, 2, 10)
        for a, r in zip((to_bits(ks[l]), to_bits(vs[l]), w[l].cpu().numpy(), pos[l].cpu().numpy()), ref):
            assert np.array_equal(a, r), l


def test_accumulate_nan_lse_shows_in_the_rows_that_it_counts_in():
    """A query that is not finite (lse NaN) is not passed over like an empty one."""
    L, T, n = 200, 3, 2
    x = Block([L, L], T, 8, 2, 64, seed=36)
    p = params(x)
    seen, new = i32([L, L]), i32([n, n])
    runs = []
    for bad in (False, True):
        w, pos = torch.ones((2, 2, x.cap), device="cuda"), torch.zeros((2, 2, x.cap), dtype=torch.int32, device="cuda")
        lse = torch.full((2, T, 8), 5.0, device="cuda")
        if bad:
            lse[1, 0, 6] = float("nan")
        dk.dustin_accumulate(p, x.q, lse, x.k, new, x.seq, seen, w, pos)
        runs.append(w)
    # query 0 of sequence 1 sits at row L - n; head 6 is KV head 1's
    assert runs[1][1, 1, :L - n + 1].isnan().all()
    runs[1][1, 1, :L - n + 1] = runs[0][1, 1, :L - n + 1]
    assert torch.equal(runs[0], runs[1])
