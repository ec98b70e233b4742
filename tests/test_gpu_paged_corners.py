"""Corners of the paged-cache operators: calls that their documentation allows and
that the other tests do not make."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU too
    pytest.skip("needs a GPU", allow_module_level=True)

import sparse_kv_verify_gb300 as dk  # noqa: E402
from synth import to_bits  # noqa: E402
from oracle.dustin_oracle import bf16  # noqa: E402

from _cache_cases import assert_attended, attend64, i32, logit_error, normal  # noqa: E402
from _paged_cases import Paged, assert_rotated, pages_of  # noqa: E402
from _turns import angles  # noqa: E402
from test_gpu_paged import check_map, random_pool  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


# --------------------------------------------------------------- norm, rope


FAR = [0, 1, 5, -1, 2 ** 20, 2 ** 24 + 1, 10 ** 9 + 7, 2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 12345, -2 ** 31, 1 - 2 ** 31]
FREQS = [1.0, 0.649, 1e-3, 1e-6, 1e-30, 1e-42, 0.0, -0.5, 6.2831855, 3.1415927, 1000.0, 1e6, 12345.678, 1e9, 2.0 ** 38, -2.0 ** 38 - 2.0 ** 15]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_rope_angles_lose_nothing_at_far_positions(d, interleaved):
    """Against angles reduced in whole numbers: fp64 products of 31 bits of position and
    24 of frequency would be rounded already.  The bounds are those of near ones."""
    N, rot, rng = len(FAR), 2 * len(FREQS), np.random.default_rng(d)
    freqs = np.float32(rng.permutation(FREQS))
    q, k, v = normal(d, N, 3, d), normal(d + 1, N, 1, d), normal(d + 2, N, 1, d)
    kc, vc = (torch.zeros((N, 1, 16, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = dk.binding.Workspace(dk.paged_workspace_bytes(dk.Batch(1, 1, 1, 1)))
    got = dk.dustin_norm_rope(dk.Rope(rot, interleaved), q, k, v, None, None, torch.as_tensor(freqs, device="cuda"),
                              i32(FAR), i32(16 * np.arange(N)), kc, vc, ws=ws)
    assert dk.check(ws) == 0
    t = angles(freqs, FAR)
    for x, out in ((q, got), (k, kc[:, :, 0])):
        x = bf16(to_bits(x))
        y, size = x.copy(), np.abs(x)
        for j in range(rot // 2):
            ia, ib = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
            c, s, a, b = np.cos(t[:, j])[:, None], np.sin(t[:, j])[:, None], x[..., ia], x[..., ib]
            y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
            size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
        assert_rotated(out, y, size)


def rope_heads(q, k, v, w, eps, d, page=16):
    """One call without a rotation over pools of zeros: (q_out, rows of k, flags)."""
    N, hkv = k.shape[:2]
    kc, vc = (torch.zeros((pages_of(N, page), hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = dk.binding.Workspace(dk.paged_workspace_bytes(dk.Batch(1, 1, 1, 1)))
    got = dk.dustin_norm_rope(dk.Rope(0, eps=eps), q, k, v, *w, None, i32(np.zeros(N)), i32(np.arange(N)), kc, vc, ws=ws)
    at = torch.arange(N, device="cuda")
    return got, kc[at // page, :, at % page], dk.check(ws)


@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-38, 1e-32, 2.0 ** -100 * (1 - 2.0 ** -24), 2.0 ** -100, 1e-12, 1e-6, 1.0, 1e30])
@pytest.mark.parametrize("d", [64, 128])
def test_rope_norms_heads_however_small(d, eps):
    """Heads from the smallest bf16 to 2^60, the largest that the call takes: the squares
    of small ones leave fp32's range, the norm does not.  Also heads with elements of
    very different sizes."""
    sizes = list(range(-126, 57, 3))
    N = len(sizes)
    f = torch.tensor([2.0 ** s for s in sizes], dtype=torch.float64, device="cuda").view(-1, 1, 1)
    of_size = lambda t: (t.double().clamp(-3.9, 3.9) * f).to(torch.bfloat16)
    q, k, v = of_size(normal(d, N, 3, d)), of_size(normal(d + 1, N, 2, d)), normal(d + 2, N, 2, d)
    q[:, 1] = 2.0 ** -133                               # a head of denormals, and one large element among them
    q[:, 2, 1:] = 2.0 ** -133
    q[:, 2, 0] = f[:, 0, 0].to(torch.bfloat16)
    k[:, 1, ::2] = 1.0
    w = [(1 + normal(s, d, scale=0.3).float()).to(torch.bfloat16) for s in (3, 4)]
    got, rows, flags = rope_heads(q, k, v, w, eps, d)
    assert flags == 0
    for x, y, wt in ((q, got, w[0]), (k, rows, w[1])):
        xb = bf16(to_bits(x))
        ref = xb / np.sqrt((xb * xb).mean(axis=-1, keepdims=True) + float(np.float32(eps))) * bf16(to_bits(wt))
        assert_rotated(y, ref, np.abs(ref))


def test_rope_zeros_without_eps_are_nan():
    """0 / 0, in that head alone."""
    q, k, v = normal(1, 4, 2, 64), normal(2, 4, 1, 64), normal(3, 4, 1, 64)
    q[2, 1] = 0
    w = [torch.ones(64, dtype=torch.bfloat16, device="cuda")] * 2
    got, rows, flags = rope_heads(q, k, v, w, 0.0, 64)
    assert flags == 0 and bool(got[2, 1].isnan().all()) and int(got.isnan().sum()) == 64 and not bool(rows.isnan().any())
    got, _, _ = rope_heads(q, k, v, w, 1e-45, 64)
    assert bool((got[2, 1] == 0).all()) and not bool(got.isnan().any())


# ---------------------------------------------------------------- page map


@pytest.mark.parametrize("n,held", [(1, 0), (1, 3), (0, 1)])
def test_map_of_a_length_next_to_2_to_31(n, held):
    """seq_len + n_new passes 32 bits by itself: that request alone is flagged."""
    rng = np.random.default_rng(1)
    seq, new, table, have, free, n_free = random_pool(rng, 12, 16, 8, 20, 1)
    seq[3], new[3] = 2 ** 31 - 1, n
    have[3] = min(held, have[3])
    r = check_map(seq, new, table, have, free, n_free, 16, int(new.sum()) + 7, 20)
    assert r["flags"] == 16 and r["kv_len"][3] == 0 and (r["kv_len"][:3] == (seq + new)[:3]).all()


# --------------------------------------------------------------- attention


@pytest.mark.parametrize("B,hq,hkv,d,page,longest", [
    (40, 8, 1, 128, 16, 400), (40, 16, 4, 64, 128, 400), (300, 8, 2, 128, 64, 300), (300, 14, 2, 64, 16, 300),
    (2000, 8, 1, 64, 16, 70)])
def test_attn_batches_of_many_requests_with_chunks(B, hq, hkv, d, page, longest):
    """More requests than a warp has lanes in the shape for chunks: single tokens, runs of
    idle requests, and requests of more than four pairs of row tiles among them."""
    rng = np.random.default_rng(B + d)
    ctx = rng.integers(0, longest, B)
    new = np.where(rng.random(B) < 0.2, rng.integers(2, 30, B), 1)
    G = hq // hkv
    pair = 2 * (128 // G)                                # tokens
    for b in (0, B // 3, B - 5):                         # idle ones, the last five among them
        new[b:b + 5] = 0
    many = rng.permutation(np.flatnonzero(new))[:6 + B // 60]
    new[many] = rng.integers(4 * pair + 1, 9 * pair, many.size)
    new[B // 3 - 1] = 6 * pair                           # and some behind a chunk
    assert (new > 4 * pair).sum() >= 4
    x = Paged(ctx.tolist(), new.tolist(), hq, hkv, d, page, seed=B, pad=3)
    ws = dk.binding.Workspace(dk.paged_workspace_bytes(x.batch(dk), hq, hkv, d))
    o = torch.full((x.N, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((x.N, hq), 7.0, device="cuda")
    dk.dustin_paged_attn(x.batch(dk), x.q, x.kc, x.vc, x.table, x.cu, x.kv_len, o, lse, ws=ws)
    assert dk.check(ws) == 0
    assert bool((o[-3:] == 7).all()) and bool((lse[-3:] == 7).all())
    for b in range(B):
        n, kv, at = int(new[b]), x.kv[b], int(x.cu_host[b])
        if n == 0 or (B > 300 and n <= 4 * pair and b % 11):
            continue
        seen = torch.arange(kv, device="cuda") <= torch.arange(kv - n, kv, device="cuda").repeat_interleave(G).view(-1, 1)
        for g in range(hkv):
            pick = lambda t: t[at:at + n, g * G:(g + 1) * G].reshape(n * G, -1)
            q, k, v = pick(x.q), x.rows(b, g, x.kc), x.rows(b, g, x.vc)
            ro, rl, ra = [t.cpu().numpy() for t in attend64(q, k, v, seen)]
            assert_attended(pick(o), pick(lse).squeeze(-1), ro, rl, ra, logit_error(q, k), kv)
