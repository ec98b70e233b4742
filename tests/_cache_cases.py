"""Inputs, error bounds and a float64 torch reference for the cache operators' tests."""
from __future__ import annotations

import math

import numpy as np
import torch

from synth import to_bits

U16 = 2.0 ** -8     # a bf16 rounding is off by at most this share of the value


def normal(seed, *shape, scale=1.0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=device) * scale).to(torch.bfloat16)


def i32(x, device="cuda"):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device=device)


class Block:
    """A draft block over a batch's caches; rows at or beyond seq_len are NaN."""

    def __init__(self, lens, T, hq, hkv, d, seed=0, cap=None, slack=70):
        B = len(lens)
        self.lens, self.T, self.hq, self.hkv, self.d, self.B = list(lens), T, hq, hkv, d, B
        self.cap = cap if cap is not None else max(lens) + slack
        self.q = normal(seed + 1, B, T, hq, d, scale=2.0)
        self.k = normal(seed + 2, B, hkv, self.cap, d)
        self.v = normal(seed + 3, B, hkv, self.cap, d)
        self.kb = normal(seed + 4, B, hkv, T, d)
        self.vb = normal(seed + 5, B, hkv, T, d)
        for b, L in enumerate(lens):
            self.k[b, :, L:] = float("nan")
            self.v[b, :, L:] = float("nan")
        self.seq = i32(lens)

    def bits(self, *names):
        return [to_bits(getattr(self, n)) for n in names]


def logit_error(q, *ks):
    """A bound of the error of a scaled fp32 logit: a dot product of d bf16
    pairs (exact products) accumulated with at most one unit of 2^-23 of the
    running sum of magnitudes per term, which |q| |k| bounds."""
    d = q.shape[-1]
    top = max([float(torch.nan_to_num(k.float()).norm(dim=-1).max()) for k in ks if k.numel()] + [0.0])
    return d * 2.0 ** -23 * float(q.float().norm(dim=-1).max()) * top / math.sqrt(d)


def assert_attended(o, lse, ref_o, ref_lse, mean_abs, zerr, keys):
    """o: each weight is rounded to bf16 once (off by U16 of its share of
    mean_abs = sum p |v|) and the output once more; both carry the logits'
    error (2 zerr: weight and normaliser) and fp32 sums of ``keys`` terms.
    lse: the logits' error, the sum's and the exponentials' (2^-21 each)."""
    o = o.double().cpu().numpy()
    lse = lse.double().cpu().numpy()
    small = keys * 2.0 ** -24 + 2.0 ** -20
    assert np.all(np.isfinite(o))
    bound = U16 * (mean_abs * (1 + U16) + np.abs(ref_o)) + (2 * zerr + 2 * small) * mean_abs + 1e-30
    off = np.abs(o - ref_o) - bound
    assert off.max() <= 0, f"o is {off.max():.3e} past its bound"
    empty = np.isneginf(ref_lse)
    assert np.array_equal(empty, np.isneginf(lse))
    got, want = lse[~empty], ref_lse[~empty]
    off = np.abs(got - want) - (zerr + small + 2.0 ** -22 * np.abs(want))
    assert off.size == 0 or off.max() <= 0, f"lse is {off.max():.3e} past its bound"


def attend64(q, keys, vals, seen):
    """float64 (o, lse, sum p |v|) of q [n, d] over keys [m, d] with a mask [n, m]."""
    z = q.double() @ keys.double().T / math.sqrt(q.shape[-1])
    z = z.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(z, dim=-1)
    p = torch.exp(z - lse.unsqueeze(-1)).nan_to_num(0.0)
    return p @ vals.double(), lse, p @ vals.double().abs()


def assert_weights(w, ref, prior, zerr, rows):
    """Each of up to ``rows`` terms carries the logit's error, the exponential's
    (2^-21) and, with the prior weight, a sum's roundings."""
    w = w.double().cpu().numpy()
    off = np.abs(w - ref) - (2 * zerr + 2.0 ** -20 + rows * 2.0 ** -24) * ref - 2.0 ** -23 * np.abs(prior) - 1e-30
    assert off.max() <= 0, f"weight is {off.max():.3e} past its bound"
