"""Inputs and bounds for the paged-cache operators' tests."""
from __future__ import annotations

import numpy as np
import torch

from _cache_cases import U16, i32, normal

NAN = float("nan")


def pages_of(rows, page):
    return -(-rows // page)


class Paged:
    """Requests with ``ctx[b]`` cached rows and ``new[b]`` new tokens over pools of
    pages in random order; rows that hold no token are NaN, the pages of no
    request too."""

    def __init__(self, ctx, new, hq, hkv, d, page=16, seed=0, spare=3, extra=2, pad=0, layout="head", far=0):
        self.ctx, self.new, self.hq, self.hkv, self.d, self.page, self.B = list(ctx), list(new), hq, hkv, d, page, len(ctx)
        rng = np.random.default_rng(seed)
        self.kv = [c + n for c, n in zip(ctx, new)]
        counts = [pages_of(x, page) for x in self.kv]
        self.n_pages = sum(counts) + spare + far
        order = rng.permutation(sum(counts) + spare) + far
        self.width = max(counts) + extra
        table = np.full((self.B, self.width), -7)     # entries past a request's pages are never read
        at = 0
        for b, c in enumerate(counts):
            table[b, :c] = order[at:at + c]
            at += c
        self.table_host, self.left = table, order[at:]
        self.table, self.kv_len = i32(table), i32(self.kv)
        self.cu_host = np.concatenate([[0], np.cumsum(new)])
        self.cu = i32(self.cu_host)
        self.N = int(self.cu_host[-1]) + pad
        self.q = normal(seed + 1, self.N, hq, d, scale=2.0)
        self.kc, self.vc = (self._pool(layout) for _ in range(2))
        for b, x in enumerate(self.kv):
            for j in range(counts[b]):
                n = min(page, x - j * page)
                for t, s in ((self.kc, 2), (self.vc, 3)):
                    t[int(table[b, j]), :, :n] = normal(seed + 1000 * b + 10 * j + s, hkv, n, d)

    def _pool(self, layout):
        P, h, r, d = self.n_pages, self.hkv, self.page, self.d
        if layout == "token":
            return torch.full((P, r, h, d), NAN, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
        if layout == "padded":
            return torch.full((P, h + 1, r + 3, d + 8), NAN, dtype=torch.bfloat16, device="cuda")[:, :h, :r, :d]
        return torch.full((P, h, r, d), NAN, dtype=torch.bfloat16, device="cuda")

    def batch(self, dk, **over):
        a = dict(B=self.B, N=self.N, max_new=max(1, max(self.new)), max_pages=self.width)
        a.update(over)
        return dk.Batch(**a)

    def rows(self, b, g, pool):
        """Request b's rows of KV head g, in order."""
        ids = self.table[b, :pages_of(self.kv[b], self.page)].long()
        return pool[ids, g].reshape(-1, self.d)[:self.kv[b]]


def assert_rotated(got, ref, size):
    """bf16 outputs of dustin_norm_rope.  The sum of squares takes at most 16
    additions in a lane and 3 across lanes, each off by 2^-24 of itself (half of
    that in the root), rsqrtf 2^-22, the two products 2^-24 each: under 2^-20 of a
    normed element.  cos and sin: the angle is off by 2^-23 (its rounding to 24 bits
    of a half-turn) and the functions by 2^-23, the two products and the sum by
    2^-24 each: under 2^-21 of |a| + |b|.  Then one rounding to bf16."""
    got = got.double().cpu().numpy()
    off = np.abs(got - ref) - U16 * np.abs(ref) - (1 + U16) * (2.0 ** -20 + 2.0 ** -21) * size - 1e-38
    assert np.all(np.isfinite(got)) and off.max() <= 0, f"{off.max():.3e} past its bound"
