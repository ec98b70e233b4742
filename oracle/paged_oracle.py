"""fp64 CPU oracle of the paged-cache operators: block tables and slot maps,
head norms with the position rotation, attention over pages.

TEST INFRASTRUCTURE, like ``dustin_oracle``: plain loops, whole numbers in
Python, everything else in float64 over bf16 bit patterns (host ``uint16``
arrays), nothing shared with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

from .dustin_oracle import bf16

SEQLEN, PAGES, INDEX = 16, 32, 1


def page_map(seq_len, n_new, table, held, free_list, n_free, page, N, max_new):
    """Copies of the tables after the call, the outputs and the flags, in a dict."""
    table, held, free = np.array(table), [int(h) for h in held], [int(x) for x in free_list]
    B, width, top, flags = len(held), table.shape[1], int(n_free), 0
    total, cu, good, need = 0, [0], [], []
    for b in range(B):
        L, n = int(seq_len[b]), int(n_new[b])
        ok = (L >= 0 and 0 <= n <= max_new and L + n <= width * page and total + n <= N and 0 <= held[b] <= width)
        total += max(n, 0)
        cu.append(min(total, N))
        good.append(ok)
        need.append(math.ceil((L + n) / page) if ok else held[b])
        flags |= 0 if ok else SEQLEN
    back = [(b, j) for b in range(B) for j in range(need[b], held[b])]
    pool = 0 <= top <= len(free) and top + len(back) <= len(free)
    served = list(good)
    if not pool:
        flags |= PAGES
        for b in range(B):
            served[b] = served[b] and need[b] <= held[b]
    else:
        for b, j in back:
            free[top] = int(table[b, j])
            top += 1
        short = False
        for b in range(B):
            more = need[b] - held[b]
            if more > 0:
                short = short or more > top
                if short:
                    served[b] = False
                    flags |= PAGES
                    continue
                for _ in range(more):
                    top -= 1
                    table[b, held[b]] = free[top]
                    held[b] += 1
            else:
                held[b] = need[b]
    slot, pos = [-1] * N, [0] * N
    for b in range(B):
        for i in range(cu[b], cu[b + 1]):
            p = int(seq_len[b]) + i - cu[b]
            pos[i] = p
            if served[b]:
                at = int(table[b, p // page])
                if 0 <= at < len(free):
                    slot[i] = at * page + p % page
                else:
                    flags |= INDEX
    kv_len = [int(seq_len[b]) + int(n_new[b]) if served[b] else 0 for b in range(B)]
    return dict(table=table, held=np.array(held), free_list=np.array(free), n_free=np.array([top]), cu=np.array(cu),
                kv_len=np.array(kv_len), slot=np.array(slot), pos=np.array(pos), flags=flags)


def norm_rope(x, w, eps, inv_freq, pos, rot, interleaved):
    """Heads ``x`` (bits [N][heads][d]) normed by ``w`` (bits [d] or None) and
    rotated: ``(y, bound)`` in float64, bound[...] = |a| + |b| of the pair that
    the element belongs to."""
    x = bf16(x)
    if w is not None:
        x = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * bf16(w)
    y, size = x.copy(), np.abs(x)
    for j in range(rot // 2):
        ia, ib = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
        t = np.asarray(pos, np.float64) * float(inv_freq[j])
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    return y, size


def paged_attn(Q, KC, VC, table, cu, kv_len):
    """``(o [N][hq][d], lse [N][hq], sum p |v|)``; rows of no request are NaN.
    Table entries outside the pool stand for pages of zeros."""
    N, hq, d = Q.shape
    pages, hkv, page, _ = KC.shape
    G = hq // hkv
    o, lse, size = np.full((N, hq, d), np.nan), np.full((N, hq), np.nan), np.full((N, hq, d), np.nan)
    for b in range(len(kv_len)):
        n, kv = int(cu[b + 1]) - int(cu[b]), int(kv_len[b])
        rows = np.arange(kv)
        ids = np.asarray(table[b], int)[rows // page]
        real = (ids >= 0) & (ids < pages)
        for h in range(hq):
            k, v = np.zeros((kv, d)), np.zeros((kv, d))
            k[real] = bf16(KC[ids[real], h // G, rows[real] % page])
            v[real] = bf16(VC[ids[real], h // G, rows[real] % page])
            for t in range(n):
                i, p = int(cu[b]) + t, kv - n + t
                if p < 0:
                    o[i, h], lse[i, h], size[i, h] = 0.0, -math.inf, 0.0
                    continue
                z = k[:p + 1] @ bf16(Q[i, h]) / math.sqrt(d)
                top = z.max()
                e = np.exp(z - top)
                o[i, h], size[i, h] = e @ v[:p + 1] / e.sum(), e @ np.abs(v[:p + 1]) / e.sum()
                lse[i, h] = top + math.log(e.sum())
    return o, lse, size
