"""fp64 CPU oracle of the cache operators: windowed attention with sinks,
shared-prefix attention, accumulated attention weights and eviction by them.

TEST INFRASTRUCTURE, like ``dustin_oracle``: plain loops in float64 over bf16
bit patterns (host ``uint16`` arrays), one query row at a time, nothing shared
with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

from .dustin_oracle import bf16


def _attend(q, keys, vals):
    """(o, lse) of one fp64 query over fp64 keys; nothing visible: (0, -inf)."""
    if keys.shape[0] == 0:
        return np.zeros(q.shape[0]), -math.inf
    z = keys @ q / math.sqrt(q.shape[0])
    top = z.max()
    e = np.exp(z - top)
    return e @ vals / e.sum(), top + math.log(e.sum())


def window_attn(Q, K, V, Kb, Vb, seq_len, sinks, window):
    """``(o [B][T][hq][d], lse [B][T][hq])`` of the draft block.

    The key at position j is visible to the query at position i iff j <= i and
    (i - j < window or j < sinks); cache row j has position j, query and block
    row t position seq_len[b] + t.
    """
    B, T, hq, d = Q.shape
    G = hq // K.shape[1]
    o, lse = np.zeros((B, T, hq, d)), np.full((B, T, hq), -math.inf)
    for b in range(B):
        L = int(seq_len[b])
        for t in range(T):
            i = L + t
            seen = [j for j in range(i + 1) if i - j < window or j < sinks]
            cache = [j for j in seen if j < L]
            block = [j - L for j in seen if j >= L]
            for h in range(hq):
                g = h // G
                keys = np.concatenate([bf16(K[b, g, cache]), bf16(Kb[b, g, block])])
                vals = np.concatenate([bf16(V[b, g, cache]), bf16(Vb[b, g, block])])
                o[b, t, h], lse[b, t, h] = _attend(bf16(Q[b, t, h]), keys, vals)
    return o, lse


def prefix_attn(Q, PK, PV, P, K, V, Kb, Vb, seq_len):
    """``(o, lse)``: keys are rows [0, P) of the shared prefix ``PK[0]``, then
    the sequence's own rows, then block rows u <= t."""
    B, T, hq, d = Q.shape
    G = hq // K.shape[1]
    o, lse = np.zeros((B, T, hq, d)), np.full((B, T, hq), -math.inf)
    pk, pv = bf16(PK[0, :, :P]), bf16(PV[0, :, :P])
    for b in range(B):
        L = int(seq_len[b])
        for g in range(K.shape[1]):
            for t in range(T):
                keys = np.concatenate([pk[g], bf16(K[b, g, :L]), bf16(Kb[b, g, :t + 1])])
                vals = np.concatenate([pv[g], bf16(V[b, g, :L]), bf16(Vb[b, g, :t + 1])])
                for h in range(g * G, (g + 1) * G):
                    o[b, t, h], lse[b, t, h] = _attend(bf16(Q[b, t, h]), keys, vals)
    return o, lse


def accumulate(Q, lse, K, n_new, seq_len, n_seen, weight, pos):
    """New ``(weight float64, pos)``: the first ``n_new[b]`` query rows, which
    sit at the cache's last ``n_new[b]`` rows, add their probabilities."""
    B, _, hq, d = Q.shape
    G = hq // K.shape[1]
    weight, pos = weight.astype(np.float64).copy(), pos.copy()
    for b in range(B):
        L, n = int(seq_len[b]), int(n_new[b])
        for g in range(K.shape[1]):
            keys = bf16(K[b, g, :L])
            weight[b, g, L - n:L] = 0.0
            pos[b, g, L - n:L] = int(n_seen[b]) - L + np.arange(L - n, L)
            for t in range(n):
                for h in range(g * G, (g + 1) * G):
                    upto = L - n + t + 1
                    if lse[b, t, h] == -math.inf:
                        continue
                    z = keys[:upto] @ bf16(Q[b, t, h]) / math.sqrt(d)
                    weight[b, g, :upto] += np.exp(z - float(lse[b, t, h]))
    return weight, pos


def evict_rows(weight, pos, n, k, sinks, window, n_seen):
    """Which rows of one unit stay: ``(holes, movers)``, both ascending, the
    i-th hole taking the i-th mover."""
    if n <= k:
        return np.zeros(0, int), np.zeros(0, int)
    safe = (pos[:n] < sinks) | (pos[:n] >= n_seen - window)
    w = weight[:n].astype(np.float64)
    w = np.where(np.isnan(w) | (w < 0), 0.0, w)
    order = sorted(range(n), key=lambda j: (not safe[j], 0.0 if safe[j] else -w[j], j))
    kept = np.zeros(n, bool)
    kept[order[:k]] = True
    return np.nonzero(~kept[:k])[0], k + np.nonzero(kept[k:])[0]


def evict(K, V, weight, pos, n_seen, seq_len, k, sinks, window):
    """Copies of one layer's ``(K, V, weight, pos, seq_len)`` after the eviction."""
    K, V, weight, pos = K.copy(), V.copy(), weight.copy(), pos.copy()
    for b in range(K.shape[0]):
        for g in range(K.shape[1]):
            dst, src = evict_rows(weight[b, g], pos[b, g], int(seq_len[b]), k, sinks, window, int(n_seen[b]))
            for a in (K, V, weight, pos):
                a[b, g, dst] = a[b, g, src]
    return K, V, weight, pos, np.minimum(seq_len, k)
