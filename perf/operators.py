"""Cases and plain forms of the cache operators: windowed attention with
sinks, shared-prefix attention, accumulated attention weights and eviction by
them.

``run`` computes an operator in elementary torch operations in fp32 (``own``
false) or through the framework's entry points (``own`` true).  ``exact``
restates each definition in float64.

Shapes: ``hq``/``hkv``/``d`` are 64/8/128 (the target model of the workloads
in ``synth``) or 14/2/64 (its draft model); a draft block has ``gamma + 1``
rows.  Sequence lengths spread evenly from ``L`` down to ``L - L * ragged``.
"""
import math

import numpy as np
import torch

own = False

_TARGET = {"hq": 64, "hkv": 8, "d": 128}
_DRAFT = {"hq": 14, "hkv": 2, "d": 64}


def listed():
    return [
        # One token of one sequence through a short-window layer: the smallest
        # call, where latency counts.
        dict(_TARGET, name="window_token", op="window", B=1, gamma=0, L=32768, ragged=0.0,
             sinks=4, window=128),
        # A batched draft block through a layer with a 4096-token window.
        dict(_TARGET, name="window_batch", op="window", B=16, gamma=5, L=32768, ragged=0.5,
             sinks=16, window=4096),
        # The draft model's heads, odd sizes throughout, some sequences shorter
        # than the window.
        dict(_DRAFT, name="window_odd", op="window", B=9, gamma=4, L=5003, ragged=0.95,
             sinks=3, window=1001),
        # Single tokens of a few sequences behind one system prompt.
        dict(_TARGET, name="prefix_token", op="prefix", B=4, gamma=0, P=8192, L=512, ragged=0.5),
        # Batched draft blocks behind a long shared document.
        dict(_TARGET, name="prefix_batch", op="prefix", B=16, gamma=5, P=32768, L=2048, ragged=0.5),
        # The largest: many sequences behind a 64 K prefix, short own parts.
        dict(_TARGET, name="prefix_large", op="prefix", B=32, gamma=4, P=65536, L=1000, ragged=0.9),
        # The draft model's heads, a prefix that ends inside every tile, own
        # parts down to a few rows.
        dict(_DRAFT, name="prefix_odd", op="prefix", B=5, gamma=2, P=3001, L=301, ragged=1.0),
        # One accepted token accumulated over one sequence's cache.
        dict(_TARGET, name="accumulate_token", op="accumulate", B=1, gamma=0, L=4097, ragged=0.0),
        # Accepted rows of a batch over full-length caches, before a first eviction.
        dict(_TARGET, name="accumulate_batch", op="accumulate", B=16, gamma=5, L=32768, ragged=0.25),
        # The steady state of a bounded cache: a block of new rows in, as many
        # rows out, for a batch.
        dict(_TARGET, name="evict_step", op="evict", B=16, gamma=5, n=2054, k=2048, sinks=16,
             window=256, first=False),
        # The first eviction after a long prompt: 32 K positions down to the budget.
        dict(_TARGET, name="evict_prompt", op="evict", B=16, gamma=5, n=32768, k=2048, sinks=16,
             window=256, first=True),
        # One sequence of the draft model, odd sizes.
        dict(_DRAFT, name="evict_odd", op="evict", B=1, gamma=4, n=10007, k=1023, sinks=3, window=65,
             first=True),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "prefix", "accumulate", "evict"])
    shape = dict(rng.choice([_TARGET, _TARGET, _DRAFT]))
    if rng.random() < 0.3:   # other group sizes: one to sixteen query heads per KV head
        shape["hkv"] = rng.choice([1, 2, 4, 8])
        shape["hq"] = shape["hkv"] * rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
    group = shape["hq"] // shape["hkv"]
    gamma = rng.choice([0, 0, 1, 2, 4, 5, 8])
    gamma = min(gamma, 128 // group - 1)
    c = dict(shape, op=op, gamma=gamma)
    if op == "window":
        c.update(B=_logu(rng, 1, 24), L=_logu(rng, 1, 32768), ragged=rng.choice([0.0, 0.5, 1.0]),
                 sinks=rng.choice([0, 1, 4, 16, 100]), window=_logu(rng, 1, 4096))
    elif op == "prefix":
        B = _logu(rng, 1, 32)
        most = 5 * 8 * 32 * 8 * 128 * 65536 // (B * (gamma + 1) * c["hq"] * c["d"])   # the largest's products
        c.update(B=B, P=_logu(rng, 1, min(65536, most)), L=_logu(rng, 1, 2048), ragged=rng.choice([0.0, 0.5, 1.0]))
    elif op == "accumulate":
        c.update(B=_logu(rng, 1, 16), L=_logu(rng, 16, 32768), ragged=rng.choice([0.0, 0.5]))
    else:
        first = rng.random() < 0.5
        k = _logu(rng, 64, 4096)
        c.update(B=_logu(rng, 1, 16), k=k, n=k + (_logu(rng, 1, 24 * 1024) if first else gamma + 1),
                 sinks=rng.choice([0, 3, 16]), window=rng.choice([0, 7, 32]), first=first)
    return c


def _lengths(c):
    """Sequence lengths of a case, from L down to L - L * ragged."""
    L, B = c["L"], c["B"]
    low = L - int(L * c["ragged"])
    if c["op"] == "accumulate":   # the block's own rows are in the cache
        low = max(low, c["gamma"] + 1)
    return [L - (L - low) * b // max(1, B - 1) for b in range(B)]


def _cap(n):
    return (n + 127) // 64 * 64   # cache capacity: room for the next appends


def _gen(seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)

    def normal(*shape, scale=1.0):
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
        return (x * scale).to(torch.bfloat16)
    return g, normal


def prepare(case, seed):
    c = dict(case)
    g, normal = _gen(seed)
    B, hq, hkv, d, T = c["B"], c["hq"], c["hkv"], c["d"], c["gamma"] + 1
    s = {"c": c}
    if c["op"] in ("window", "prefix"):
        lens = _lengths(c)
        cap = _cap(c["L"])
        s.update(cap=cap, longest=max(lens),
                 q=normal(B, T, hq, d, scale=2.0), k=normal(B, hkv, cap, d), v=normal(B, hkv, cap, d),
                 kb=normal(B, hkv, T, d), vb=normal(B, hkv, T, d),
                 seq_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        if c["op"] == "prefix":
            pcap = _cap(c["P"])
            s.update(pk=normal(1, hkv, pcap, d), pv=normal(1, hkv, pcap, d),
                     prefix_len=torch.tensor([c["P"]], dtype=torch.int32, device="cuda"))
        s["o"] = torch.empty((B, T, hq, d), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((B, T, hq), dtype=torch.float32, device="cuda")
    elif c["op"] == "accumulate":
        lens = _lengths(c)
        cap = _cap(c["L"])
        s.update(cap=cap, q=normal(B, T, hq, d, scale=2.0), k=normal(B, hkv, cap, d),
                 seq_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 n_new=torch.tensor([1 + (3 * b) % T for b in range(B)], dtype=torch.int32, device="cuda"))
        s["n_seen"] = s["seq_len"] + 1000
        s["weight"] = torch.randn((B, hkv, cap), generator=g, device="cuda").mul_(1.5).exp_()
        s["pos"] = torch.arange(cap, dtype=torch.int32, device="cuda").expand(B, hkv, cap).contiguous()
        # the log-sum-exp that the verification attention returned for these rows
        x, seen = _scores(s, torch.float32)
        s["lse"] = torch.logsumexp(torch.where(seen, x, -math.inf), dim=-1).permute(0, 2, 1, 3).reshape(B, T, hq).contiguous()
        del x, seen
    else:
        n, k = c["n"], c["k"]
        cap = _cap(n)
        s.update(cap=cap, ks=[normal(B, hkv, cap, d)], vs=[normal(B, hkv, cap, d)])
        w = torch.randn((B, hkv, cap), generator=g, device="cuda").mul_(1.5).exp_()
        w *= torch.rand((B, hkv, cap), generator=g, device="cuda") > 0.1   # never attended: exact zeros
        seen = n if c["first"] else 3 * n + 100
        if c["first"]:
            pos = torch.arange(cap, dtype=torch.int32, device="cuda").expand(B, hkv, cap).contiguous()
        else:
            # an earlier eviction's cache: sinks, recent window and other
            # positions in any order, then the new rows
            old = seen - (n - k)
            rank = torch.rand((B, hkv, old), generator=g, device="cuda")
            rank[..., :c["sinks"]] += 1.0
            rank[..., max(0, old - c["window"]):] += 1.0
            pos = torch.zeros((B, hkv, cap), dtype=torch.int32, device="cuda")
            held = rank.topk(k, dim=-1).indices
            mix = torch.rand((B, hkv, k), generator=g, device="cuda").argsort(dim=-1)
            pos[..., :k] = held.gather(-1, mix).to(torch.int32)
            pos[..., k:n] = torch.arange(old, seen, dtype=torch.int32, device="cuda")
        # weights and positions side by side, so that a pass restores both at once
        meta = torch.stack([w.view(torch.int32), pos])
        s.update(meta=meta, head=meta[..., :k].clone(), weights=[meta[0].view(torch.float32)], poss=[meta[1]],
                 n0=torch.full((B,), n, dtype=torch.int32, device="cuda"),
                 seq_len=torch.full((B,), n, dtype=torch.int32, device="cuda"),
                 n_seen=torch.full((B,), seen, dtype=torch.int32, device="cuda"))
    return s


# ------------------------------------------------------------- plain forms


def _rows(q, hkv):
    """[B, T, hq, d] -> [B, hkv, T, G, d]."""
    B, T, hq, d = q.shape
    return q.reshape(B, T, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4)


def _out(o, lse):
    """[B, hkv, T, G, d] and [B, hkv, T, G] -> the operators' layouts."""
    B, hkv, T, G, d = o.shape
    return (o.permute(0, 2, 1, 3, 4).reshape(B, T, hkv * G, d).to(torch.bfloat16),
            lse.permute(0, 2, 1, 3).reshape(B, T, hkv * G))


def _softmax(x):
    """Weights and log-sum-exp of scores with -inf for hidden keys; a row that
    sees nothing gets zero weights and -inf."""
    m = x.amax(dim=-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isfinite(m), m, 0.0))
    total = e.sum(dim=-1, keepdim=True)
    lse = torch.where(total > 0, m + torch.log(total), -math.inf)
    return e / torch.where(total > 0, total, 1.0), lse.squeeze(-1)


def _window(s):
    c = s["c"]
    hkv, d, T, W, S = c["hkv"], c["d"], c["gamma"] + 1, c["window"], c["sinks"]
    L = s["seq_len"].long().view(-1, 1)
    # the cache positions that some query of the block can see: the sinks, then
    # the window of the first query
    n_s, n_w = min(S, s["longest"]), min(W, s["longest"])
    near = torch.arange(n_w, device="cuda") + L - n_w
    at = torch.cat([torch.arange(n_s, device="cuda").expand(L.shape[0], n_s), near], dim=1)
    real = (at >= 0) & (at < L)
    real[:, n_s:] &= near >= n_s                     # sinks counted once
    idx = at.clamp(0, s["cap"] - 1)
    b = torch.arange(L.shape[0], device="cuda").view(-1, 1)
    k = torch.cat([s["k"][b, :, idx].transpose(1, 2), s["kb"]], dim=2).float()
    v = torch.cat([s["v"][b, :, idx].transpose(1, 2), s["vb"]], dim=2).float()
    at = torch.cat([at, L + torch.arange(T, device="cuda")], dim=1)
    real = torch.cat([real, torch.ones((L.shape[0], T), dtype=torch.bool, device="cuda")], dim=1)
    i = (L + torch.arange(T, device="cuda")).unsqueeze(-1)                     # [B, T, 1]
    j = at.unsqueeze(1)
    seen = real.unsqueeze(1) & (j <= i) & ((i - j < W) | (j < S))             # [B, T, n]
    q = _rows(s["q"], hkv).float()
    B, _, _, G, _ = q.shape
    x = (q.reshape(B, hkv, T * G, d) @ k.transpose(-1, -2)).view(B, hkv, T, G, -1) / math.sqrt(d)
    p, lse = _softmax(torch.where(seen[:, None, :, None], x, -math.inf))
    o = (p.view(B, hkv, T * G, -1) @ v).view(B, hkv, T, G, d)
    return _out(o, lse)


def _prefix(s):
    c = s["c"]
    hkv, d, T, P, n = c["hkv"], c["d"], c["gamma"] + 1, c["P"], s["longest"]
    q = _rows(s["q"], hkv).float()
    B, _, _, G, _ = q.shape
    L = s["seq_len"].view(-1, 1)
    own_real = (torch.arange(n, device="cuda") < L).view(B, 1, n, 1)
    k = torch.cat([s["k"][:, :, :n], s["kb"]], dim=2).float()
    v = torch.cat([torch.where(own_real, s["v"][:, :, :n], 0.0), s["vb"]], dim=2).float()
    x = torch.empty((B, hkv, T, G, P + n + T), dtype=torch.float32, device="cuda")
    flat = q.permute(1, 0, 2, 3, 4).reshape(hkv, B * T * G, d)
    x[..., :P] = (flat @ s["pk"][0, :, :P].float().transpose(-1, -2)).view(hkv, B, T, G, P).transpose(0, 1)
    x[..., P:] = (q.reshape(B, hkv, T * G, d) @ k.transpose(-1, -2)).view(B, hkv, T, G, n + T)
    x /= math.sqrt(d)
    t = torch.arange(T, device="cuda")
    x[..., P:P + n].masked_fill_((torch.arange(n, device="cuda") >= L).view(B, 1, 1, 1, n), -math.inf)
    x[..., P + n:].masked_fill_((t.view(1, T) > t.view(T, 1)).view(T, 1, T), -math.inf)
    p, lse = _softmax(x)
    o = (p[..., :P].transpose(0, 1).reshape(hkv, B * T * G, P) @ s["pv"][0, :, :P].float())
    o = o.view(hkv, B, T, G, d).transpose(0, 1) + (p[..., P:].reshape(B, hkv, T * G, n + T) @ v).view(B, hkv, T, G, d)
    return _out(o, lse)


def _scores(s, dtype):
    """Scaled scores [B, hkv, T, G, cap] of the block's rows over the cache and
    which of them the causal rule shows."""
    c = s["c"]
    q, k = _rows(s["q"], c["hkv"]).to(dtype), s["k"].to(dtype)
    B, hkv, T, G, d = q.shape
    x = (q.reshape(B, hkv, T * G, d) @ k.transpose(-1, -2)).view(B, hkv, T, G, -1) / math.sqrt(d)
    first = (s["seq_len"] - s["n_new"]).view(-1, 1, 1)
    seen = torch.arange(s["cap"], device=x.device) <= first + torch.arange(T, device=x.device).view(1, T, 1)
    return x, seen[:, None, :, None]


def _accumulate(s):
    c = s["c"]
    B, hkv, T = c["B"], c["hkv"], c["gamma"] + 1
    x, seen = _scores(s, torch.float32)
    lse = _rows(s["lse"].unsqueeze(-1), hkv)
    counts = (torch.arange(T, device="cuda") < s["n_new"].view(-1, 1)).view(B, 1, T, 1, 1)
    add = torch.where(seen & counts, torch.exp(x - lse), 0.0).sum(dim=(2, 3))
    j = torch.arange(s["cap"], device="cuda")
    L, n = s["seq_len"].view(-1, 1, 1), s["n_new"].view(-1, 1, 1)
    new = (j >= L - n) & (j < L)
    s["weight"].copy_(torch.where(new, 0.0, s["weight"]) + add)
    s["pos"].copy_(torch.where(new, s["n_seen"].view(-1, 1, 1) - L + j, s["pos"]))
    return s["weight"], s["pos"]


def _evict(s):
    c = s["c"]
    n, k = c["n"], c["k"]
    w, pos = s["weights"][0][..., :n], s["poss"][0][..., :n]
    safe = (pos < c["sinks"]) | (pos >= s["n_seen"].view(-1, 1, 1) - c["window"])
    order = torch.where(safe, math.inf, w).sort(dim=-1, descending=True, stable=True).indices
    keep = torch.zeros_like(safe).scatter_(-1, order[..., :k], True)
    hole, move = ~keep[..., :k], keep[..., k:]
    # the i-th hole takes the i-th kept row beyond the budget
    b, g, dst = hole.nonzero(as_tuple=True)
    bm, gm, src = move.nonzero(as_tuple=True)
    src = src + k
    for t in (s["ks"][0], s["vs"][0], s["weights"][0], s["poss"][0]):
        t[b, g, dst] = t[bm, gm, src]
    s["seq_len"].clamp_(max=k)
    return _held(s)


def _held(s):
    """What the caches hold after an eviction."""
    k = s["c"]["k"]
    return {"k": s["ks"][0][:, :, :k], "v": s["vs"][0][:, :, :k], "weight": s["weights"][0][..., :k],
            "pos": s["poss"][0][..., :k], "seq_len": s["seq_len"]}


# ------------------------------------------------- the framework's operators


def _call(s):
    """The prepared call that a user's program keeps and repeats."""
    import sparse_kv_verify_gb300 as dk
    c = s["c"]
    S, W = c.get("sinks", 0), c.get("window", 0)
    p = dk.Params(B=c["B"], Lcap=s["cap"], gamma=c["gamma"], sinks=S, window=W, m=0,
                  k=c.get("k", max(1, S + W)))
    if c["op"] == "window":
        return dk.WindowCall(p, s["q"], s["k"], s["v"], s["kb"], s["vb"], s["seq_len"], s["o"], s["lse"])
    if c["op"] == "prefix":
        return dk.PrefixCall(p, s["q"], s["pk"], s["pv"], s["prefix_len"], s["k"], s["v"], s["kb"], s["vb"],
                             s["seq_len"], s["o"], s["lse"])
    if c["op"] == "accumulate":
        return dk.AccumulateCall(p, s["q"], s["lse"], s["k"], s["n_new"], s["seq_len"], s["n_seen"],
                                 s["weight"], s["pos"])
    return dk.EvictCall(p, s["ks"], s["vs"], s["weights"], s["poss"], s["n_seen"], s["seq_len"])


_PLAIN = {"window": _window, "prefix": _prefix, "accumulate": _accumulate, "evict": _evict}


def run(state):
    s = state
    if s["c"]["op"] == "evict":
        # the cache before the eviction again: its length, and after a long
        # prompt also the weights and positions that the last pass moved (the
        # rows it moved are the ones this pass moves)
        s["seq_len"].copy_(s["n0"])
        if s["c"]["first"]:
            s["meta"][..., :s["c"]["k"]].copy_(s["head"])
    if own:
        if "call" not in s:
            s["call"] = _call(s)
        out = s["call"]()
        return _held(s) if s["c"]["op"] == "evict" else out
    return _PLAIN[s["c"]["op"]](s)


# ------------------------------------------------------------------- work


def work(case):
    c = case
    B, hq, hkv, d, T = c["B"], c["hq"], c["hkv"], c["d"], c["gamma"] + 1
    G = hq // hkv
    if c["op"] in ("window", "prefix"):
        block = B * (T * hq * (2 * d + 2 * d + 4) + 2 * hkv * T * d * 2)      # q, o, lse, kb, vb
        lens = _lengths(c)
        if c["op"] == "window":
            # (pairs of query and key that the rule shows, rows of the cache read)
            pairs = rows = 0
            for L in lens:
                lo = max(0, L - c["window"] + 1)
                rows += min(L, c["sinks"]) + max(0, L - max(lo, c["sinks"]))
                for t in range(T):
                    i = L + t
                    first = max(0, i - c["window"] + 1)
                    pairs += i + 1 - first + min(first, c["sinks"])
        else:
            rows = c["P"] + sum(lens)
            pairs = sum(T * (c["P"] + L) + T * (T + 1) // 2 for L in lens)
        return {"bytes": block + rows * hkv * d * 4, "flops": 4 * pairs * hq * d}
    if c["op"] == "accumulate":
        lens = _lengths(c)
        news = [1 + (3 * b) % T for b in range(B)]
        read = sum(lens) * hkv * (2 * d + 8) + sum(news) * hq * (2 * d + 4)
        return {"bytes": read, "flops": 2 * d * hq * sum(L * n for L, n in zip(lens, news))}
    n, k = c["n"], c["k"]
    if c["first"]:
        # the recent window and the kept share of the rest lie beyond the budget
        recent = min(c["window"], n - k)
        share = max(0, k - c["sinks"] - c["window"]) / max(1, n - c["sinks"] - c["window"])
        moved = recent + share * (n - k - recent)
    else:
        moved = min(n - k, c["window"]) if c["window"] >= n - k else n - k
    return {"bytes": B * hkv * (8 * n + 2 * moved * (4 * d + 8)), "flops": 0}


# ------------------------------------------------------------------- exact


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    B, hq, hkv, d, T = c["B"], c["hq"], c["hkv"], c["d"], c["gamma"] + 1
    G = hq // hkv
    if c["op"] == "evict":
        return _exact_evict(s)
    if c["op"] == "accumulate":
        return _exact_accumulate(s)
    o = torch.zeros((B, T, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, hq), -math.inf, dtype=torch.float64, device="cuda")
    lens = _lengths(c)
    t = torch.arange(T, device="cuda")
    for b, L in enumerate(lens):
        if c["op"] == "window":
            j = torch.arange(L + T, device="cuda")
            i = (L + t).view(-1, 1)
            seen = (j <= i) & ((j > i - c["window"]) | (j < c["sinks"]))
            use = seen.any(dim=0).nonzero().squeeze(-1)
            seen = seen[:, use]
        for g in range(hkv):
            k = torch.cat([s["k"][b, g, :L], s["kb"][b, g]])
            v = torch.cat([s["v"][b, g, :L], s["vb"][b, g]])
            if c["op"] == "window":
                k, v = k[use], v[use]
            else:
                k = torch.cat([s["pk"][0, g, :c["P"]], k])
                v = torch.cat([s["pv"][0, g, :c["P"]], v])
                seen = torch.cat([torch.ones((T, c["P"] + L), dtype=torch.bool, device="cuda"),
                                  torch.ones((T, T), device="cuda").tril().bool()], dim=1)
            if k.shape[0] == 0:
                continue
            k, v = k.double(), v.double()
            q = s["q"][b, :, g * G:(g + 1) * G].double()                     # [T, G, d]
            z = torch.einsum("tgd,nd->tgn", q, k) * d ** -0.5
            z = z.masked_fill(~seen.unsqueeze(1), -math.inf)
            l = torch.logsumexp(z, dim=-1)
            e = torch.exp(z - l.unsqueeze(-1)).nan_to_num(0.0)
            o[b, :, g * G:(g + 1) * G] = torch.einsum("tgn,nd->tgd", e, v)
            lse[b, :, g * G:(g + 1) * G] = l
    return o, lse


def _exact_accumulate(s):
    c = s["c"]
    G, d = c["hq"] // c["hkv"], c["d"]
    w, pos = s["weight"].double(), s["pos"].clone()
    for b, (L, n, seen) in enumerate(zip(s["seq_len"].tolist(), s["n_new"].tolist(), s["n_seen"].tolist())):
        w[b, :, L - n:L] = 0.0
        pos[b, :, L - n:L] = torch.arange(seen - n, seen, device="cuda")
        for g in range(c["hkv"]):
            k = s["k"][b, g, :L].double()
            for t in range(n):
                upto = L - n + t + 1
                z = k[:upto] @ s["q"][b, t, g * G:(g + 1) * G].double().T / math.sqrt(d)
                w[b, g, :upto] += torch.exp(z - s["lse"][b, t, g * G:(g + 1) * G].double()).sum(dim=1)
    return w, pos


def _exact_evict(s):
    c = s["c"]
    n, k = c["n"], c["k"]
    seen = s["n_seen"].tolist()
    out = {"k": s["ks"][0][:, :, :k].double(), "v": s["vs"][0][:, :, :k].double(),
           "weight": s["weights"][0][..., :k].double(), "pos": s["poss"][0][..., :k].clone(),
           "seq_len": torch.full_like(s["seq_len"], min(n, k))}
    w, pos = s["weights"][0].cpu().numpy(), s["poss"][0].cpu().numpy()
    for b in range(c["B"]):
        for g in range(c["hkv"]):
            wl, pl = w[b, g, :n].astype(np.float64), pos[b, g, :n]
            rest = (pl >= c["sinks"]) & (pl < seen[b] - c["window"])   # not protected
            kept = np.lexsort((np.arange(n), np.where(rest, -wl, 0.0), rest))[:k]
            holes = np.setdiff1d(np.arange(k), kept)
            moves = np.sort(kept[kept >= k])
            at = torch.tensor(holes, dtype=torch.long, device="cuda")
            of = torch.tensor(moves, dtype=torch.long, device="cuda")
            out["k"][b, g, at] = s["ks"][0][b, g, of].double()
            out["v"][b, g, at] = s["vs"][0][b, g, of].double()
            out["weight"][b, g, at] = s["weights"][0][b, g, of].double()
            out["pos"][b, g, at] = s["poss"][0][b, g, of]
    return out
