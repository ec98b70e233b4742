"""Cases and plain forms of the paged-cache operators: block tables and slot
maps from request lengths, head norms with the position rotation and the cache
write, and attention of a ragged batch of new tokens over the paged cache.

``run`` computes an operator in elementary torch operations in fp32 (``own``
false) or through the framework's entry points (``own`` true).  ``exact``
restates each definition in float64 (whole numbers: with numpy).

Shapes: ``hq``/``hkv``/``d`` are 64/8/128 (the target model of the workloads
in ``synth``) or 14/2/64 (its draft model).  ``page`` rows make a page of the
cache ``[pages][hkv][page][d]``; with ``token_major`` its memory holds
``[pages][page][hkv][d]``.  Context lengths spread evenly from ``L`` down to
``L - L * ragged``.
"""
import math

import numpy as np
import torch

own = False

_TARGET = {"hq": 64, "hkv": 8, "d": 128}
_DRAFT = {"hq": 14, "hkv": 2, "d": 64}


def listed():
    return [
        # The tables of a small batch before a step of single tokens: latency counts.
        dict(name="map_tokens", op="map", B=16, page=16, n=1, nrag=0.0, L=32768, ragged=0.5, back=0, done=0,
             spare=1.0, pad=0),
        # A large batch: prompt chunks and finished requests whose pages come back.
        dict(name="map_chunks", op="map", B=256, page=16, n=256, nrag=0.9, L=8192, ragged=1.0, back=5, done=7,
             spare=1.0, pad=1000),
        # One token of the target model through one layer: the smallest call.
        dict(_TARGET, name="rope_token", op="rope", N=1, run=1, rot=128, interleaved=False, norm=True, fused=True,
             page=16, token_major=False, far=32768, pad=0),
        # The draft blocks of a batch, keys far into long contexts.
        dict(_TARGET, name="rope_blocks", op="rope", N=96, run=6, rot=128, interleaved=False, norm=True, fused=True,
             page=64, token_major=False, far=1 << 20, pad=0),
        # Prompt chunks of a batch.
        dict(_TARGET, name="rope_chunks", op="rope", N=16384, run=2048, rot=128, interleaved=False, norm=True,
             fused=True, page=64, token_major=False, far=131072, pad=0),
        # The draft model's heads: half of each head rotated, interleaved pairs,
        # an odd number of rows, padding rows, token-major pages.
        dict(_DRAFT, name="rope_odd", op="rope", N=5003, run=501, rot=32, interleaved=True, norm=True, fused=False,
             page=16, token_major=True, far=40000, pad=3),
        # One token of one request: the smallest attention call.
        dict(_TARGET, name="paged_token", op="paged", B=1, n=1, nrag=0.0, L=4096, ragged=0.0, chunk=0, idle=0,
             page=16, token_major=False, pad=0),
        # Draft blocks of a batch of long requests.
        dict(_TARGET, name="paged_blocks", op="paged", B=16, n=6, nrag=0.0, L=32768, ragged=0.5, chunk=0, idle=0,
             page=64, token_major=False, pad=0),
        # Single tokens of many requests with one prompt chunk among them.
        dict(_TARGET, name="paged_mixed", op="paged", B=33, n=1, nrag=0.0, L=16384, ragged=0.8, chunk=1000, idle=0,
             page=16, token_major=False, pad=24),
        # Prompts of a batch from their first token on, of very different lengths.
        dict(_TARGET, name="paged_prompts", op="paged", B=8, n=2048, nrag=0.9, L=0, ragged=0.0, chunk=0, idle=0,
             page=64, token_major=False, pad=0),
        # The largest: a chunk of a long prompt behind the part that is cached.
        dict(_TARGET, name="paged_chunk", op="paged", B=1, n=4096, nrag=0.0, L=28672, ragged=0.0, chunk=0, idle=0,
             page=128, token_major=False, pad=0),
        # The draft model's heads, odd sizes throughout, idle requests and padding.
        dict(_DRAFT, name="paged_odd", op="paged", B=11, n=77, nrag=1.0, L=5003, ragged=0.95, chunk=0, idle=4,
             page=32, token_major=True, pad=13),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["map", "rope", "rope", "paged", "paged", "paged"])
    if op == "map":
        n = rng.choice([1, 1, 2, 6, _logu(rng, 1, 512)])
        B = _logu(rng, 1, min(512, 65536 // n))
        return dict(op=op, B=B, page=rng.choice([16, 32, 64, 128, 256]), n=n, nrag=rng.choice([0.0, 0.5, 1.0]),
                    L=_logu(rng, 1, 8192), ragged=rng.choice([0.0, 0.5, 1.0]), back=rng.choice([0, 1, 5]),
                    done=rng.choice([0, 2, 5]), spare=rng.choice([1.0, 1.0, 0.5, 0.0]),
                    pad=rng.choice([0, 1, 37]))
    shape = dict(rng.choice([_TARGET, _TARGET, _DRAFT]))
    if rng.random() < 0.3:   # other group sizes: one to sixteen query heads per KV head
        shape["hkv"] = rng.choice([1, 2, 4, 8])
        shape["hq"] = shape["hkv"] * rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
    page = rng.choice([16, 32, 64, 128, 256])
    c = dict(shape, op=op, page=page, token_major=rng.random() < 0.3, pad=rng.choice([0, 0, 1, 37]))
    if op == "rope":
        N = _logu(rng, 1, min(16384, 16384 * 80 // (c["hq"] + 2 * c["hkv"])))
        # long batches come in runs of a page at least, so that the pool stays near what they fill
        c.update(N=N, run=max(_logu(rng, 1, min(N, 4096)), page if N > 256 else 1),
                 rot=rng.choice([c["d"], c["d"], c["d"] // 2, 16]), interleaved=rng.random() < 0.3,
                 norm=rng.random() < 0.8, fused=rng.random() < 0.5, far=_logu(rng, 8192, 1 << 20))
        c["pad"] = min(c["pad"], N - 1)
        return c
    most = max(_pairs(x) * x["hq"] * x["d"] for x in listed() if x["op"] == "paged") // (c["hq"] * c["d"])
    n = rng.choice([1, 1, 2, 6, _logu(rng, 1, 2048)])
    B = _logu(rng, 1, 32)
    c.update(B=B, n=n, nrag=rng.choice([0.0, 0.5, 1.0]), L=0 if rng.random() < 0.15 else _logu(rng, 1, 32768),
             ragged=rng.choice([0.0, 0.5, 1.0]), chunk=rng.choice([0, 0, 0, _logu(rng, 2, 1024)]),
             idle=rng.choice([0, 0, 3]))
    while _pairs(c) > most:
        c["B"] = max(1, c["B"] // 2)
        c["n"] = max(1, c["n"] * 2 // 3)
    return c


def _spread(top, ragged, B):
    """B numbers from top down to top - top * ragged."""
    low = top - int(top * ragged)
    return [top - (top - low) * b // max(1, B - 1) for b in range(B)]


def _requests(c):
    """Context lengths and new tokens of a case's requests."""
    B = c["B"]
    ctx = _spread(c["L"], c["ragged"], B)
    # the longest chunk behind the shortest context, one token at least
    new = [max(1, x) for x in reversed(_spread(c["n"], c["nrag"], B))]
    if c.get("chunk"):
        new[B // 2] = c["chunk"]
    if c.get("idle"):
        new = [0 if b % c["idle"] == c["idle"] - 1 else x for b, x in enumerate(new)]
    if c.get("done"):
        for b in range(c["done"] - 1, B, c["done"]):
            ctx[b] = new[b] = 0
    return ctx, new


def _pairs(c):
    return sum(n * L + n * (n + 1) // 2 for L, n in zip(*_requests(c)))


def _pages(rows, page):
    return (rows + page - 1) // page


def _gen(seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)

    def normal(*shape, scale=1.0):
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
        return (x * scale).to(torch.bfloat16)
    return g, normal


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device="cuda")


def _cache(normal, c, pages):
    """A pool of pages [pages][hkv][page][d]."""
    if c["token_major"]:
        return normal(pages, c["page"], c["hkv"], c["d"]).transpose(1, 2)
    return normal(pages, c["hkv"], c["page"], c["d"])


def _tables(g, counts, width, pages):
    """Tables [len(counts)][width] that hold random pages of the pool, counts[b]
    of them for request b, and the pages that are left, in any order."""
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(counts), width), dtype=torch.int32, device="cuda")
    used = torch.arange(width, device="cuda") < torch.as_tensor(counts, device="cuda").view(-1, 1)
    table[used] = order[:sum(counts)]
    return table, order[sum(counts):]


def prepare(case, seed):
    c = dict(case)
    g, normal = _gen(seed)
    s = {"c": c}
    if c["op"] == "map":
        ctx, new = _requests(c)
        B, page = c["B"], c["page"]
        # pages held: of the rows in the cache and of `back` draft rows that were
        # rejected since; a finished request still holds its context's
        was = _spread(c["L"], c["ragged"], B)
        held = [_pages(w + c["back"], page) for w in was]
        take = sum(max(0, _pages(L + n, page) - h) for L, n, h in zip(ctx, new, held))
        width = max(max(held), max(_pages(L + n, page) for L, n in zip(ctx, new)), 1) + 2
        pages = sum(held) + int(take * c["spare"]) + (7 if c["spare"] >= 1.0 else 0) + 1
        table, left = _tables(g, held, width, pages)
        n_free = pages - sum(held) - 1           # one page stays reserved
        N = sum(new) + c["pad"]
        s.update(N=max(N, 1), width=width, seq_len=_i32(ctx), n_new=_i32(new), table=table,
                 free=torch.cat([left[:n_free], torch.zeros(pages - n_free, dtype=torch.int32, device="cuda")]))
        # pages held and free side by side, so that a pass restores both at once
        s["meta0"] = _i32(held + [n_free])
        s["meta"] = s["meta0"].clone()
        s.update(held=s["meta"][:B], n_free=s["meta"][B:])
        s["out"] = [torch.zeros(k, dtype=torch.int32, device="cuda") for k in (B + 1, B, s["N"], s["N"])]
    elif c["op"] == "rope":
        N, hq, hkv, d, page, run = c["N"], c["hq"], c["hkv"], c["d"], c["page"], c["run"]
        # runs of consecutive positions, each of a request of its own
        reqs = (N + run - 1) // run
        rng = np.random.default_rng(seed)
        first = rng.integers(max(1, c["far"] // 2), c["far"] - run + 1, size=reqs) if c["far"] > 2 * run else np.zeros(reqs, int)
        i = np.arange(N)
        pos = first[i // run] + i % run
        width = (run + page - 2) // page + 1
        pages = reqs * width
        at = rng.permutation(pages).reshape(reqs, width)
        slot = at[i // run, pos // page - first[i // run] // page] * page + pos % page
        if c["pad"]:
            slot[-c["pad"]:] = -1                # rows that belong to no request
            pos[-c["pad"]:] = 0
        if c["fused"]:                           # one projection's output
            x = normal(N, hq + 2 * hkv, d)
            q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        else:
            q, k, v = normal(N, hq, d), normal(N, hkv, d), normal(N, hkv, d)
        s.update(q=q, k=k, v=v, pos=_i32(pos), slot=_i32(slot),
                 q_w=(1 + normal(d, scale=0.2)) if c["norm"] else None,
                 k_w=(1 + normal(d, scale=0.2)) if c["norm"] else None,
                 inv_freq=torch.tensor([1e6 ** (-2 * j / c["rot"]) for j in range(c["rot"] // 2)],
                                       dtype=torch.float32, device="cuda"),
                 kc=_cache(normal, c, pages), vc=_cache(normal, c, pages),
                 q_out=torch.empty((N, hq, d), dtype=torch.bfloat16, device="cuda"))
    else:
        ctx, new = _requests(c)
        kv = [L + n if n else 0 for L, n in zip(ctx, new)]
        counts = [_pages(x, c["page"]) for x in kv]
        width, pages = max(max(counts), 1), sum(counts) + 3
        table, _ = _tables(g, counts, width, pages)
        N = sum(new) + c["pad"]
        s.update(N=N, width=width, kv=kv, new=new, table=table, kv_len=_i32(kv),
                 cu=_i32(np.concatenate([[0], np.cumsum(new)])),
                 q=normal(N, c["hq"], c["d"], scale=2.0), kc=_cache(normal, c, pages), vc=_cache(normal, c, pages),
                 o=torch.zeros((N, c["hq"], c["d"]), dtype=torch.bfloat16, device="cuda"),
                 lse=torch.zeros((N, c["hq"]), dtype=torch.float32, device="cuda"))
    return s


# ------------------------------------------------------------- plain forms


def _map(s):
    c = s["c"]
    B, N, page = c["B"], s["N"], c["page"]
    L, n, held, table, free = s["seq_len"].long(), s["n_new"].long(), s["held"].long(), s["table"], s["free"]
    need = (L + n + page - 1) // page
    rel, take = (held - need).clamp(min=0), (need - held).clamp(min=0)
    avail = s["n_free"].long() + rel.sum()
    served = (take == 0) | (take.cumsum(0) <= avail)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), n.cumsum(0)])
    # given back: pushed in order of request, then of table position
    j = torch.arange(s["width"], device="cuda")
    back = (j >= need.view(-1, 1)) & (j < held.view(-1, 1))
    rank = back.flatten().cumsum(0) - 1
    spot = torch.where(back.flatten(), s["n_free"].long() + rank, free.numel())   # one past the end: nowhere
    room = torch.cat([free, free.new_zeros(1)])
    room[spot] = table.flatten()
    free.copy_(room[:-1])
    # taken: from the top, in the same order
    grow = (j >= held.view(-1, 1)) & (j < need.view(-1, 1)) & served.view(-1, 1)
    rank = grow.flatten().cumsum(0) - 1
    page_of = free[(avail - 1 - rank).clamp(min=0)].view(B, -1)
    table.copy_(torch.where(grow, page_of, table))
    s["n_free"].copy_(avail - torch.where(served, take, 0).sum())
    s["held"].copy_(torch.where(served, need, held))
    i = torch.arange(N, device="cuda")
    b = torch.searchsorted(cu[1:], i, right=True).clamp(max=B - 1)
    real = i < cu[B]
    pos = torch.where(real, L[b] + i - cu[b], 0)
    slot = table[b, (pos // page).clamp(max=s["width"] - 1)].long() * page + pos % page
    out = s["out"]
    out[0].copy_(cu)
    out[1].copy_(torch.where(served, L + n, 0))
    out[2].copy_(torch.where(real & served[b], slot, -1))
    out[3].copy_(pos)
    return _mapped(s)


def _mapped(s):
    """What a pass over the tables leaves."""
    return {"table": s["table"], "held": s["held"], "free": s["free"], "n_free": s["n_free"], "cu": s["out"][0],
            "kv_len": s["out"][1], "slot": s["out"][2], "pos": s["out"][3]}


def _turned(x, w, cos, sin, c):
    """Normed and rotated heads [N, h, d] in fp32."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + 1e-6) * w.float()
    r = c["rot"]
    y = x.clone()
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * cos - b * sin, b * cos + a * sin
    return y.to(torch.bfloat16)


def _rope(s):
    c = s["c"]
    angle = s["pos"].double().view(-1, 1) * s["inv_freq"].double()     # 32 bits lose the turns of far positions
    cos, sin = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    s["q_out"].copy_(_turned(s["q"], s["q_w"], cos, sin, c))
    n = c["N"] - c["pad"]                        # the padding rows, which have no slot, come last
    at, row = s["slot"][:n].long() // c["page"], s["slot"][:n].long() % c["page"]
    s["kc"][at, :, row] = _turned(s["k"], s["k_w"], cos, sin, c)[:n]
    s["vc"][at, :, row] = s["v"][:n]
    return s["q_out"], s["kc"], s["vc"]


def _paged(s):
    c = s["c"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    G, at = hq // hkv, 0
    for b, (L, n) in enumerate(zip(s["kv"], s["new"])):
        if n == 0:
            continue
        ids = s["table"][b, :_pages(L, c["page"])].long()
        k = s["kc"][ids].transpose(0, 1).reshape(hkv, -1, d)[:, :L].float()
        v = s["vc"][ids].transpose(0, 1).reshape(hkv, -1, d)[:, :L].float()
        step = max(1, (1 << 29) // (hq * L))     # queries at a time: 2 GB of scores
        for t0 in range(0, n, step):
            t1 = min(n, t0 + step)
            q = s["q"][at + t0:at + t1].float().view(t1 - t0, hkv, G, d).permute(1, 0, 2, 3).reshape(hkv, -1, d)
            x = (q @ k.transpose(-1, -2)).view(hkv, t1 - t0, G, L)
            x /= math.sqrt(d)
            i = L - n + torch.arange(t0, t1, device="cuda").view(-1, 1)
            x.masked_fill_((torch.arange(L, device="cuda") > i).unsqueeze(1), -math.inf)
            m = x.amax(dim=-1, keepdim=True)
            e = torch.exp(x - m)
            total = e.sum(dim=-1, keepdim=True)
            o = (e.view(hkv, -1, L) @ v).view(hkv, t1 - t0, G, d) / total
            s["o"][at + t0:at + t1] = o.permute(1, 0, 2, 3).reshape(-1, hq, d).to(torch.bfloat16)
            s["lse"][at + t0:at + t1] = (m + torch.log(total)).squeeze(-1).permute(1, 0, 2).reshape(-1, hq)
        at += n
    return s["o"], s["lse"]


# ------------------------------------------------- the framework's operators


def _call(s):
    """The prepared call that a user's program keeps and repeats."""
    import sparse_kv_verify_gb300 as dk
    c = s["c"]
    if c["op"] == "rope":
        r = dk.Rope(rot=c["rot"], interleaved=c["interleaved"], eps=1e-6)
        return dk.NormRopeCall(r, s["q"], s["k"], s["v"], s["q_w"], s["k_w"], s["inv_freq"], s["pos"], s["slot"],
                               s["kc"], s["vc"], s["q_out"])
    _, new = _requests(c)
    bt = dk.Batch(B=c["B"], N=s["N"], max_new=max(1, max(new)), max_pages=s["width"])
    if c["op"] == "map":
        return dk.PageMapCall(bt, c["page"], s["seq_len"], s["n_new"], s["table"], s["held"], s["free"],
                              s["n_free"], *s["out"])
    return dk.PagedAttnCall(bt, s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["kv_len"], s["o"], s["lse"])


_PLAIN = {"map": _map, "rope": _rope, "paged": _paged}


def run(state):
    s = state
    op = s["c"]["op"]
    if op == "map":
        # the counts before the pass again (what it pushes and takes stays the same)
        s["meta"].copy_(s["meta0"])
    if not own:
        return _PLAIN[op](s)
    if "call" not in s:
        s["call"] = _call(s)
    out = s["call"]()
    if op == "map":
        return _mapped(s)
    return (out, s["kc"], s["vc"]) if op == "rope" else out


# ------------------------------------------------------------------- work


def work(case):
    c = case
    if c["op"] == "map":
        ctx, new = _requests(c)
        was = _spread(c["L"], c["ragged"], c["B"])
        held = [_pages(w + c["back"], c["page"]) for w in was]
        need = [_pages(L + n, c["page"]) for L, n in zip(ctx, new)]
        moved = sum(abs(a - b) for a, b in zip(held, need))
        touched = sum(_pages(L % c["page"] + n, c["page"]) for L, n in zip(ctx, new) if n)
        return {"bytes": 24 * c["B"] + 8 * moved + 4 * touched + 8 * (sum(new) + c["pad"]), "flops": 0}
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    if c["op"] == "rope":
        return {"bytes": c["N"] * ((hq + 2 * hkv) * d * 4 + 8), "flops": c["N"] * (hq + hkv) * d * 7}
    ctx, new = _requests(c)
    rows = sum(L + n for L, n in zip(ctx, new) if n)
    return {"bytes": rows * hkv * d * 4 + sum(new) * hq * (4 * d + 4), "flops": 4 * _pairs(c) * hq * d}


# ------------------------------------------------------------------- exact


def exact(case, seed):
    s = prepare(case, seed)
    return {"map": _exact_map, "rope": _exact_rope, "paged": _exact_paged}[case["op"]](s)


def _exact_map(s):
    c = s["c"]
    page, N = c["page"], s["N"]
    host = {k: s[k].cpu().numpy().astype(np.int64) for k in ("seq_len", "n_new", "table", "free", "held", "n_free")}
    table, free, held, top = host["table"], host["free"], host["held"], int(host["n_free"][0])
    need = [-(-(int(L) + int(n)) // page) for L, n in zip(host["seq_len"], host["n_new"])]
    for b, want in enumerate(need):              # give back
        for j in range(want, held[b]):
            free[top] = table[b, j]
            top += 1
        held[b] = min(held[b], want)
    kv_len, cu = [], [0]
    slot, pos = np.full(N, -1), np.zeros(N, np.int64)
    short = False                                # from the first that finds too few pages on, none gets any
    for b, want in enumerate(need):
        L, n = int(host["seq_len"][b]), int(host["n_new"][b])
        more = want - held[b]
        short = short or more > top
        served = more == 0 or not short
        if served:
            for _ in range(more):
                top -= 1
                table[b, held[b]] = free[top]
                held[b] += 1
        for t in range(n):
            pos[cu[-1] + t] = L + t
            if served:
                slot[cu[-1] + t] = table[b, (L + t) // page] * page + (L + t) % page
        kv_len.append(L + n if served else 0)
        cu.append(cu[-1] + n)
    return {"table": _i32(table), "held": _i32(held), "free": _i32(free), "n_free": _i32([top]), "cu": _i32(cu),
            "kv_len": _i32(kv_len), "slot": _i32(slot), "pos": _i32(pos)}


def _exact_rope(s):
    c = s["c"]
    r, d = c["rot"], c["d"]
    # the rotation as complex products: z e^(i t)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["pos"].double().view(-1, 1, 1) * s["inv_freq"].double())
    index = torch.arange(r, device="cuda").view(r // 2, 2) if c["interleaved"] else torch.arange(r, device="cuda").view(2, r // 2).T

    def heads(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x * x).sum(dim=-1, keepdim=True) / d + 1e-6) * w.double()
        z = torch.view_as_complex(x[..., index].contiguous()) * turn
        y = x.clone()
        y[..., index] = torch.view_as_real(z)
        return y
    kc, vc = s["kc"].double(), s["vc"].double()
    rows = heads(s["k"], s["k_w"])
    use = (s["slot"] >= 0).nonzero().squeeze(-1)
    where = s["slot"][use].long()
    kc[where // c["page"], :, where % c["page"]] = rows[use]
    vc[where // c["page"], :, where % c["page"]] = s["v"][use].double()
    return heads(s["q"], s["q_w"]), kc, vc


def _exact_paged(s):
    c = s["c"]
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    G = hq // hkv
    o, lse = s["o"].double(), s["lse"].double()
    cu = s["cu"].tolist()
    for b, L in enumerate(s["kv"]):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        row = torch.arange(L, device="cuda")
        at, r = s["table"][b].long()[row // page], row % page
        for g in range(hkv):
            k, v = s["kc"][at, g, r].double(), s["vc"][at, g, r].double()
            for t0 in range(0, n, 512):
                t1 = min(n, t0 + 512)
                m = L - n + t1                   # rows that some query of these sees
                q = s["q"][cu[b] + t0:cu[b] + t1, g * G:(g + 1) * G].double()
                z = torch.einsum("tgd,nd->tgn", q, k[:m]) * d ** -0.5
                hidden = row[:m] > L - n + torch.arange(t0, t1, device="cuda").view(-1, 1, 1)
                z = z.masked_fill_(hidden, -math.inf)
                l = torch.logsumexp(z, dim=-1)
                z -= l.unsqueeze(-1)
                o[cu[b] + t0:cu[b] + t1, g * G:(g + 1) * G] = torch.einsum("tgn,nd->tgd", z.exp_(), v[:m])
                lse[cu[b] + t0:cu[b] + t1, g * G:(g + 1) * G] = l
    return o, lse
