"""The prompt and page operators of the paged KV cache, as measured cases.

Three operators that work on the cache the ISD step reads:

* ``chunk``: attention of a chunk of new tokens per request over the paged
  cache (the chunk's keys and values are appended to their pages first); a
  chunk of one token per request is plain decoding;
* ``fork``: a new batch made of an old one: a request may go on, be continued
  by several children (whole pages shared, the part-filled last page copied),
  change its slot or be dropped, and room is made for the tokens to come;
* ``compact``: the pages still in use move to the front of the pools, so that
  the bump allocator gets the others back.

``run`` computes them with elementary torch operations in 32 bits, or, where
``own`` is true, with the library's calls.
"""
import math
import random

import torch

own = False


def listed():
    q3 = dict(Hq=32, Hkv=8, D=128)  # the head layout of the benchmark's workloads
    return [
        # one user, one new token behind a short prompt: nothing but latency
        dict(name="decode_1", op="chunk", B=1, P=16, n_lo=1, n_hi=1, ctx_lo=1000, ctx_hi=1000, lens=1, **q3),
        # the benchmark's batch and prefixes, one token per request
        dict(name="decode_32", op="chunk", B=32, P=16, n_lo=1, n_hi=1, ctx_lo=512, ctx_hi=8192, lens=2, **q3),
        # few requests with long contexts: the work must be split over a request's keys
        dict(name="decode_long", op="chunk", B=3, P=64, n_lo=1, n_hi=1, ctx_lo=30000, ctx_hi=50001, lens=3, **q3),
        # a serving batch: requests that decode next to requests that are in their prompts
        dict(name="mixed", op="chunk", B=16, P=16, n_lo=1, n_hi=480, ctx_lo=0, ctx_hi=6000, lens=4, **q3),
        # a whole prompt at once, nothing cached before it
        dict(name="prompt", op="chunk", B=1, P=16, n_lo=2048, n_hi=2048, ctx_lo=0, ctx_hi=0, lens=5, **q3),
        # long prompts in pieces: the largest
        dict(name="prompt_piece", op="chunk", B=4, P=64, n_lo=1900, n_hi=2048, ctx_lo=4096, ctx_hi=8192, lens=6, **q3),
        # a smaller model: 64-wide heads in groups of seven, pages that do not divide a tile
        dict(name="small_heads", op="chunk", B=5, P=24, n_lo=3, n_hi=333, ctx_lo=0, ctx_hi=2999, lens=7, Hq=14, Hkv=2, D=64),
        # one answer continued in four ways, one layer's cache
        dict(name="fork_4", op="fork", B=1, fan=4, keep=1.0, reserve=7, layers=1, Hkv=8, D=128, P=16, ctx_lo=1000, ctx_hi=1000, lens=8),
        # a batch of the benchmark's size re-made: some answers end, others go on in up to four ways, at full depth
        dict(name="fork_batch", op="fork", B=32, fan=4, keep=0.6, reserve=7, layers=36, Hkv=8, D=128, P=16, ctx_lo=100, ctx_hi=700, lens=9),
        # a small cache, one layer
        dict(name="compact_1", op="compact", B=8, live=0.5, layers=1, Hkv=8, D=128, P=16, ctx_lo=100, ctx_hi=600, lens=10),
        # full depth, half of the requests gone
        dict(name="compact_deep", op="compact", B=32, live=0.5, layers=36, Hkv=8, D=128, P=16, ctx_lo=200, ctx_hi=1500, lens=11),
        # few wide pages of odd size
        dict(name="compact_pages", op="compact", B=21, live=0.7, layers=12, Hkv=2, D=64, P=100, ctx_lo=1, ctx_hi=4001, lens=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    what = rng.random()
    lens = rng.randrange(1 << 20)
    if what < 0.6:
        while True:
            Hq, Hkv, D = rng.choice([(32, 8, 128), (16, 8, 128), (28, 4, 128), (12, 12, 128), (64, 8, 128), (14, 2, 64), (32, 8, 64), (9, 3, 64)])
            B = _log_int(rng, 1, 64)
            n_hi = rng.choice([1, 1, _log_int(rng, 2, 64), _log_int(rng, 64, 2048), _log_int(rng, 64, 2048)])
            n_lo = 1 if rng.random() < 0.5 else n_hi
            ctx_hi = _log_int(rng, 8, 40000)
            ctx_lo = 0 if rng.random() < 0.5 else ctx_hi // 2
            P = rng.choice([8, 16, 16, 32, 64, 128, 24, 100, 256, 1, 5])
            case = dict(op="chunk", B=B, P=P, n_lo=n_lo, n_hi=n_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, lens=lens, Hq=Hq, Hkv=Hkv, D=D)
            w = work(case)
            padded = B * Hq * n_hi * (ctx_hi + n_hi) * 4
            if w["flops"] <= 8e11 and padded <= 10e9 and w["bytes"] <= 4e9:
                return case
    D, Hkv = rng.choice([(128, 8), (128, 4), (128, 1), (64, 2), (64, 8)])
    P = rng.choice([8, 16, 16, 32, 64, 24, 100, 1, 5])
    while True:
        B, layers = _log_int(rng, 1, 64), _log_int(rng, 1, 36)
        ctx_hi = _log_int(rng, 16, 4000)
        ctx_lo = rng.choice([0, ctx_hi // 3])
        if B * ctx_hi * layers * Hkv * D * 4 > 4e9:
            continue
        if what < 0.8:
            return dict(op="fork", B=B, fan=rng.randint(1, 6), keep=rng.choice([0.4, 0.8, 1.0]), reserve=rng.choice([0, 1, 7, 300]),
                        layers=layers, Hkv=Hkv, D=D, P=P, ctx_lo=ctx_lo, ctx_hi=ctx_hi, lens=lens)
        if B >= 3:
            return dict(op="compact", B=B, live=rng.choice([0.3, 0.5, 0.8]), layers=layers, Hkv=Hkv, D=D, P=P,
                        ctx_lo=max(ctx_lo, 1), ctx_hi=ctx_hi, lens=lens)


def _lengths(case):
    """Cached lengths and new tokens of the requests: whole numbers that the case fixes."""
    rng = random.Random(case["lens"])
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    if case["op"] != "chunk":
        return ctx, None
    return ctx, [_log_int(rng, case["n_lo"], case["n_hi"]) for _ in range(case["B"])]


def _parents(case):
    """Of each slot of the new batch: the request it continues, or -1."""
    rng = random.Random(case["lens"] + 1)
    kept = [b for b in range(case["B"]) if rng.random() < case["keep"]] or [0]
    par = [b for b in kept for _ in range(rng.randint(1, case["fan"]) if case["B"] > 1 else case["fan"])]
    if case["keep"] < 1:
        par.append(-1)
    rng.shuffle(par)
    return par


def _kept(case):
    """Which requests of a cache to compact are still there: at least one goes and one stays."""
    rng = random.Random(case["lens"] + 2)
    live = [rng.random() < case["live"] for _ in range(case["B"])]
    live[0], live[-1] = False, True
    return live


def _ceil(a, b):
    return -(-a // b)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    normal = lambda *s: torch.randn(*s, generator=gen, device=dev, dtype=torch.bfloat16)  # noqa: E731
    B, P, Hkv, D = case["B"], case["P"], case["Hkv"], case["D"]
    ctx, n = _lengths(case)
    if case["op"] == "chunk":
        used = [_ceil(c + m, P) for c, m in zip(ctx, n)]
    else:
        used = [_ceil(c, P) for c in ctx]
    s = {"op": case["op"], "P": P}
    cols = max(used) + 1
    first = 0  # pages of the pool that are handed out
    if case["op"] == "fork":
        par = _parents(case)
        cols = max(used) + _ceil(case["reserve"], P) + 1
        first = sum(used)
        pages = first + sum(_ceil(ctx[p] + case["reserve"], P) - ctx[p] // P + 1 for p in par if p >= 0) + 1
    elif case["op"] == "compact":
        pages = max(1, sum(used))
    else:
        pages = sum(used) + 3
    # a cache that has seen requests come and go: pages in no order
    perm = torch.randperm(first or pages, generator=gen, device=dev)[:sum(used)].to(torch.int32)
    table = torch.full((B, cols), -1, dtype=torch.int32, device=dev)
    at = torch.arange(cols, device=dev)[None] < torch.tensor(used, device=dev)[:, None]
    table[at] = perm
    s["page_table"], s["kv_len"] = table, ints(ctx)
    if case["op"] == "chunk":
        Hq, T = case["Hq"], sum(n)
        s["q"], s["k_new"], s["v_new"] = normal(T, Hq, D), normal(T, Hkv, D), normal(T, Hkv, D)
        s["k_pool"], s["v_pool"] = normal(pages, P, Hkv, D), normal(pages, P, Hkv, D)
        starts = [0]
        for m in n:
            starts.append(starts[-1] + m)
        s["q_start"] = ints(starts)
        s["n_max"], s["keys_max"] = max(n), max(c + m for c, m in zip(ctx, n))
        s["out"] = torch.empty(T, Hq * D, dtype=torch.bfloat16, device=dev)
        if own:
            from speculative_verification_isd_b200 import isd
            d = isd.make_dims(B, 1, Hq, Hkv, D, 1, P, pages, cols)
            s["call"] = isd.ChunkCall(d, s["q"], s["k_new"], s["v_new"], s["k_pool"], s["v_pool"], table, s["kv_len"], s["q_start"],
                                      s["out"], isd.alloc_chunk_workspace(d, T))
        return s
    s["pool"] = normal(2 * case["layers"], pages, P, Hkv, D)
    if case["op"] == "fork":
        s["parent"], s["reserve"] = ints(par), ints([case["reserve"]] * len(par))
        s["pages_used"], s["next_free"] = ints(used), ints([first])
        s["next_kv_len"], s["next_pages_used"] = ints([0] * len(par)), ints([0] * len(par))
        s["next_table"] = torch.empty(len(par), cols, dtype=torch.int32, device=dev)
    else:
        s["pages_used"] = ints([u if k else 0 for u, k in zip(used, _kept(case))])
        s["next_table"] = torch.empty_like(table)
    s["next_free_out"] = ints([0])
    if own:
        from speculative_verification_isd_b200 import isd
        s["dims"] = isd.make_dims(B, 1, Hkv, Hkv, D, 1, P, pages, cols)
        s["pools"] = isd.pool_array(s["dims"], s["pool"].unbind(0))
        if case["op"] == "compact":
            s["ws"] = isd.alloc_pages_workspace(s["dims"])
    return s


def _chunk(s):
    q, kv_len, start, table, P = s["q"], s["kv_len"].long(), s["q_start"].long(), s["page_table"].long(), s["P"]
    (T, Hq, D), Hkv, B = q.shape, s["k_new"].shape[1], kv_len.shape[0]
    n = start[1:] - start[:-1]
    req = torch.repeat_interleave(torch.arange(B, device=q.device), n, output_size=T)
    i = torch.arange(T, device=q.device) - start[req]
    pos = kv_len[req] + i
    page = table[req, pos // P]
    s["k_pool"][page, pos % P] = s["k_new"]
    s["v_pool"][page, pos % P] = s["v_new"]
    at = torch.arange(s["keys_max"], device=q.device)
    page = table[:, at // P].clamp(min=0)
    k = s["k_pool"][page, at % P].permute(0, 2, 3, 1).float()  # [B, Hkv, D, keys]
    v = s["v_pool"][page, at % P].permute(0, 2, 1, 3).float()  # [B, Hkv, keys, D]
    rows = torch.zeros(B, s["n_max"], Hq, D, device=q.device)
    rows[req, i] = q.float()
    G = Hq // Hkv
    rows = rows.view(B, s["n_max"], Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * s["n_max"], D)
    x = torch.matmul(rows * D ** -0.5, k).view(B, Hkv, G, s["n_max"], -1)
    last = kv_len[:, None] + torch.arange(s["n_max"], device=q.device)
    x.masked_fill_((at > last[..., None])[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(x.view(B, Hkv, G * s["n_max"], -1), v).view(B, Hkv, G, s["n_max"], D)
    o = o / x.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4)[req, i]
    s["out"].copy_(o.reshape(T, Hq * D))
    return s["out"], s["k_pool"], s["v_pool"]


def _fork(s):
    P, parent, kv_len, used, table = s["P"], s["parent"].long(), s["kv_len"], s["pages_used"], s["page_table"]
    R = parent.shape[0]
    slot = torch.arange(R, device=parent.device)
    par, there = parent.clamp(min=0), parent >= 0
    first = torch.full((kv_len.shape[0],), R, device=parent.device).scatter_reduce(0, par, torch.where(there, slot, R), "amin")
    first = (first[par] == slot) & there
    kv = kv_len[par]
    whole, tail = kv // P, kv % P
    have = torch.where(first, used[par], whole)
    need = torch.maximum(torch.maximum((kv + s["reserve"] + P - 1) // P, (kv + P - 1) // P), have)
    have, need = have * there, need * there
    new = (need - have).cumsum(0)
    base = s["next_free"] + new - (need - have)
    col = torch.arange(table.shape[1], device=parent.device)[None]
    made = torch.where(col < have[:, None], table[par], base[:, None] + col - have[:, None])
    s["next_table"].copy_(torch.where(col < need[:, None], made, -1))
    s["next_kv_len"].copy_(kv * there)
    s["next_pages_used"].copy_(need)
    s["next_free_out"].copy_(s["next_free"] + new[-1:])
    r, t = ((torch.arange(P, device=parent.device)[None] < tail[:, None]) & (there & ~first)[:, None]).nonzero(as_tuple=True)
    s["pool"][:, base[r], t] = s["pool"][:, table[par[r], whole[r]], t]
    return s["next_kv_len"], s["next_pages_used"], s["next_table"], s["next_free_out"], s["pool"]


def _compact(s):
    table, pages = s["page_table"], s["pool"].shape[1]
    at = torch.arange(pages, device=table.device)
    there = torch.arange(table.shape[1], device=table.device)[None] < s["pages_used"][:, None]
    live = torch.zeros(pages + 1, dtype=torch.bool, device=table.device)
    live[torch.where(there, table, pages).long()] = True
    live = live[:-1]
    count = live.sum()
    src, dst = (live & (at >= count)).nonzero()[:, 0], (~live & (at < count)).nonzero()[:, 0]
    to = at.to(torch.int32)
    to[src] = dst.to(torch.int32)
    s["next_table"].copy_(torch.where(there, to[table.clamp(min=0).long()], -1))
    s["next_free_out"].copy_(count)
    s["pool"][:, dst] = s["pool"][:, src]
    return s["next_table"], s["next_free_out"], s["pool"]


def run(s):
    if own:
        if s["op"] == "chunk":
            s["call"]()
            return s["out"], s["k_pool"], s["v_pool"]
        from speculative_verification_isd_b200 import isd
        if s["op"] == "fork":
            isd.fork_requests(s["dims"], s["parent"], s["kv_len"], s["pages_used"], s["page_table"], s["next_free"], s["pools"],
                              s["next_kv_len"], s["next_pages_used"], s["next_table"], s["next_free_out"], reserve=s["reserve"])
            return s["next_kv_len"], s["next_pages_used"], s["next_table"], s["next_free_out"], s["pool"]
        isd.compact_pages(s["dims"], s["page_table"], s["pages_used"], s["pools"], s["next_table"], s["next_free_out"], s["ws"])
        return s["next_table"], s["next_free_out"], s["pool"]
    return {"chunk": _chunk, "fork": _fork, "compact": _compact}[s["op"]](s)


def work(case):
    ctx, n = _lengths(case)
    P, Hkv, D = case["P"], case["Hkv"], case["D"]
    row = Hkv * D * 2  # one token's keys, or values, of one layer
    if case["op"] == "chunk":
        T = sum(n)
        pairs = sum(m * c + m * (m + 1) // 2 for c, m in zip(ctx, n))
        table = sum(_ceil(c + m, P) for c, m in zip(ctx, n)) * 4 + case["B"] * 8
        # queries in, answers out; cached keys and values in; the new ones in and into their pages
        return {"bytes": 2 * T * case["Hq"] * D * 2 + 2 * sum(ctx) * row + 4 * T * row + table, "flops": 4 * pairs * case["Hq"] * D}
    if case["op"] == "fork":
        par, seen, copied, cells = _parents(case), set(), 0, 0
        for p in par:
            if p < 0:
                continue
            cells += ctx[p] // P
            copied += ctx[p] % P if p in seen else 0
            seen.add(p)
        cols = max(_ceil(c, P) for c in ctx) + _ceil(case["reserve"], P) + 1
        return {"bytes": copied * 2 * case["layers"] * row * 2 + 4 * (cells + len(par) * (cols + 4)), "flops": 0}
    used = [_ceil(c, P) for c in ctx]
    total = sum(used)
    left = sum(u for u, k in zip(used, _kept(case)) if k)
    # pages lie in no order: of the ones in use, the share past the new end moves
    moved = left * (total - left) // total
    return {"bytes": moved * P * row * 2 * case["layers"] * 2 + 4 * (left + case["B"] * (max(used) + 1)), "flops": 0}


def exact(case, seed):
    """Request by request, from the definitions, in 64 bits. A pool holds copies, which have no other value."""
    s = prepare(case, seed)
    P, table, kv = case["P"], s["page_table"].tolist(), s["kv_len"].tolist()
    if case["op"] == "chunk":
        start, dev = s["q_start"].tolist(), s["q"].device
        out = torch.empty(s["out"].shape, dtype=torch.float64, device=dev)
        G = case["Hq"] // case["Hkv"]
        for b, (a, e) in enumerate(zip(start, start[1:])):
            ids = torch.tensor(table[b], device=dev)[: _ceil(kv[b], P)]
            old = lambda pool: pool[ids].reshape(-1, case["Hkv"], case["D"])[: kv[b]]  # noqa: E731
            k = torch.cat([old(s["k_pool"]), s["k_new"][a:e]]).double()
            v = torch.cat([old(s["v_pool"]), s["v_new"][a:e]]).double()
            hidden = torch.arange(k.shape[0], device=dev) > kv[b] + torch.arange(e - a, device=dev)[:, None]
            for h in range(case["Hq"]):
                w = s["q"][a:e, h].double() @ k[:, h // G].T / math.sqrt(case["D"])
                w = torch.softmax(w.masked_fill(hidden, -math.inf), -1)
                out[a:e, h * case["D"]:(h + 1) * case["D"]] = w @ v[:, h // G]
        return out, None, None
    used = s["pages_used"].tolist()
    if case["op"] == "fork":
        free, seen = s["next_free"].item(), set()
        lens, counts, rows = [], [], []
        for p, more in zip(s["parent"].tolist(), s["reserve"].tolist()):
            row = []
            if p >= 0:
                row = table[p][: kv[p] // P] if p in seen else table[p][: used[p]]
                while len(row) * P < kv[p] + more:
                    row = row + [free]
                    free += 1
                seen.add(p)
            lens.append(kv[p] if p >= 0 else 0)
            counts.append(len(row))
            rows.append(row + [-1] * (len(table[0]) - len(row)))
        return torch.tensor(lens), torch.tensor(counts), torch.tensor(rows), torch.tensor([free]), None
    live = sorted({p for row, u in zip(table, used) for p in row[:u]})
    moved = dict(zip([p for p in live if p >= len(live)], [p for p in range(len(live)) if p not in set(live)]))
    rows = [[moved.get(p, p) for p in row[:u]] + [-1] * (len(row) - u) for row, u in zip(table, used)]
    return torch.tensor(rows), torch.tensor([len(live)]), None
