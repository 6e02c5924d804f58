"""The operators of a decode step over a paged key-value cache, as cases that can be timed and compared.

Four operators: the page plan (block tables and slot maps from request lengths), the store of new keys and
values into the cache, the attention of one new token per request over the cache, and the low-rank adapters
that many requests have beside a shared projection.

``run`` computes them in plain torch operations where ``own`` is false, and by the package's entry points
where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
FP8 = torch.float8_e4m3fn
K_SCALE, V_SCALE = 0.0625, 0.03125      # static scales of an e4m3 cache (powers of two, as calibration rounds them)


# ----------------------------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------------------------
def listed():
    return [
        # one request that decodes its next token: the smallest call, all latency
        dict(name="plan one request", op="plan", requests=1, page=16, max_pages=256, max_cached=700, max_fresh=1),
        # a full decode batch, one token each, tables for 8k tokens
        dict(name="plan decode batch", op="plan", requests=1024, page=16, max_pages=512, max_cached=8000, max_fresh=1),
        # prompts and continuations of uneven length admitted together
        dict(name="plan ragged prompts", op="plan", requests=97, page=64, max_pages=256, max_cached=9001, max_fresh=4099),
        # the keys and values of one decode step of 64 requests, read from the rows of a fused QKV product
        dict(name="store decode bf16", op="store", tokens=64, kv_heads=8, dim=128, page=16, cache="bf16", row=6144),
        # a long prompt's keys and values, quantised on the way into the cache
        dict(name="store prompt fp8", op="store", tokens=16411, kv_heads=8, dim=128, page=64, cache="fp8", row=6144),
        # a single user in the middle of a chat: few rows, latency counts
        dict(name="attention one request", op="attn", requests=1, heads=32, kv_heads=8, dim=128, page=16,
             max_len=777, window=0, cache="bf16"),
        # an ordinary serving batch of uneven lengths, grouped heads
        dict(name="attention batch", op="attn", requests=64, heads=32, kv_heads=8, dim=128, page=16,
             max_len=8191, window=0, cache="bf16"),
        # two very long documents: few rows, work only in the cache's length
        dict(name="attention long", op="attn", requests=2, heads=32, kv_heads=8, dim=128, page=64,
             max_len=131072, window=0, cache="bf16"),
        # every head with its own keys, e4m3 cache
        dict(name="attention fp8 heads", op="attn", requests=48, heads=32, kv_heads=32, dim=128, page=32,
             max_len=2048, window=0, cache="fp8"),
        # one token, one adapter of the smallest rank on a wide projection: latency
        dict(name="adapters one token", op="lora", rows=1, n=11008, k=4096, rank=8, adapters=4, run=1, base=True),
        # a decode batch in which nearly every request has an adapter of its own
        dict(name="adapters decode batch", op="lora", rows=96, n=4096, k=4096, rank=16, adapters=64, run=1, base=True),
        # prompts of several tenants in one batch, rank 64
        dict(name="adapters prompts", op="lora", rows=8192, n=4096, k=4096, rank=64, adapters=8, run=900, base=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "store", "attn", "attn", "attn", "lora", "lora"])
    if op == "plan":
        page = rng.choice([16, 32, 64, 128])
        requests = _log(rng, 1, 2048)
        # at most about 128k new tokens in all
        fresh = rng.choice([1, _log(rng, 2, min(8192, max(3, 131072 // requests)))])
        max_pages = _log(rng, 8, 1024)
        cached = _log(rng, 1, max(2, max_pages * page - fresh))
        return dict(op=op, requests=requests, page=page, max_pages=max_pages, max_cached=cached, max_fresh=fresh)
    if op == "store":
        kv_heads, dim = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([64, 128, 256])
        tokens = _log(rng, 1, max(2, min(32768, (1 << 24) // (kv_heads * dim))))
        row = kv_heads * dim * rng.choice([1, 3, 6])
        return dict(op=op, tokens=tokens, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128]),
                    cache=rng.choice(["bf16", "fp8"]), row=row)
    if op == "attn":
        dim = rng.choice([64, 128, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8, 16, 32])
        group = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 12, 16])
        cache = rng.choice(["bf16", "bf16", "fp8"])
        # requests x longest length, kept to a cache of about 1 GB in bf16
        total = (1 << 28) // (kv_heads * dim)
        requests = _log(rng, 1, 256)
        max_len = _log(rng, 1, max(2, min(131072, total // requests)))
        window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
        return dict(op=op, requests=requests, heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                    page=rng.choice([16, 32, 64, 128]), max_len=max_len, window=window, cache=cache)
    rank = rng.choice([8, 16, 16, 24, 32, 64, 128])
    n, k = 8 * _log(rng, 16, 1376), 8 * _log(rng, 16, 1376)
    if n * k > (1 << 25):
        n = max(128, (1 << 25) // k // 8 * 8)
    rows = _log(rng, 1, 8192)
    if rows * max(n, k) > (1 << 25):
        rows = max(1, (1 << 25) // max(n, k))
    adapters = _log(rng, 1, min(64, max(2, (1 << 13) // rank)))
    run = 1 if rows <= 256 else _log(rng, 16, rows)
    return dict(op="lora", rows=rows, n=n, k=k, rank=rank, adapters=adapters, run=run, base=rng.random() < 0.75)


# ----------------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------------
def _lengths(count, longest):
    """Uneven lengths up to `longest`, many short ones, the same for every seed (their order is not);
    in a batch of 16 or more every 16th place is unused, as in one padded for a captured graph."""
    got = [max(1, round(longest * ((i + 1) / count) ** 2)) for i in range(count)]
    return [0 if count >= 16 and i % 16 == 3 else v for i, v in enumerate(got)]


def _fresh(case):
    r = case["requests"]
    if case["max_fresh"] == 1:
        return [0 if r >= 16 and i % 16 == 3 else 1 for i in range(r)]
    return [max(1, round(case["max_fresh"] * ((r - i) / r) ** 2)) for i in range(r)]


def _shuffled(values, g):
    order = torch.randperm(len(values), generator=g)
    return torch.tensor(values, dtype=torch.int32)[order].to(DEV)


def _randn(shape, g, dtype=torch.bfloat16, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16).mul_(scale).to(dtype)


def _pages_of(tokens, page):
    return (tokens + page - 1) // page


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    if op == "plan":
        r, page, mp = case["requests"], case["page"], case["max_pages"]
        cached = _shuffled(_lengths(r, case["max_cached"]), host)
        fresh = _shuffled(_fresh(case), host)
        lim = mp * page
        have = _pages_of(cached.long().clamp(max=lim), page)
        need = int((_pages_of((cached.long() + fresh).clamp(max=lim), page) - have).sum())
        pool = torch.randperm(int(have.sum()) + need + 5, generator=host).to(torch.int32).to(DEV)
        # the pages that the requests hold already, row by row; the rest of the pool is free
        cols = torch.arange(mp, device=DEV)
        held = cols[None, :] < have[:, None]
        table = torch.full((r, mp), -1, dtype=torch.int32, device=DEV)
        table[held] = pool[:int(have.sum())]
        free = pool[int(have.sum()):].contiguous()
        tokens = int(fresh.sum())
        cap = tokens + 7                        # a few padded places at the end
        i32 = dict(dtype=torch.int32, device=DEV)
        return dict(case, cached=cached, fresh=fresh, free=free, head=torch.full((1,), 2, **i32), table=table,
                    starts=torch.empty(r + 1, **i32), lens=torch.empty(r, **i32),
                    slots=torch.empty(cap, dtype=torch.int64, device=DEV), rows=torch.empty(cap, **i32),
                    counts=torch.empty(4, **i32))
    if op == "store":
        t, hk, d, page = case["tokens"], case["kv_heads"], case["dim"], case["page"]
        pages = _pages_of(t, page) + 9
        both = case["row"] >= 2 * hk * d        # keys and values are column blocks of one product's rows
        x = _randn((t, case["row"]), g)
        y = x if both else _randn((t, case["row"]), g)
        k = x[:, case["row"] - hk * d:].unflatten(1, (hk, d))
        at = case["row"] - 2 * hk * d if both else 0
        v = y[:, at:at + hk * d].unflatten(1, (hk, d))
        slots = torch.randperm(pages * page, generator=host)[:t].to(DEV)
        if t >= 8:
            slots[t // 2] = -1                  # a padded place: nothing is stored for it
        codes = case["cache"] == "fp8"
        shape = (pages, hk, page, d)
        kc, vc = (_randn(shape, g, FP8 if codes else torch.bfloat16) for _ in range(2))
        return dict(case, k=k, v=v, slots=slots, kc=kc, vc=vc, pages=pages)
    if op == "attn":
        r, h, hk, d, page = case["requests"], case["heads"], case["kv_heads"], case["dim"], case["page"]
        lens = _shuffled(_lengths(r, case["max_len"]), host)
        mp = _pages_of(case["max_len"], page) + 1
        held = _pages_of(lens.long(), page)
        used = int(held.sum())
        pages = used + 3
        table = torch.full((r, mp), -1, dtype=torch.int32, device=DEV)
        table[torch.arange(mp, device=DEV)[None, :] < held[:, None]] = (
            torch.randperm(pages, generator=host)[:used].to(torch.int32).to(DEV))
        codes = case["cache"] == "fp8"
        shape = (pages, hk, page, d)
        if codes:
            kc, vc = _randn(shape, g, FP8, 1 / K_SCALE), _randn(shape, g, FP8, 1 / V_SCALE)
        else:
            kc, vc = _randn(shape, g), _randn(shape, g)
        q = _randn((r, h, d), g, scale=1.5)
        return dict(case, q=q, kc=kc, vc=vc, table=table, lens=lens, pages=pages,
                    out=torch.empty((r, h, d), dtype=torch.bfloat16, device=DEV),
                    lse=torch.empty((r, h), dtype=torch.float32, device=DEV))
    m, n, k, rank, count = case["rows"], case["n"], case["k"], case["rank"], case["adapters"]
    ids = torch.randint(0, count, (_pages_of(m, case["run"]),), generator=host)
    ids = ids.repeat_interleave(case["run"])[:m].to(torch.int32)
    if case["run"] == 1:
        ids[5::16] = -1                         # requests without an adapter
    return dict(case, x=_randn((m, k), g), a=_randn((count, rank, k), g, scale=k ** -0.5),
                b=_randn((count, n, rank), g, scale=rank ** -0.5), ids=ids.to(DEV),
                scales=torch.rand(count, generator=host).add_(0.5).to(DEV),
                y=_randn((m, n), g) if case["base"] else None,
                out=torch.empty((m, n), dtype=torch.bfloat16, device=DEV))


# ----------------------------------------------------------------------------------------------
# Plain forms
# ----------------------------------------------------------------------------------------------
def _plain_plan(s):
    page, mp = s["page"], s["max_pages"]
    lim = mp * page
    cached, fresh = s["cached"].long().clamp(0, lim), s["fresh"].long().clamp(min=0)
    lens = (cached + fresh).clamp(max=lim)
    have = (cached + page - 1) // page
    need = (lens + page - 1) // page - have
    ends, taken = fresh.cumsum(0), need.cumsum(0)
    starts, first = ends - fresh, s["head"].long() + taken - need
    cols = torch.arange(mp, device=DEV)
    new = (cols >= have[:, None]) & (cols < (have + need)[:, None])
    at = first[:, None] + cols - have[:, None]
    count = s["free"].numel()
    page_ids = torch.where(at < count, s["free"].long()[at.clamp(0, count - 1)], -1)
    table = torch.where(new, page_ids, s["table"].long())
    t = torch.arange(s["slots"].numel(), device=DEV)
    row = torch.searchsorted(ends, t, right=True)
    there = row < cached.numel()
    r = row.clamp(max=cached.numel() - 1)
    pos = cached[r] + t - starts[r]
    held = table[r, (pos // page).clamp(max=mp - 1)]
    s["table"].copy_(table)
    s["starts"][:1].zero_()
    s["starts"][1:].copy_(ends)
    s["lens"].copy_(lens)
    s["slots"].copy_(torch.where(there & (pos < lim) & (held >= 0), held * page + pos % page, -1))
    s["rows"].copy_(torch.where(there, row, -1))
    want = s["head"].long() + taken[-1:]
    s["counts"].copy_(torch.cat([ends[-1:], want.clamp(max=count), lens.max()[None], (want - count).clamp(min=0)]))


def _plain_store(s):
    there = s["slots"] >= 0
    page, off = s["slots"][there] // s["page"], s["slots"][there] % s["page"]
    for new, cache, scale in ((s["k"], s["kc"], K_SCALE), (s["v"], s["vc"], V_SCALE)):
        new = new[there]
        if s["cache"] == "fp8":
            new = (new.float() * (1 / scale)).clamp(-448, 448).to(FP8)
            cache, new = cache.view(torch.uint8), new.view(torch.uint8)
        cache[page, :, off] = new


def _plain_attention(s):
    r, h, hk, d = s["requests"], s["heads"], s["kv_heads"], s["dim"]
    table, lens = s["table"].long(), s["lens"].long()
    codes = s["cache"] == "fp8"
    rows = []
    for cache, scale in ((s["kc"], K_SCALE), (s["vc"], V_SCALE)):
        c = (cache.view(torch.uint8) if codes else cache)[table.clamp(min=0)]
        c = (c.view(FP8) if codes else c).float()
        rows.append(c.transpose(1, 2).reshape(r * hk, -1, d) * (scale if codes else 1.0))
    k, v = rows
    q = s["q"].float().view(r * hk, h // hk, d).transpose(1, 2).contiguous()
    score = (torch.bmm(k, q) * d ** -0.5).view(r, hk, -1, h // hk)
    at = torch.arange(score.shape[2], device=DEV)
    seen = at < lens[:, None]
    if s["window"]:
        seen &= at >= (lens - s["window"])[:, None]
    score = score.masked_fill(~seen[:, None, :, None], float("-inf")).transpose(2, 3)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p.reshape(r * hk, h // hk, -1), v).view(r, hk, h // hk, d)
    o = torch.where(total > 0, o / total, 0.0)
    s["out"].copy_(o.reshape(r, h, d))
    s["lse"].copy_((top + total.log()).reshape(r, h))


def _plain_adapters(s):
    m, rank, count = s["rows"], s["rank"], s["adapters"]
    h = s["x"].float() @ s["a"].float().view(count * rank, -1).t()
    ids = s["ids"].long()
    one = (torch.arange(count, device=DEV) == ids[:, None]).float() * s["scales"]
    h = (h.view(m, count, rank) * one[:, :, None]).view(m, count * rank)
    b = s["b"].float().transpose(1, 2).reshape(count * rank, -1)
    y = h @ b
    if s["y"] is not None:
        y = y + s["y"].float()
    s["out"].copy_(y)


# ----------------------------------------------------------------------------------------------
# The package's entry points
# ----------------------------------------------------------------------------------------------
def _own(s):
    import dl_fusion_amd as dlf
    op = s["op"]
    d = s.get("desc")                       # descriptors and workspaces are kept, as a program keeps them
    if op == "plan":
        if d is None:
            d = s["desc"] = dlf.page_plan_desc(s["requests"], s["page"], s["max_pages"], s["slots"].numel(),
                                               s["free"].numel())
        dlf.dlf_page_plan(d, s["cached"], s["fresh"], s["free"], s["head"], s["table"], s["starts"], s["lens"],
                          s["slots"], s["rows"], s["counts"])
        return
    if op == "store":
        if d is None:
            d = s["desc"] = dlf.kv_cache_desc(s["pages"], s["kv_heads"], s["page"], s["dim"], s["cache"], K_SCALE,
                                              V_SCALE)
        dlf.dlf_paged_store(d, s["k"], s["v"], s["slots"], s["kc"], s["vc"])
        return
    if op == "attn":
        if d is None:
            cache = dlf.kv_cache_desc(s["pages"], s["kv_heads"], s["page"], s["dim"], s["cache"], K_SCALE, V_SCALE)
            d = s["desc"] = dlf.paged_attn_desc(cache, s["requests"], s["heads"], s["table"].shape[1],
                                                softmax_scale=s["dim"] ** -0.5, window=s["window"],
                                                max_len=s["max_len"])
            s["ws"] = torch.empty(dlf.dlf_paged_attention_workspace_bytes(d), dtype=torch.uint8, device=DEV)
        dlf.dlf_paged_attention(d, s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["out"], s["lse"], s["ws"],
                                s["ws"].numel())
        return
    if d is None:
        d = s["desc"] = dlf.lora_desc(s["rows"], s["n"], s["k"], s["rank"], s["adapters"])
        s["ws"] = torch.empty(dlf.dlf_lora_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    dlf.dlf_lora_add(d, s["x"], s["a"], s["b"], s["scales"], s["ids"], None, s["y"], s["out"], s["ws"],
                     s["ws"].numel())


_PLAIN = {"plan": _plain_plan, "store": _plain_store, "attn": _plain_attention, "lora": _plain_adapters}


def run(state):
    (_own if own else _PLAIN[state["op"]])(state)
    if state["op"] == "plan":
        return {n: state[n] for n in ("table", "starts", "lens", "slots", "rows", "counts")}
    if state["op"] == "store":
        return {"kc": state["kc"], "vc": state["vc"]}
    if state["op"] == "attn":
        return {"out": state["out"], "lse": state["lse"]}
    return state["out"]


# ----------------------------------------------------------------------------------------------
# What a pass cannot do without
# ----------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "plan":
        r, page = case["requests"], case["page"]
        tokens = sum(_fresh(case))
        # new pages, each read from the free list and written to a table, for tokens in random order
        pages = sum(_pages_of(f, page) for f in _fresh(case)) if case["max_fresh"] > 1 else tokens / page
        return {"bytes": 16 * r + 8 * pages + 12 * (tokens + 7) + 4 * r, "flops": 0}
    if op == "store":
        t, w = case["tokens"], case["kv_heads"] * case["dim"]
        return {"bytes": 2 * t * w * (2 + (1 if case["cache"] == "fp8" else 2)) + 8 * t, "flops": 0}
    if op == "attn":
        r, h, hk, d = case["requests"], case["heads"], case["kv_heads"], case["dim"]
        seen = sum(min(v, case["window"] or v) for v in _lengths(r, case["max_len"]))
        size = 1 if case["cache"] == "fp8" else 2
        return {"bytes": 2 * seen * hk * d * size + 4 * r * h * d + 4 * r * h + 4 * seen // case["page"] + 4 * r,
                "flops": 4 * seen * h * d}
    m, n, k, rank = case["rows"], case["n"], case["k"], case["rank"]
    groups = _pages_of(m, case["run"])
    used = case["adapters"] * (1 - (1 - 1 / case["adapters"]) ** groups)       # expected distinct adapters
    return {"bytes": 2 * m * k + 2 * m * n * (2 if case["base"] else 1) + 2 * used * rank * (n + k) + 4 * m,
            "flops": 2 * m * rank * (n + k)}


# ----------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ----------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None
    if op == "store":
        got = []
        for new, cache, scale in ((s["k"], s["kc"], K_SCALE), (s["v"], s["vc"], V_SCALE)):
            whole = cache.double().permute(0, 2, 1, 3).reshape(-1, case["kv_heads"], case["dim"])
            keep = (s["slots"] >= 0).nonzero().flatten()
            value = new.double()[keep]
            whole[s["slots"][keep]] = value / scale if case["cache"] == "fp8" else value
            got.append(whole.view(s["pages"], case["page"], case["kv_heads"], case["dim"]).permute(0, 2, 1, 3).contiguous())
        return {"kc": got[0], "vc": got[1]}
    if op == "attn":
        h, hk, d = case["heads"], case["kv_heads"], case["dim"]
        out = torch.zeros((case["requests"], h, d), dtype=torch.float64, device=DEV)
        lse = torch.full((case["requests"], h), float("-inf"), dtype=torch.float64, device=DEV)
        codes = case["cache"] == "fp8"
        ks, vs = (K_SCALE, V_SCALE) if codes else (1.0, 1.0)
        kc, vc = (c.view(torch.uint8) if codes else c for c in (s["kc"], s["vc"]))
        for i, n in enumerate(s["lens"].tolist()):
            lo = max(0, n - case["window"]) if case["window"] else 0
            if n == 0:
                continue
            at = s["table"][i, :_pages_of(n, case["page"])].long()
            for j in range(hk):
                k = kc[:, j][at]
                k = (k.view(FP8) if codes else k).double().reshape(-1, d)[lo:n] * ks
                v = vc[:, j][at]
                v = (v.view(FP8) if codes else v).double().reshape(-1, d)[lo:n] * vs
                q = s["q"][i, j * (h // hk):(j + 1) * (h // hk)].double()
                z = (q @ k.t()) / math.sqrt(d)
                lse[i, j * (h // hk):(j + 1) * (h // hk)] = torch.logsumexp(z, 1)
                out[i, j * (h // hk):(j + 1) * (h // hk)] = torch.softmax(z, 1) @ v
        return {"out": out, "lse": lse}
    y = torch.zeros((case["rows"], case["n"]), dtype=torch.float64, device=DEV) if s["y"] is None else s["y"].double()
    for i in range(case["adapters"]):
        rows = (s["ids"] == i).nonzero().flatten()
        if rows.numel():
            y[rows] += float(s["scales"][i]) * ((s["x"][rows].double() @ s["a"][i].double().t()) @ s["b"][i].double().t())
    return y
