"""The paged-cache operators and cross attention, case by case: the plain form of each in
elementary torch operations, and the library's calls for the same inputs.

  plan    block tables, slot maps and free pages of a step, from request lengths
  write   rotary embedding of a step's q and k, and k / v into their pages
  attn    attention of each request's new tokens over its pages (chunks and single tokens)
  cross   attention of queries to an encoder's states of another length
"""
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
THETA = 1e6


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a handful of requests that each decode one token: launch latency
        dict(name="plan_decode_8", op="plan", requests=8, page=64, ctx=4096, chunk=1, chunked=0, finished=1),
        # a busy server: two thousand requests, some prompts among them, small pages
        dict(name="plan_mixed_2048", op="plan", requests=2048, page=16, ctx=8192, chunk=1024, chunked=64, finished=40),
        # one layer's decode step of 64 requests: latency
        dict(name="write_decode_64", op="write", tokens=64, hq=32, hkv=8, d=128, page=64, dtype="bf16"),
        # an odd token count of a small model with seven query heads per kv head
        dict(name="write_odd_d64", op="write", tokens=4097, hq=14, hkv=2, d=64, page=48, dtype="fp16"),
        # prompts of a prefill step
        dict(name="write_prefill_16k", op="write", tokens=16384, hq=32, hkv=8, d=128, page=64, dtype="bf16"),
        # one reasoning token after a 4-view, 4-frame window (3136 tokens): latency
        dict(name="attn_decode_1", op="attn", requests=1, ctx_lo=3136, ctx_hi=3136, new=1, chunked=0, hq=32, hkv=8, d=128,
             page=64, dtype="bf16"),
        # a decode batch of uneven contexts in small pages
        dict(name="attn_decode_64", op="attn", requests=64, ctx_lo=400, ctx_hi=8000, new=1, chunked=0, hq=32, hkv=8, d=128,
             page=16, dtype="bf16"),
        # two requests with very long contexts: the keys of one row split over the whole GPU
        dict(name="attn_long_2", op="attn", requests=2, ctx_lo=100000, ctx_hi=131000, new=1, chunked=0, hq=32, hkv=8, d=128,
             page=128, dtype="bf16"),
        # prompt chunks and single tokens in one call, odd sizes, seven heads per kv head
        dict(name="attn_mixed_d64", op="attn", requests=24, ctx_lo=0, ctx_hi=4000, new=701, chunked=5, hq=14, hkv=2, d=64,
             page=48, dtype="fp16"),
        # chunked prefill up to the 12,800 keys of the 6-view, 8-frame window: compute
        dict(name="attn_chunk_2048", op="attn", requests=4, ctx_lo=6000, ctx_hi=10752, new=2048, chunked=4, hq=32, hkv=8,
             d=128, page=64, dtype="bf16"),
        # an action expert's 64 trajectory tokens reading the window's states, one denoising step
        dict(name="cross_action_16", op="cross", requests=16, queries=64, ragged=0, key_lo=1800, key_hi=3136, hq=32, hkv=8,
             d=128, dtype="bf16"),
        # long decoder sequences over encoder states of very different lengths, one kv head per query head
        dict(name="cross_long_6", op="cross", requests=6, queries=1536, ragged=1, key_lo=256, key_hi=12800, hq=16, hkv=16,
             d=64, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["plan", "write", "attn", "attn", "cross"])
    page = rng.choice([16, 32, 48, 64, 96, 128])
    dtype = rng.choice(["bf16", "fp16"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 7, 8])
    d = rng.choice([64, 128])
    if op == "plan":
        b = _log(rng, 1, 2000)
        return dict(op=op, requests=b, page=page, ctx=_log(rng, 1, 8000), chunk=_log(rng, 1, 1000),
                    chunked=rng.randint(0, min(b, 60)), finished=rng.randint(0, b // 8))
    if op == "write":
        return dict(op=op, tokens=_log(rng, 1, 16000), hq=min(hq, 32), hkv=hkv, d=d, page=page, dtype=dtype)
    if op == "cross":
        return dict(op=op, requests=_log(rng, 1, 16), queries=_log(rng, 1, 1000), ragged=rng.randint(0, 1),
                    key_lo=_log(rng, 1, 250), key_hi=_log(rng, 251, 8000), hq=min(hq, 16), hkv=min(hkv, 16), d=d, dtype=dtype)
    if rng.random() < 0.5:   # decode
        b = _log(rng, 1, 64)
        return dict(op=op, requests=b, ctx_lo=_log(rng, 1, 400), ctx_hi=_log(rng, 401, 8000 if b > 4 else 120000),
                    new=1, chunked=0, hq=hq, hkv=hkv, d=d, page=page, dtype=dtype)
    b = _log(rng, 1, 12)
    return dict(op=op, requests=b, ctx_lo=rng.randint(0, 500), ctx_hi=_log(rng, 501, 5000), new=_log(rng, 2, 800),
                chunked=rng.randint(1, b), hq=min(hq, 32), hkv=hkv, d=d, page=page, dtype=dtype)


def _lengths(case):
    """(ctx, new) of the requests, from the case alone: every seed has the same lengths, in another order."""
    c, r = case, random.Random(12345)
    n = c["requests"]
    if c["op"] == "plan":
        ctx = [r.randint(1, c["ctx"]) for _ in range(n)]
        new = [r.randint(max(1, c["chunk"] // 2), c["chunk"]) if i < c["chunked"] else 1 for i in range(n)]
        new = [-1 if i >= n - c["finished"] else x for i, x in enumerate(new)]
    elif c["op"] == "attn":
        ctx = [c["ctx_lo"] + (c["ctx_hi"] - c["ctx_lo"]) * i // max(1, n - 1) if n > 1 else c["ctx_hi"] for i in range(n)]
        r.shuffle(ctx)
        new = [c["new"] if i < c["chunked"] else 1 for i in range(n)]
    else:
        ctx = [c["key_lo"] + (c["key_hi"] - c["key_lo"]) * i // max(1, n - 1) if n > 1 else c["key_hi"] for i in range(n)]
        new = [max(1, c["queries"] * (i + 1) // n) if c["ragged"] else c["queries"] for i in range(n)]
    return ctx, new


def _pages(tokens, page):
    return (tokens + page - 1) // page


# ------------------------------------------------------------------ inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(lens):
    s = [0]
    for x in lens:
        s.append(s[-1] + x)
    return s


def _rope(n_pos, d):
    inv = THETA ** (-2.0 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d)
    a = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * inv[None, :]
    return torch.stack([a.cos(), a.sin()], -1).float()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    order = random.Random(seed)
    s = dict(case=c)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(DTYPES[c["dtype"]])

    if c["op"] == "write":
        n = c["tokens"]
        n_page = _pages(n, c["page"]) + 3
        span = max(1, 32768 - n)
        s["rope"] = _rope(32768, c["d"])
        s["position"] = torch.arange(n, device="cuda", dtype=torch.int32) + order.randrange(span)
        s["slot"] = torch.randperm(n_page * c["page"], generator=g, device="cuda")[:n].to(torch.int32)
        # q, k and v are parts of one projection's output, a row per token
        qkv = normal(n, c["hq"] + 2 * c["hkv"], c["d"])
        s["q"], s["k"], s["v"] = qkv[:, :c["hq"]], qkv[:, c["hq"]:c["hq"] + c["hkv"]], qkv[:, c["hq"] + c["hkv"]:]
        s["k_pages"], s["v_pages"] = (normal(n_page, c["hkv"], c["page"], c["d"]) for _ in range(2))
        s["q_out"] = torch.empty((n, c["hq"], c["d"]), dtype=DTYPES[c["dtype"]], device="cuda")
        s["table"] = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    else:
        ctx, new = _lengths(c)
        pairs = list(zip(ctx, new))
        order.shuffle(pairs)
        ctx, new = [p[0] for p in pairs], [p[1] for p in pairs]
        n_req, span = len(ctx), [max(0, x) for x in new]
        n_tok = sum(span)
        s["n_tok"] = n_tok
        if c["op"] == "plan":
            most = max(_pages(a + b, c["page"]) for a, b in zip(ctx, span))
            used = [_pages(a, c["page"]) for a in ctx]
            n_page = sum(_pages(a + b, c["page"]) for a, b in zip(ctx, span)) + 16
            ids = torch.randperm(n_page, generator=g, device="cuda").to(torch.int32)
            held = sum(used)
            have = torch.arange(most, device="cuda")[None, :] < _ints(used)[:, None]
            s["table"] = torch.full((n_req, most), -1, dtype=torch.int32, device="cuda")
            s["table"][have] = ids[:held]
            head = order.randrange(n_page)
            s["queue"] = torch.full((n_page,), -1, dtype=torch.int32, device="cuda")
            s["queue"][(head + torch.arange(n_page - held, device="cuda")) % n_page] = ids[held:]
            # a multiple of 64 token rows, as a captured graph would have; those past the last token are padding
            s["n_tok"] = (n_tok + 63) // 64 * 64
            # the step's state: cached tokens per request, then the free queue's head and count
            s["state"] = _ints(ctx + [head, n_page - held])
            s["new_len"] = _ints(new)
            s["next"] = torch.zeros_like(s["state"])
            s["q_start"], s["kv_len"] = _ints([0] * (n_req + 1)), _ints([0] * n_req)
            s["position"], s["slot"] = _ints([0] * s["n_tok"]), _ints([0] * s["n_tok"])
        else:
            kv = [a + b for a, b in zip(ctx, new)] if c["op"] == "attn" else ctx
            s["q_start"], s["kv_len"] = _ints(_starts(span)), _ints(kv)
            s["max_q"], s["max_k"] = max(span), max(kv)
            s["q"] = normal(n_tok, c["hq"], c["d"])
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty((c["hq"], n_tok), dtype=torch.float32, device="cuda")
            if c["op"] == "attn":
                most, used = _pages(max(kv), c["page"]), [_pages(x, c["page"]) for x in kv]
                n_page = sum(used) + 3
                have = torch.arange(most, device="cuda")[None, :] < _ints(used)[:, None]
                s["table"] = torch.full((n_req, most), -1, dtype=torch.int32, device="cuda")
                s["table"][have] = torch.randperm(n_page, generator=g, device="cuda")[:sum(used)].to(torch.int32)
                s["k_pages"], s["v_pages"] = (normal(n_page, c["hkv"], c["page"], c["d"]) for _ in range(2))
            else:
                s["k_start"] = _ints(_starts(kv)[:-1])
                s["k"], s["v"] = (normal(sum(kv), c["hkv"], c["d"]) for _ in range(2))
    if own:   # the handle and the workspace that a program keeps
        from streaming_kv_cache_gb300 import skv
        if c["op"] == "cross":
            s["ws"], s["status"] = skv.attn_workspace(), torch.zeros((1,), dtype=torch.int32, device="cuda")
        elif c["op"] == "plan":
            s["cache"] = skv.PagedCache.wrap(block_table=s["table"], page_queue=s["queue"], page_size=c["page"],
                                             state=s["state"])
            s["plan"] = skv.PagedPlan(s["q_start"], s["kv_len"], s["next"], s["position"], s["slot"])
        else:
            s["cache"] = skv.PagedCache.wrap(k=s["k_pages"], v=s["v_pages"], block_table=s["table"], rope=s.get("rope"))
            s["ws"] = skv.attn_workspace()
    return s


# --------------------------------------------------------------- one pass

def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        from streaming_kv_cache_gb300 import skv
        scale = s["case"].get("d", 64) ** -0.5
        if op == "plan":
            p = skv.kv_paged_plan(s["cache"], s["new_len"], s["n_tok"], plan=s["plan"])
            return (p.q_start, p.kv_len, p.next_state, p.position, p.slot, s["table"], s["queue"])
        if op == "write":
            skv.kv_paged_write(s["cache"], s["q"], s["k"], s["v"], s["position"], s["slot"], q_out=s["q_out"])
            return s["q_out"], s["k_pages"], s["v_pages"]
        if op == "attn":
            return skv.paged_attn(s["cache"], s["q"], s["q_start"], s["kv_len"], scale, out=s["out"], lse=s["lse"],
                                  ws=s["ws"])
        return skv.cross_attn(s["q"], s["k"], s["v"], s["q_start"], s["k_start"], s["kv_len"], scale, out=s["out"],
                              lse=s["lse"], ws=s["ws"], status=s["status"])
    return {"plan": _plain_plan, "write": _plain_write, "attn": _plain_attn, "cross": _plain_cross}[op](s)


def _exclusive(x):
    return torch.cumsum(x, 0) - x


def _plain_plan(s):
    page, n_tok = s["case"]["page"], s["n_tok"]
    table, queue, new = s["table"], s["queue"], s["new_len"].long()
    n_req, n_page = new.numel(), queue.numel()
    ctx, head, free = s["state"][:n_req].long(), s["state"][n_req].long(), s["state"][n_req + 1].long()
    span = new.clamp(min=0)
    q_start = torch.cat([span.new_zeros(1), torch.cumsum(span, 0)])
    done = new < 0
    old = (ctx + page - 1) // page
    total = (ctx + span + page - 1) // page
    need = torch.where(done, 0, total - old)
    first = _exclusive(need)
    fits = (need == 0) | (first + need <= free)
    need = torch.where(fits, need, 0)
    given = need.sum()
    kv = torch.where(done | ~fits, 0, ctx + span)
    after = torch.where(done, 0, torch.where(fits, ctx + span, ctx))
    # the new pages of each request, from the queue's head
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    fresh = (col >= old[:, None]) & (col < (old + need)[:, None])
    at = (head + first[:, None] + col - old[:, None]) % n_page
    table.copy_(torch.where(fresh, queue[at], table))
    # finished requests' pages go to the queue's tail
    back = torch.where(done, old, 0)
    rel = col < back[:, None]
    to = torch.where(rel, (head + free + _exclusive(back)[:, None] + col) % n_page, n_page)
    pushed = torch.cat([queue, queue[:1]]).scatter_(0, to.view(-1), table.view(-1))
    queue.copy_(pushed[:n_page])
    nxt = torch.cat([after, ((head + given) % n_page)[None], (free - given + back.sum())[None]])
    # a slot and a position per token
    t = torch.arange(n_tok, device="cuda")
    b = torch.searchsorted(q_start[1:].contiguous(), t, right=True).clamp(max=n_req - 1)
    live = t < q_start[-1]
    pos = ctx[b] + t - q_start[b]
    slot = table[b, (pos // page).clamp(0, table.shape[1] - 1)].long() * page + pos % page
    slot = torch.where(live & fits[b], slot, -1)
    i32 = torch.int32
    return (q_start.to(i32), kv.to(i32), nxt.to(i32), torch.where(live, pos, 0).to(i32), slot.to(i32), table, queue)


def _plain_write(s):
    d, page = s["case"]["d"], s["case"]["page"]
    cs = s["rope"][s["position"].long()][:, None]
    c, z = cs[..., 0], cs[..., 1]

    def rotate(x):
        a, b = x[..., :d // 2].float(), x[..., d // 2:].float()
        return torch.cat([a * c - b * z, b * c + a * z], -1).to(x.dtype)

    p, r = s["slot"].long() // page, s["slot"].long() % page
    s["k_pages"][p, :, r] = rotate(s["k"])
    s["v_pages"][p, :, r] = s["v"]
    return rotate(s["q"]), s["k_pages"], s["v_pages"]


def _plain_softmax(s, k, v, limit):
    """q (packed, padded per request here) over k, v [requests, keys, kv heads, d]; row (b, t) sees keys below limit[b, t]."""
    c = s["case"]
    q, start = s["q"], s["q_start"].long()
    n_req, d, hkv = start.numel() - 1, c["d"], c["hkv"]
    g, mq = c["hq"] // hkv, s["max_q"]
    rows = (start[:-1, None] + torch.arange(mq, device="cuda")).clamp(max=q.shape[0] - 1)
    x = q[rows].float().view(n_req, mq, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n_req, hkv, g * mq, d)
    z = torch.matmul(x, k.permute(0, 2, 3, 1)) * d ** -0.5
    seen = torch.arange(k.shape[1], device="cuda") < limit[:, :, None]
    z = z.view(n_req, hkv, g, mq, -1).masked_fill_(~seen[:, None, None], float("-inf"))
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = torch.exp(z.sub_(m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n_req, hkv, g * mq, -1), v.permute(0, 2, 1, 3)).view(n_req, hkv, g, mq, d)
    o = torch.where(l > 0, o / l, 0.0)
    lse = (m + torch.log(l))[..., 0]
    t = torch.arange(q.shape[0], device="cuda")
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    i = t - start[b]
    o = o.permute(0, 3, 1, 2, 4).reshape(n_req, mq, c["hq"], d)[b, i]
    lse = lse.permute(0, 3, 1, 2).reshape(n_req, mq, c["hq"])[b, i]
    return o.to(q.dtype), lse.t().contiguous()


def _plain_attn(s):
    page, kv, start = s["case"]["page"], s["kv_len"].long(), s["q_start"].long()
    pos = torch.arange(s["max_k"], device="cuda")
    at = torch.where(pos < kv[:, None], s["table"][:, pos // page].long(), 0)
    k, v = (s[n][at, :, pos % page].float() for n in ("k_pages", "v_pages"))
    first = kv - (start[1:] - start[:-1])
    return _plain_softmax(s, k, v, first[:, None] + 1 + torch.arange(s["max_q"], device="cuda"))


def _plain_cross(s):
    kv = s["kv_len"].long()
    pos = torch.arange(s["max_k"], device="cuda")
    at = s["k_start"].long()[:, None] + torch.minimum(pos, kv[:, None] - 1)
    k, v = (s[n][at].float() for n in ("k", "v"))
    return _plain_softmax(s, k, v, kv[:, None].expand(-1, s["max_q"]))


# ----------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "write":
        row = c["d"] * 2
        n = c["tokens"]
        return {"bytes": n * (2 * (c["hq"] + 2 * c["hkv"]) * row + c["d"] * 4 + 8),
                "flops": n * (c["hq"] + c["hkv"]) * c["d"] * 3}
    ctx, new = _lengths(c)
    span = [max(0, x) for x in new]
    n_tok = sum(span)
    if c["op"] == "plan":
        pages = sum(_pages(a + b, c["page"]) - _pages(a, c["page"]) for a, b in zip(ctx, span))
        back = sum(_pages(a, c["page"]) for a, b in zip(ctx, new) if b < 0)
        return {"bytes": len(ctx) * 20 + n_tok * 8 + (pages + back) * 8, "flops": 0}
    if c["op"] == "attn":
        kv = [a + b for a, b in zip(ctx, new)]
        pairs = sum(b * a + b * (b + 1) // 2 for a, b in zip(ctx, new))
    else:
        kv = ctx
        pairs = sum(a * b for a, b in zip(ctx, new))
    return {"bytes": 2 * sum(kv) * c["hkv"] * c["d"] * 2 + n_tok * c["hq"] * (c["d"] * 4 + 4),
            "flops": 4 * c["hq"] * c["d"] * pairs}


# ---------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    c = case
    if c["op"] == "plan":
        return None
    s = prepare(case, seed)
    f64 = torch.float64
    if c["op"] == "write":
        h = c["d"] // 2
        cos, sin = (s["rope"][s["position"].long(), :, i].to(f64)[:, None, :] for i in (0, 1))
        got = []
        for name in ("q", "k"):
            x = s[name].to(f64)
            y = torch.empty_like(x)
            y[..., :h] = x[..., :h] * cos - x[..., h:] * sin
            y[..., h:] = x[..., :h] * sin + x[..., h:] * cos
            got.append(y)
        flat = s["slot"].long()
        kp, vp = s["k_pages"].to(f64), s["v_pages"].to(f64)
        for pool, rows in ((kp, got[1]), (vp, s["v"].to(f64))):
            for hd in range(c["hkv"]):
                plane = pool[:, hd].reshape(-1, c["d"])
                plane[flat] = rows[:, hd]
                pool[:, hd] = plane.view(pool.shape[0], c["page"], c["d"])
        return got[0], kp, vp
    starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    out = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=f64, device="cuda")
    grp = c["hq"] // c["hkv"]
    for b, n in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        for hk in range(c["hkv"]):
            if c["op"] == "attn":
                ids = s["table"][b, :_pages(n, c["page"])].long()
                k, v = (s[p][ids, hk].reshape(-1, c["d"])[:n].to(f64) for p in ("k_pages", "v_pages"))
            else:
                r = int(s["k_start"][b])
                k, v = (s[p][r:r + n, hk].to(f64) for p in ("k", "v"))
            for hd in range(hk * grp, (hk + 1) * grp):
                w = (s["q"][lo:hi, hd].to(f64) @ k.T) / c["d"] ** 0.5
                if c["op"] == "attn":
                    w += torch.full_like(w, float("-inf")).triu_(n - (hi - lo) + 1)
                lse[hd, lo:hi] = torch.logsumexp(w, -1)
                out[lo:hi, hd] = torch.softmax(w, -1) @ v
    return out, lse
