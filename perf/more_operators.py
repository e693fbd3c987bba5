"""Eviction from the paged cache by accumulated attention weight, and sampled verification of drafted
tokens, case by case: the plain form of each in elementary torch operations, and the library's calls for
the same inputs.

  weight  the attention weight that a step's rows give each cached key, added to what it had
  select  the tokens that every (layer, request, kv head) over its budget keeps, as moves into its first places
  move    the moved tokens' keys, values, weights and positions
  trim    requests cut to fewer tokens: their lengths, and the pages behind them back to the free queue
  verify  drafted tokens accepted by the target's and the drafter's probabilities, and the token that follows
"""
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one reasoning token after a 4-view, 4-frame window (3136 tokens), one layer: latency
        dict(name="weight_decode_1", op="weight", requests=1, ctx_lo=3136, ctx_hi=3136, new=1, chunked=0, hq=32, hkv=8, d=128,
             page=64, dtype="bf16"),
        # one layer's decode step of uneven contexts in small pages: the keys are read once
        dict(name="weight_decode_64", op="weight", requests=64, ctx_lo=400, ctx_hi=8000, new=1, chunked=0, hq=32, hkv=8,
             d=128, page=16, dtype="bf16"),
        # prompt chunks and single tokens in one call, odd sizes, seven heads per kv head
        dict(name="weight_mixed_d64", op="weight", requests=24, ctx_lo=0, ctx_hi=4000, new=701, chunked=5, hq=14, hkv=2, d=64,
             page=48, dtype="fp16"),
        # chunked prefill up to the 12,800 keys of the 6-view, 8-frame window: compute
        dict(name="weight_chunk_2048", op="weight", requests=4, ctx_lo=6000, ctx_hi=10752, new=2048, chunked=4, hq=32, hkv=8,
             d=128, page=64, dtype="bf16"),
        # a server at its budget: every step each request is one token over, four layers at once
        dict(name="select_step_64", op="select", layers=4, requests=64, held_lo=2049, held_hi=2049, keep=2048, sink=4, recent=256,
             hkv=8, page=64),
        # prompts cut to a budget after their prefill, all 36 layers at once
        dict(name="select_prompt_4", op="select", layers=36, requests=4, held_lo=6000, held_hi=12800, keep=4096, sink=4,
             recent=512, hkv=8, page=64),
        # the rows of such a step: one token of every kv head
        dict(name="move_step_64", op="move", layers=4, requests=64, held_lo=2049, held_hi=2049, keep=2048, sink=4, recent=256,
             hkv=8, d=128, page=64, dtype="bf16"),
        # the rows of such prompts, eight layers
        dict(name="move_prompt_4", op="move", layers=8, requests=4, held_lo=6000, held_hi=12800, keep=4096, sink=4, recent=512,
             hkv=8, d=128, page=64, dtype="bf16"),
        # a decode batch gives back the rejected ones of up to 16 drafts: latency
        dict(name="trim_drafts_64", op="trim", requests=64, held=8000, drop=16, evict=0, page=64),
        # two thousand requests in small pages, cut to a budget
        dict(name="trim_evict_2048", op="trim", requests=2048, held=8192, drop=4096, evict=1, page=16),
        # one request's eight drafts over the vocabulary of 151,936: latency
        dict(name="verify_1", op="verify", requests=1, block=9, ragged=0, vocab=151936, draft=1, dtype="fp32"),
        # a batch of blocks of up to 16 drafts
        dict(name="verify_64", op="verify", requests=64, block=17, ragged=1, vocab=151936, draft=1, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["weight", "weight", "select", "move", "trim", "verify"])
    page = rng.choice([16, 32, 48, 64, 96, 128])
    dtype = rng.choice(["bf16", "fp16"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([64, 128])
    if op == "verify":
        return dict(op=op, requests=_log(rng, 1, 60), block=rng.randint(1, 17), ragged=rng.randint(0, 1), vocab=_log(rng, 40, 151000),
                    draft=rng.randint(0, 1), dtype=rng.choice(["fp32", "bf16", "fp16"]))
    if op == "trim":
        held = _log(rng, 2, 8000)
        return dict(op=op, requests=_log(rng, 1, 2000), held=held, drop=_log(rng, 1, held), evict=rng.randint(0, 1), page=page)
    if op in ("select", "move"):
        b = _log(rng, 1, 60)
        lo = _log(rng, 1, 2000)
        hi = _log(rng, lo + 1, max(lo + 2, 60000 // b))
        keep = max(1, hi - 1 if rng.random() < 0.3 else _log(rng, 1, hi))
        c = dict(op=op, layers=rng.randint(1, 4), requests=b, held_lo=lo, held_hi=hi, keep=keep, sink=rng.randint(0, 8),
                 recent=rng.randint(0, keep), hkv=hkv, page=page)
        return dict(c, d=d, dtype=dtype) if op == "move" else c
    hq = hkv * rng.choice([1, 2, 4, 5, 7, 8])
    if rng.random() < 0.5:   # decode
        b = _log(rng, 1, 64)
        return dict(op=op, requests=b, ctx_lo=_log(rng, 1, 400), ctx_hi=_log(rng, 401, 8000 if b > 4 else 120000),
                    new=1, chunked=0, hq=hq, hkv=hkv, d=d, page=page, dtype=dtype)
    b = _log(rng, 1, 12)
    return dict(op=op, requests=b, ctx_lo=rng.randint(0, 500), ctx_hi=_log(rng, 501, 5000), new=_log(rng, 2, 800),
                chunked=rng.randint(1, b), hq=min(hq, 32), hkv=hkv, d=d, page=page, dtype=dtype)


def _spread(lo, hi, n):
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)] if n > 1 else [hi]


def _lengths(case):
    """(tokens held, new rows) of the requests, from the case alone: every seed has the same lengths, in another order."""
    c, r = case, random.Random(12345)
    n = c["requests"]
    if c["op"] == "weight":
        ctx = _spread(c["ctx_lo"], c["ctx_hi"], n)
        r.shuffle(ctx)
        new = [c["new"] if i < c["chunked"] else 1 for i in range(n)]
        return [a + b for a, b in zip(ctx, new)], new
    if c["op"] == "verify":
        new = [max(1, c["block"] * (i + 1) // n) if c["ragged"] else c["block"] for i in range(n)]
        return [1000 + x for x in new], new
    if c["op"] == "trim":
        held = [r.randint(1, c["held"]) for _ in range(n)]
        return held, [max(0, h - r.randint(0, c["drop"])) for h in held]   # second: tokens kept
    held = _spread(c["held_lo"], c["held_hi"], n)
    return held, [c["keep"]] * n


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


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    order = random.Random(seed)
    s = dict(case=c)
    first, second = _lengths(c)
    pairs = list(zip(first, second))
    order.shuffle(pairs)
    held, new = [x[0] for x in pairs], [x[1] for x in pairs]
    n_req = len(held)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    if c["op"] == "verify":
        v, dt = c["vocab"], DTYPES[c["dtype"]]
        start = _starts(new)
        n_tok = start[-1]
        s["q_start"], s["kv_len"] = _ints(start), _ints(held)
        # the drafter's logits are the target's with an error
        logits = normal(n_tok, v) * 3
        s["p"] = torch.softmax(logits, -1).to(dt)
        guess = torch.softmax(logits + normal(n_tok, v) * 0.5, -1)
        del logits
        # token t + 1 of a block is drawn from the drafter's distribution after token t
        s["token"] = torch.multinomial(guess, 1, generator=g)[:, 0].to(torch.int32).roll(1)
        s["q"] = guess.to(dt) if c["draft"] else None
        s["u"], s["r"] = (torch.rand(n, generator=g, device="cuda") for n in (n_tok, n_req))
        s["accept_len"], s["next_token"], s["held"] = (_ints([0] * n_req) for _ in range(3))
        s["status"] = _ints([0])
        return s

    page = c["page"]
    used = [_pages(x, page) for x in held]
    n_page, most = sum(used) + 3, max(used)
    have = torch.arange(most, device="cuda")[None, :] < _ints(used)[:, None]
    ids = torch.randperm(n_page, generator=g, device="cuda").to(torch.int32)
    s["table"] = torch.zeros((n_req, most), dtype=torch.int32, device="cuda")
    s["table"][have] = ids[:sum(used)]
    s["kv_len"] = _ints(held)
    s["max_k"] = max(held)

    if c["op"] == "trim":
        head = order.randrange(n_page)
        s["queue"] = torch.full((n_page,), -1, dtype=torch.int32, device="cuda")
        s["queue"][(head + torch.arange(3, device="cuda")) % n_page] = ids[sum(used):]
        # tokens held, the free queue's head and count, tokens evicted before
        s["state"] = _ints(held + [head, 3] + [order.randrange(1000) for _ in held])
        s["next"] = torch.zeros_like(s["state"])
        s["keep"] = _ints(new)
    elif c["op"] == "weight":
        n_tok, grp = sum(new), c["hq"] // c["hkv"]
        s["q_start"], s["max_q"] = _ints(_starts(new)), max(new)
        s["q"] = normal(n_tok, c["hq"], c["d"]).to(DTYPES[c["dtype"]])
        s["k"] = normal(n_page, c["hkv"], page, c["d"]).to(DTYPES[c["dtype"]])
        s["add"] = normal(n_page, c["hkv"], page).exp()
        s["score"] = torch.zeros_like(s["add"])
        s["pos"] = torch.zeros((n_page, c["hkv"], page), dtype=torch.int32, device="cuda")
        s["position"] = torch.cat([torch.arange(a - b, a) for a, b in zip(held, new)]).to(torch.int32).cuda()
        # what the step's attention left: log of the sum of exp, per row and head
        s["lse"] = torch.empty((c["hq"], n_tok), dtype=torch.float32, device="cuda")
        at = 0
        for b, (m, n) in enumerate(pairs):
            k = s["k"][s["table"][b, :used[b]].long()].transpose(0, 1).reshape(c["hkv"], -1, c["d"])[:, :m].float()
            seen = torch.arange(m, device="cuda")[None, :] <= (m - n + torch.arange(n, device="cuda"))[:, None]
            for h in range(c["hkv"]):
                x = s["q"][at:at + n, h * grp:(h + 1) * grp].float()
                z = torch.matmul(x.reshape(n * grp, -1), k[h].t()).mul_(c["d"] ** -0.5).view(n, grp, m)
                s["lse"][h * grp:(h + 1) * grp, at:at + n] = z.masked_fill_(~seen[:, None], float("-inf")).logsumexp(-1).t()
            at += n
    else:
        n_layer, hkv = c["layers"], c["hkv"]
        pool = (n_layer, n_page, hkv, page)
        gone = [order.randrange(5000) for _ in held]
        s["keep"], s["state"] = _ints(new), _ints(held + [0, 0] + gone)
        # accumulated weights: few large, many small, some none at all
        w = (normal(*pool) * 2).exp()
        s["score"] = torch.where(torch.rand(pool, generator=g, device="cuda") < 0.02, 0.0, w)
        # tokens lie in any order of their positions, as earlier moves left them
        z = torch.rand((n_layer, n_req, hkv, s["max_k"]), generator=g, device="cuda")
        z = z.masked_fill_(torch.arange(s["max_k"], device="cuda") >= s["kv_len"][:, None, None], 2.0)
        rank = torch.empty(z.shape, dtype=torch.int32, device="cuda")
        rank.scatter_(-1, z.argsort(-1), torch.arange(s["max_k"], dtype=torch.int32, device="cuda").expand(z.shape))
        del z
        rank = torch.where(rank >= c["sink"], rank + s["state"][n_req + 2:, None, None], rank)
        s["pos"] = torch.zeros(pool, dtype=torch.int32, device="cuda")
        flat, live = _places(s)
        s["pos"].view(-1)[flat[live]] = rank[live]
        s["move"] = torch.zeros(pool, dtype=torch.int32, device="cuda")
        s["n_move"] = torch.zeros((n_layer, n_req, hkv), dtype=torch.int32, device="cuda")
        if c["op"] == "move":
            _plain_select(s)
            s["k"], s["v"] = (torch.empty(pool + (c["d"],), dtype=DTYPES[c["dtype"]], device="cuda").normal_(generator=g)
                              for _ in range(2))
    if own:   # the handle and the workspace that a program keeps
        from streaming_kv_cache_gb300 import skv
        if c["op"] == "trim":
            s["cache"] = skv.PagedCache.wrap(block_table=s["table"], page_queue=s["queue"], page_size=page, state=s["state"])
        elif c["op"] == "weight":
            s["cache"] = skv.PagedCache.wrap(k=s["k"], v=s["k"], block_table=s["table"])
            s["scores"] = skv.PagedScores(s["score"], s["pos"])
            s["ws"] = skv.attn_workspace()
        else:
            pool = s["score"].shape
            k = s["k"] if c["op"] == "move" else torch.empty(pool + (64,), dtype=torch.bfloat16, device="cuda")
            s["cache"] = skv.PagedCache.wrap(k=k, v=s.get("v", k), block_table=s["table"], state=s["state"])
            s["scores"] = skv.PagedScores(s["score"], s["pos"], s["move"], s["n_move"])
    return s


# --------------------------------------------------------------- one pass

def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        from streaming_kv_cache_gb300 import skv
        c = s["case"]
        if op == "weight":
            skv.paged_attn_weight(s["cache"], s["scores"], s["q"], s["q_start"], s["kv_len"], s["lse"], s["position"],
                                  c["d"] ** -0.5, add=s["add"], ws=s["ws"])
            return s["score"], s["pos"]
        if op == "select":
            skv.kv_evict_plan(s["cache"], s["scores"], s["kv_len"], s["keep"], c["sink"], c["recent"])
            return s["move"], s["n_move"]
        if op == "move":
            skv.kv_evict_move(s["cache"], s["scores"], s["kv_len"])
            return s["k"], s["v"], s["score"], s["pos"]
        if op == "trim":
            return skv.kv_paged_trim(s["cache"], s["keep"], evict=bool(c["evict"]), next_state=s["next"]), s["queue"]
        return skv.verify_sampled(s["p"], s["token"], s["q_start"], s["u"], s["r"], q=s["q"], kv_len=s["kv_len"],
                                  accept_len=s["accept_len"], next_token=s["next_token"], held=s["held"], status=s["status"])
    return {"weight": _plain_weight, "select": _plain_select, "move": _plain_move, "trim": _plain_trim,
            "verify": _plain_verify}[op](s)


def _plain_weight(s):
    c = s["case"]
    page, d, hkv, grp, mq = c["page"], c["d"], c["hkv"], c["hq"] // c["hkv"], s["max_q"]
    kv, start = s["kv_len"].long(), s["q_start"].long()
    n_req, n_tok = kv.numel(), s["q"].shape[0]
    j = torch.arange(s["max_k"], device="cuda")
    at = torch.where(j < kv[:, None], s["table"][:, j // page].long(), 0)
    k = s["k"][at, :, j % page].float()                                        # [requests, keys, kv heads, d]
    t = torch.arange(mq, device="cuda")
    rows = (start[:-1, None] + t).clamp(max=n_tok - 1)
    span = start[1:] - start[:-1]
    x = s["q"][rows].float().view(n_req, mq, hkv, grp, d).permute(0, 2, 3, 1, 4).reshape(n_req, hkv, grp * mq, d)
    z = torch.matmul(x, k.permute(0, 2, 3, 1)).view(n_req, hkv, grp, mq, -1)
    lse = s["lse"][:, rows].view(hkv, grp, n_req, mq).permute(2, 0, 1, 3)
    p = z.mul_(d ** -0.5).sub_(lse[..., None]).exp_()
    first = kv - span
    seen = (t < span[:, None])[:, :, None] & (j <= (first[:, None] + t)[:, :, None])
    w = p.masked_fill_(~seen[:, None, None], 0.0).sum((2, 3))                  # [requests, kv heads, keys]
    live = j < kv[:, None]
    old = s["add"][at, :, j % page].permute(0, 2, 1)
    w = torch.where((j < first[:, None])[:, None], old + w, w)
    b, i = live.nonzero(as_tuple=True)
    s["score"][at[b, i], :, i % page] = w[b, :, i]
    fresh = i >= first[b]
    b, i = b[fresh], i[fresh]
    s["pos"][at[b, i], :, i % page] = s["position"][start[b] + i - first[b]][:, None]
    return s["score"], s["pos"]


def _places(s):
    """Where token j of (layer, request, kv head) lies in a pool taken flat, and which are there."""
    n_layer, n_page, hkv, page = s["score"].shape
    j = torch.arange(s["max_k"], device="cuda")
    at = s["table"][:, j // page].long()
    row = torch.arange(n_layer, device="cuda")[:, None, None, None] * n_page + at[None, :, None, :]
    flat = (row * hkv + torch.arange(hkv, device="cuda")[:, None]) * page + j % page
    return flat, (j < s["kv_len"][:, None])[None, :, None, :].expand(flat.shape)


def _plain_select(s):
    c = s["case"]
    flat, live = _places(s)
    kv, keep = s["kv_len"].long()[:, None, None], s["keep"].long()[:, None, None]
    j = torch.arange(s["max_k"], device="cuda")
    score, pos = s["score"].view(-1)[flat], s["pos"].view(-1)[flat]
    after = s["state"][kv.shape[0] + 2:].long()[:, None, None] + kv            # the next token's position
    safe = (pos < c["sink"]) | (pos >= after - c["recent"])
    key = torch.where(live, torch.where(safe, float("inf"), score), float("-inf"))
    order = torch.sort(key, dim=-1, descending=True, stable=True)[1]
    kept = torch.empty(key.shape, dtype=torch.bool, device="cuda").scatter_(-1, order, (j < keep).expand(key.shape)) & live
    over = kv > keep
    hole, come = over & (j < keep) & ~kept, over & (j >= keep) & kept
    n = come.sum(-1)
    s["n_move"].copy_(n)
    # the i-th kept token behind the budget goes to the i-th free place below it
    pair = torch.stack([hole, come], 0).nonzero(as_tuple=True)
    i = torch.stack([hole, come], 0).cumsum(-1)[pair] - 1
    entry = flat[pair[1], pair[2], pair[3], 2 * i + pair[0]]
    s["move"].view(-1)[entry] = pair[4].to(torch.int32)
    return s["move"], s["n_move"]


def _plain_move(s):
    flat, _ = _places(s)
    j = torch.arange(s["max_k"] // 2, device="cuda")
    at = (j < s["n_move"][..., None]).nonzero(as_tuple=True)
    to, src = (s["move"].view(-1)[flat[at[0], at[1], at[2], 2 * at[3] + x]].long() for x in (0, 1))
    to, src = (flat[at[0], at[1], at[2], x] for x in (to, src))
    d = s["case"]["d"]
    for pool in (s["k"].view(-1, d), s["v"].view(-1, d), s["score"].view(-1), s["pos"].view(-1)):
        pool[to] = pool[src]
    return s["k"], s["v"], s["score"], s["pos"]


def _plain_trim(s):
    page, table, queue = s["case"]["page"], s["table"], s["queue"]
    n_req, n_page = table.shape[0], queue.numel()
    held, head, free, gone = s["state"].long().split([n_req, 1, 1, n_req])
    kept = torch.minimum(held, s["keep"].long())
    old, left = (held + page - 1) // page, (kept + page - 1) // page
    back = old - left
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    rel = (col >= left[:, None]) & (col < old[:, None])
    to = (head + free + (torch.cumsum(back, 0) - back)[:, None] + col - left[:, None]) % n_page
    pushed = torch.cat([queue, queue[:1]]).scatter_(0, torch.where(rel, to, n_page).view(-1), table.view(-1))
    queue.copy_(pushed[:n_page])
    if s["case"]["evict"]:
        gone = gone + held - kept
    s["next"].copy_(torch.cat([kept, head, free + back.sum(), torch.where(kept > 0, gone, 0)]))
    return s["next"], queue


def _plain_verify(s):
    p, q, token, start = s["p"], s["q"], s["token"].long(), s["q_start"].long()
    n_tok, n_vocab = p.shape
    n = start[1:] - start[:-1]
    j = torch.arange(s["case"]["block"], device="cuda")
    row = (start[:-1, None] + j).clamp(max=n_tok - 1)
    draft = token[(row + 1).clamp(max=n_tok - 1)]
    px = p[row, draft].double()
    qx = q[row, draft].double() if q is not None else torch.ones_like(px)
    ok = (s["u"][row].double() * qx < px) & (j < n[:, None] - 1)
    accept = torch.cumprod(ok.long(), 1).sum(1)
    at = start[:-1] + accept
    full = p[at].double()
    if q is not None:
        rest = (full - q[at].double()).clamp(min=0)
    else:
        x = token[(at + 1).clamp(max=n_tok - 1)]
        rest = full.scatter(1, x[:, None], 0.0)
    rest = torch.where((accept < n - 1)[:, None], rest, full)
    total = rest.cumsum(1)
    none = total[:, -1:] <= 0
    total = torch.where(none, full.cumsum(1), total)
    nxt = (total <= s["r"].double()[:, None] * total[:, -1:]).sum(1).clamp(max=n_vocab - 1)
    held = s["kv_len"] - n + accept + 1
    for name, x in (("accept_len", accept), ("next_token", nxt), ("held", held)):
        s[name].copy_(x)
    return s["accept_len"], s["next_token"], s["held"]


# ----------------------------------------------------------------- work

def work(case):
    c = case
    held, new = _lengths(c)
    if c["op"] == "weight":
        pairs = sum(b * (a - b) + b * (b + 1) // 2 for a, b in zip(held, new))
        # keys once; the weights before and after (a new token has its position instead); queries and lse
        return {"bytes": sum(held) * c["hkv"] * (c["d"] * 2 + 8) + sum(new) * (c["hq"] * (c["d"] * 2 + 4) + 4),
                "flops": 2 * c["hq"] * c["d"] * pairs}
    if c["op"] == "verify":
        size = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": len(held) * c["vocab"] * size * (2 if c["draft"] else 1) + sum(new) * (8 + 2 * size) + len(held) * 24,
                "flops": len(held) * c["vocab"] * 2}
    if c["op"] == "trim":
        back = sum(_pages(h, c["page"]) - _pages(k, c["page"]) for h, k in zip(held, new))
        return {"bytes": len(held) * 20 + back * 8, "flops": 0}
    over = [h for h in held if h > c["keep"]]
    moves = sum((h - c["keep"]) * c["keep"] / h for h in over)   # of tokens in any order
    heads = c["layers"] * c["hkv"]
    if c["op"] == "select":
        return {"bytes": heads * (sum(over) * 8 + moves * 8 + len(held) * 4) + len(held) * 12, "flops": 0}
    return {"bytes": heads * (moves * (2 * (4 * c["d"] + 8) + 8) + len(held) * 4) + 1, "flops": 0}


# ---------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    """The weights, request by request and head by head; the other operators' outputs are whole numbers or copies."""
    c = case
    if c["op"] != "weight":
        return None
    s = prepare(case, seed)
    f64, grp = torch.float64, c["hq"] // c["hkv"]
    starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    score = s["score"].to(f64)
    for b, m in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        pages = s["table"][b, :_pages(m, c["page"])].long()
        for hk in range(c["hkv"]):
            k = s["k"][pages, hk].reshape(-1, c["d"])[:m].to(f64)
            w = torch.zeros(pages.numel() * c["page"], dtype=f64, device="cuda")
            w[:m - (hi - lo)] = s["add"][pages, hk].reshape(-1)[:m - (hi - lo)].to(f64)
            for hd in range(hk * grp, (hk + 1) * grp):
                e = s["q"][lo:hi, hd].to(f64) @ k.T / c["d"] ** 0.5 - s["lse"][hd, lo:hi].to(f64)[:, None]
                w[:m] += torch.exp(e).tril_(m - (hi - lo)).sum(0)
            tail = score[pages, hk].reshape(-1)
            w[m:] = tail[m:]
            score[pages, hk] = w.view(-1, c["page"])
    return score, None
