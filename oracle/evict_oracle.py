"""fp64 NumPy restatement of eviction from the paged cache and of sampled
verification: one request, head, page and token at a time.  It shares no code
with the CUDA path."""
from __future__ import annotations

import math

import numpy as np

from . import paged_oracle as PO

BAD_LEN, BAD_PAGE, BAD_TOKEN, BAD_PROB = 32, 64, 512, 1024
TOP = 2 ** 31 - 1


def plan_evicting(state, new_len, table, queue, page, n_tok):
    """paged_oracle.plan for a state with evicted words."""
    n_req = len(new_len)
    state = [int(x) for x in state]
    got, status = PO.plan(state[:n_req + 2], new_len, table, queue, page, n_tok)
    room = min(table.shape[1] * page, PO.MAX_KEYS)
    after, position = [], got["position"].astype(np.int64)
    for b in range(n_req):
        c, e, w = state[b], state[n_req + 2 + b], int(new_len[b])
        if c < 0 or c > room or w < -1:
            after.append(e)
            if e < 0:
                status |= BAD_LEN
            continue
        if e < 0:
            status |= BAD_LEN
        e = max(e, 0) if c > 0 else 0
        after.append(0 if w == -1 else e)
        lo, hi = int(got["q_start"][b]), int(got["q_start"][b + 1])
        position[lo:hi] += e
    got["position"] = np.minimum(position, TOP).astype(np.int32)
    got["next_state"] = np.concatenate([got["next_state"], np.asarray(after, dtype=np.int32)])
    return got, status


def trim(state, keep, table, queue, page, mode):
    """Returns (next_state, queue, status); mode 0, 1 (drafts) or 2 (evicted)."""
    n_req, n_page, status = len(keep), len(queue), 0
    state, queue = [int(x) for x in state], queue.copy()
    head, count = state[n_req], state[n_req + 1]
    if not (0 <= head < n_page and 0 <= count <= n_page):
        head, count, status = 0, 0, BAD_LEN
    room = min(table.shape[1] * page, PO.MAX_KEYS)
    nxt, words, back = [], [], []
    for b in range(n_req):
        c, k = state[b], int(keep[b])
        e = state[n_req + 2 + b] if mode else 0
        if c < 0 or c > room or k < 0:
            status |= BAD_LEN
            nxt.append(c)
            words.append(e)
            continue
        if e < 0:
            status |= BAD_LEN
        kept = min(c, k)
        nxt.append(kept)
        words.append(0 if kept == 0 else min(TOP, max(e, 0) + (c - kept if mode == 2 else 0)))
        back += [int(table[b, j]) for j in range(-(-kept // page), -(-c // page))]
    if len(back) > n_page - count:
        status |= BAD_LEN
        back = back[:n_page - count]
    for i, p in enumerate(back):
        if not 0 <= p < n_page:
            status |= BAD_PAGE
        queue[(head + count + i) % n_page] = p
    nxt += [head, count + len(back)] + (words if mode else [])
    return np.asarray(nxt, dtype=np.int32), queue, status


def weights(q, k_pages, table, q_start, kv_len, lse, scale):
    """[request][kv head][key]: the sum over rows and query heads of
    exp(scale q.k - lse), rows that see the key only; a row whose lse is not
    finite gives nothing."""
    hq, hkv = q.shape[1], k_pages.shape[1]
    grp, out = hq // hkv, []
    for b, m in enumerate(int(x) for x in kv_len):
        lo, hi = int(q_start[b]), int(q_start[b + 1])
        k = np.moveaxis(k_pages[table[b, :-(-m // k_pages.shape[2])]], 1, 2).reshape(-1, hkv, q.shape[2])[:m]
        w = np.zeros((hkv, m))
        for h in range(hq):
            for i in range(hi - lo):
                if np.isfinite(lse[h, lo + i]):
                    n = m - (hi - lo) + i + 1
                    w[h // grp, :n] += np.exp(scale * (k[:n, h // grp] @ q[lo + i, h]) - lse[h, lo + i])
        out.append(w)
    return out


def select(score, pos, keep, after, n_sink, n_recent):
    """The moves of one (layer, request, kv head): (to, from) pairs that bring
    the keep best of its tokens into its first keep places.  score, pos: of
    its tokens; after: the next token's position."""
    n = len(score)
    if n <= keep:
        return []
    def rank(j):  # best first
        if pos[j] < n_sink or after - n_recent <= pos[j] < after:
            return (0, 0.0, j)
        s = float(score[j])
        return (2, 0.0, j) if math.isnan(s) else (1, -s, j)
    kept = set(sorted(range(n), key=rank)[:keep])
    free = [j for j in range(keep) if j not in kept]
    return list(zip(free, [j for j in range(keep, n) if j in kept]))


def verify(token, p, q, u, r, status=0):
    """One request's block: (accepted drafts, next token, status).  p and q
    [rows][V] (q None: drafts without probabilities)."""
    n, v = len(token), p.shape[1]
    def prob(x):
        x = float(x)
        return x if 0.0 <= x <= 2.0 else 0.0
    a = 0
    while a < n - 1:
        x = int(token[a + 1])
        if not 0 <= x < v:
            status |= BAD_TOKEN
            break
        if not float(u[a]) * (prob(q[a, x]) if q is not None else 1.0) < prob(p[a, x]):
            break
        a += 1
    full = [prob(x) for x in p[a]]
    if any(not 0.0 <= float(x) <= 2.0 for x in p[a]):
        status |= BAD_PROB
    rest = full
    if a < n - 1:
        if q is not None:
            if any(not 0.0 <= float(x) <= 2.0 for x in q[a]):
                status |= BAD_PROB
            rest = [max(x - prob(y), 0.0) for x, y in zip(full, q[a])]
        else:
            rest = [0.0 if i == int(token[a + 1]) else x for i, x in enumerate(full)]
        if math.fsum(rest) <= 0:
            rest = full
    total = math.fsum(rest)
    if total <= 0:
        return a, -1, status | BAD_PROB
    rr = float(r)
    t = 0.0 if not rr > 0 else total * min(rr, 1.0)
    cum, last = 0.0, -1
    for i, x in enumerate(rest):
        cum += x
        if x > 0:
            last = i
            if cum > t:
                return a, i, status
    return a, last, status
