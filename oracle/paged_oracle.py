"""fp64 NumPy restatement of the paged cache's operators and of cross
attention: a scalar plan, writes row by row, attention one request and head at
a time.  It shares no code with the CUDA path."""
from __future__ import annotations

import math

import numpy as np

NO_PAGE, BAD_LEN, TABLE_FULL = 16, 32, 256
MAX_KEYS = 1 << 26   # tokens that a request may hold


def plan(state, new_len, table, queue, page, n_tok):
    """One step's plan.  Returns a dict of the outputs (table and queue are
    copies) and the status bits."""
    n_req, n_page = len(new_len), len(queue)
    table, queue = table.copy(), queue.copy()
    old_queue = queue.copy()
    head, count = int(state[n_req]), int(state[n_req + 1])
    status = 0
    if not (0 <= head < n_page and 0 <= count <= n_page):
        head, count, status = 0, 0, BAD_LEN
    room = min(table.shape[1] * page, MAX_KEYS)
    pages = lambda x: -(-x // page)  # noqa: E731
    q_start, kv_len, nxt, position, slot = [0], [], [], [0] * n_tok, [-1] * n_tok
    wanted, given, back, pushed = 0, 0, 0, []
    for b in range(n_req):
        c, w = int(state[b]), int(new_len[b])
        if c < 0 or c > room or w < -1:
            status |= BAD_LEN
            q_start.append(q_start[-1])
            kv_len.append(0)
            nxt.append(c)
            continue
        if w == -1:
            pushed += [int(table[b, j]) for j in range(pages(c))]
            q_start.append(q_start[-1])
            kv_len.append(0)
            nxt.append(0)
            continue
        lo, hi = q_start[-1], q_start[-1] + w
        q_start.append(hi)
        for i in range(min(w, max(0, n_tok - lo))):
            position[lo + i] = c + i
        fits = w == 0 or (hi <= n_tok and c + w <= room)
        if w and not fits:
            status |= TABLE_FULL
        if fits and w:
            need = pages(c + w) - pages(c)
            wanted += need
            if need and wanted > count:
                status |= NO_PAGE
                fits = False
            elif need:
                for i in range(need):
                    table[b, pages(c) + i] = old_queue[(head + given + i) % n_page]
                given = wanted
        if not fits:
            kv_len.append(0)
            nxt.append(c)
            continue
        for i in range(w):
            slot[lo + i] = int(table[b, (c + i) // page]) * page + (c + i) % page
        kv_len.append(c + w)
        nxt.append(c + w)
    if len(pushed) > n_page - count:
        status |= BAD_LEN
        pushed = pushed[:n_page - count]
    for i, p in enumerate(pushed):
        queue[(head + count + i) % n_page] = p
    nxt += [(head + given) % n_page, count - given + len(pushed)]
    i32 = lambda x: np.asarray(x, dtype=np.int32)  # noqa: E731
    return dict(q_start=i32([min(x, n_tok) for x in q_start]), kv_len=i32(kv_len), next_state=i32(nxt),
                position=i32(position), slot=i32(slot), table=table, queue=queue), status


def rotate(x, pos, theta):
    """Rotate-half embedding of x [..., d] at integer positions pos [tokens]
    (x's first axis), angles in fp64."""
    d = x.shape[-1]
    out = np.empty_like(x, dtype=np.float64)
    for t, p in enumerate(pos):
        for i in range(d // 2):
            a = float(p) * theta ** (-2.0 * i / d)
            u, w = x[t, ..., i], x[t, ..., i + d // 2]
            out[t, ..., i] = u * math.cos(a) - w * math.sin(a)
            out[t, ..., i + d // 2] = w * math.cos(a) + u * math.sin(a)
    return out


def attend(q, k, v, first, scale):
    """q [n, Hq, d] over k, v [m, Hkv, d]: row i sees keys j < first + i + 1
    (first None: all).  Returns (out, lse, mass): mass = sum of p |v|, what a
    rounding of the probabilities can move the output by, relative to it."""
    n, hq, d = q.shape
    m, hkv, _ = k.shape
    out = np.zeros((n, hq, d))
    mass = np.zeros((n, hq, d))
    lse = np.full((hq, n), -np.inf)
    if m == 0:
        return out, lse, mass
    for h in range(hq):
        hk = h // (hq // hkv)
        z = q[:, h] @ k[:, hk].T * scale
        if first is not None:
            z = np.where(np.arange(m)[None, :] <= first + np.arange(n)[:, None], z, -np.inf)
        top = z.max(1, keepdims=True)
        p = np.exp(z - top)
        s = p.sum(1, keepdims=True)
        out[:, h] = p @ v[:, hk] / s
        mass[:, h] = p @ np.abs(v[:, hk]) / s
        lse[h] = (top + np.log(s))[:, 0]
    return out, lse, mass


def paged(q, k_pages, v_pages, table, q_start, kv_len, scale):
    """attend() over pages [n_page, Hkv, page, d] for packed q; rows of no
    request stay NaN."""
    n_tok, hq, d = q.shape
    page = k_pages.shape[2]
    out = np.full((n_tok, hq, d), np.nan)
    mass = np.full((n_tok, hq, d), np.nan)
    lse = np.full((hq, n_tok), np.nan)
    for b in range(len(kv_len)):
        lo, hi, m = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        ids = table[b, :-(-m // page)]
        rows = [np.moveaxis(x[ids], 1, 2).reshape(-1, x.shape[1], d)[:m] for x in (k_pages, v_pages)]
        out[lo:hi], lse[:, lo:hi], mass[lo:hi] = attend(q[lo:hi], rows[0], rows[1], m - (hi - lo), scale)
    return out, lse, mass


def cross(q, k, v, q_start, k_start, k_len, scale):
    """attend() without the mask over packed states [n_key, Hkv, d]."""
    n_tok, hq, d = q.shape
    out = np.full((n_tok, hq, d), np.nan)
    mass = np.full((n_tok, hq, d), np.nan)
    lse = np.full((hq, n_tok), np.nan)
    for b in range(len(k_len)):
        lo, hi, s, m = int(q_start[b]), int(q_start[b + 1]), int(k_start[b]), int(k_len[b])
        out[lo:hi], lse[:, lo:hi], mass[lo:hi] = attend(q[lo:hi], k[s:s + m], v[s:s + m], None, scale)
    return out, lse, mass
