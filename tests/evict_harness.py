"""Set-up and bounds shared by the GPU tests of eviction."""
import numpy as np
import torch

from oracle import evict_oracle as EO
from paged_harness import f64, ints, score_error


def check_weights(got, pages, q, q_start, kv_len, lse, scale, add, before, what=""):
    """Scores [page][kv head][row] after a call against the oracle's.

    A term exp(x), x = scale q.k - lse, is off by e of itself: e adds the
    error of q.k (score_error), a half step of fp32 at each of the product with
    the scale, the logarithm's change of base and the difference (none above
    1.45 (|scale q.k| + |lse|)), and ex2's 2^-22 and its argument's.  A sum of n terms
    adds n 2^-24 of itself, adding to the old score a half step of the result.
    Entries that the call does not write are what was there before.
    """
    k, qd, ls = f64(pages.k), f64(q), f64(lse)
    hq, hkv = q.shape[1], pages.hkv
    w = EO.weights(qd, k, pages.table, q_start, kv_len, ls, scale)
    live = np.where(np.isnan(k), 0.0, k)
    qn, kn = np.linalg.norm(qd, axis=-1).max(initial=0), np.linalg.norm(live, axis=-1).max(initial=0)
    fin = np.abs(ls[np.isfinite(ls)]).max(initial=0)
    e = score_error(pages.d, qn, kn, scale) + 4 * 2.0 ** -24 * 1.45 * (scale * qn * kn + fin) + 2.0 ** -21
    want, tol = before.copy(), np.zeros_like(before)
    for b, m in enumerate(int(x) for x in kv_len):
        n = int(q_start[b + 1] - q_start[b])
        if n == 0:
            continue
        for j in range(m):
            at = (pages.table[b, j // pages.page], slice(None), j % pages.page)
            old = add[at] if add is not None and j < m - n else 0.0
            want[at] = w[b][:, j] + old
            tol[at] = w[b][:, j] * (np.expm1(e) + (hq // hkv * n + 2) * 2.0 ** -24) + 2.0 ** -24 * np.abs(want[at]) + 2.0 ** -126
    got = f64(got)
    same = np.isnan(want)
    assert np.array_equal(np.isnan(got), same), what
    err = np.abs(got - want)[~same]
    lim = tol[~same]
    assert (err <= lim).all(), "%s: %.3g times the bound" % (what, (err / np.maximum(lim, 1e-300)).max())
    return w


def lay(values, table, page, n_page, fill, dtype):
    """A pool [layers][n_page][Hkv][page] with values[layer][request][kv head][token]
    at the tokens' places and fill elsewhere."""
    hkv = values[0][0].shape[0]
    pool = np.full((len(values), n_page, hkv, page), fill, dtype=dtype)
    for l, reqs in enumerate(values):
        for b, x in enumerate(reqs):
            for j in range(x.shape[1]):
                pool[l, table[b, j // page], :, j % page] = x[:, j]
    return pool


def moves_of(move, n_move, table, page, l, b, h):
    """[(to, from)] of one (layer, request, kv head)."""
    at = lambda j: int(move[l, table[b, j // page], h, j % page])  # noqa: E731
    return [(at(2 * i), at(2 * i + 1)) for i in range(int(n_move[l, b, h]))]


def tables(rng, used, n_page, cols):
    ids, table, at = rng.permutation(n_page), np.full((len(used), cols), -1, dtype=np.int32), 0
    for b, n in enumerate(used):
        table[b, :n] = ids[at:at + n]
        at += n
    return table


__all__ = ["check_weights", "lay", "moves_of", "tables", "ints", "torch"]
