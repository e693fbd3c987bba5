"""verify_sampled against whole-number arithmetic: probabilities cut to 2^-55,
sums of them in 64-bit integers, and the draw's share of the sum as a fraction,
so that every answer is equal, on a border too."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from paged_harness import ints, starts
from streaming_kv_cache_gb300 import skv

pytestmark = pytest.mark.gpu


def _answer(token, p, q, u, r):
    """(accepted drafts, next token) of one request; p, q float64 [rows][V]."""
    n, a = len(token), 0
    while a < n - 1 and float(u[a]) * (q[a, token[a + 1]] if q is not None else 1.0) < p[a, token[a + 1]]:
        a += 1
    full = (p[a] * 2.0 ** 55).astype(np.int64)      # exact product of a power of two, then cut
    w = full
    if a < n - 1:
        w = full.copy()
        if q is not None:
            w = np.maximum(full - (q[a] * 2.0 ** 55).astype(np.int64), 0)
        else:
            w[token[a + 1]] = 0
        if not w.any():
            w = full
    cum = np.cumsum(w)
    return a, int(np.argmax(cum > int(Fraction(float(r)) * int(cum[-1]))))


def _strided(x, stride, dtype, offset):
    buf = torch.zeros(offset + max(len(x), 1) * stride + 8, dtype=dtype, device="cuda")
    view = torch.as_strided(buf, x.shape, (stride, 1), offset)
    view.copy_(torch.from_numpy(x))
    return view


def _check(p, q, token, spans, u, r):
    st, f32 = starts(spans), lambda x: torch.from_numpy(np.asarray(x, dtype=np.float32)).cuda()  # noqa: E731
    u, r = np.asarray(u, dtype=np.float32), np.asarray(r, dtype=np.float32)
    status = ints([0])
    acc, nxt, _ = skv.verify_sampled(p, ints(list(token)), ints(st), f32(u), f32(r), q=q, status=status)
    hp, hq = p.double().cpu().numpy(), q.double().cpu().numpy() if q is not None else None
    want = [_answer(token[lo:hi], hp[lo:hi], hq[lo:hi] if q is not None else None, u[lo:hi], r[b])
            for b, (lo, hi) in enumerate(zip(st, st[1:]))]
    assert list(zip(acc.tolist(), nxt.tolist())) == want
    assert int(status) == 0


def _parts(x):
    """fp32 numbers whose sum is x units of 2^-55."""
    out = []
    while x:
        low = max(0, x.bit_length() - 24)
        out.append(np.float32((x >> low << low) * 2.0 ** -55))
        x -= x >> low << low
    return out


@pytest.mark.parametrize("stride", [0, 1])
def test_draws_between_single_units(stride):
    """Rows in which entries of one unit surround the draw, so that the token
    tells its exact place: totals of 56 bits, draws of 24."""
    rng, rows, draws, units = np.random.default_rng(0), [], [], 40
    for _ in range(40):
        total = (1 << 55) + int(rng.integers(-1 << 40, 1 << 40)) | 1
        k = int(rng.integers(1 << 22, 1 << 24)) | 1
        at = k * total >> 24                        # whole part of the draw's share
        head = _parts(at - int(rng.integers(units)))
        tail = _parts(total - units - sum(int(float(x) * 2.0 ** 55) for x in head))
        rows.append(head + [np.float32(2.0 ** -55)] * units + tail)
        draws.append(k * 2.0 ** -24)
    v = max(len(x) for x in rows) + 3
    p = np.zeros((len(rows), v))
    for row, x in zip(p, rows):
        row[:len(x)] = x
    p = _strided(p, (v + 3) // 4 * 4 + stride, torch.float32, 0)
    _check(p, None, [0] * len(rows), [1] * len(rows), [0.0] * len(rows), draws)


def test_small_draws():
    """r below the units of the total: the first entry; r of a few units."""
    v = 300
    p = torch.full((6, v), 2.0 ** -55, device="cuda")
    for r in ([2.0 ** -149, 2.0 ** -126, 2.0 ** -100, 1 / 512, 0.25, 1 - 2.0 ** -24], [0.0, 2.0 ** -8, 0.003, 0.5, 0.7, 0.9999]):
        _check(p, None, [0] * 6, [1] * 6, [0.0] * 6, r)
