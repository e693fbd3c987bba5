"""paged_attn and cross_attn against 64 bits, with the roundings' expected size
as the limit (see paged_stats): a lost or misplaced key shows at any length."""
import numpy as np
import pytest
import torch

import paged_stats as S
from paged_harness import DT, Pages, ints, randn, starts
from streaming_kv_cache_gb300 import skv

pytestmark = pytest.mark.gpu


def _check(out, q, rows, dt, scale, rounded_p, spans, kv, causal):
    """rows(b) gives request b's keys and values; spans its token rows."""
    worst, err2, var2, n_out = 0.0, 0.0, 0.0, 0
    for b, n in enumerate(kv):
        lo, hi = int(spans[b]), int(spans[b + 1])
        if hi == lo or n < 128:
            continue
        k, v = rows(b)
        first = n - (hi - lo) if causal else None
        want, var, common = S.expected(q[lo:hi].double(), k.double(), v.double(), first, scale, dt, rounded_p)
        keys = first + 1 + torch.arange(hi - lo, device="cuda") if causal else torch.full((hi - lo,), n, device="cuda")
        row, _ = S.excess(out[lo:hi].double(), want, var, common, keys)
        worst = max(worst, row)
        live = keys >= 128
        err2 += float((((out[lo:hi].double() - want).abs() - common).clamp(min=0)[live] ** 2).sum())
        var2 += float(var[live].sum())
        n_out += int(live.sum()) * out[0].numel()
    assert n_out >= 8192
    total = (err2 / (1.21 * var2)) ** 0.5
    assert worst <= 1 and total <= 1, "rows %.3g, all %.3g times the limit" % (worst, total)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,ql,kv,hq,hkv", [
    (64, [1] * 20, [9001, 20000] + [1000 + 77 * i for i in range(18)], 32, 4),        # decode, split over CTAs
    (16, [1] * 160, [129 + 17 * i for i in range(160)], 8, 2),                         # decode, several units a CTA
    (48, [200, 1, 333, 65, 1], [5000, 3000, 333, 2048, 9001], 8, 2),                   # chunks and single tokens
    (128, [70] * 80, [3000] * 80, 14, 2),                                              # whole units
    (64, [40], [20000], 8, 1)])                                                        # one chunk over the GPU
def test_paged_error(dtype, d, page, ql, kv, hq, hkv):
    dt, scale = DT[dtype], d ** -0.5
    pg = Pages(d + page, kv, page, hkv, d, dt)
    cache, spans = pg.cache(skv), starts(ql)
    q = randn(1, (sum(ql), hq, d), dt)
    out = skv.paged_attn(cache, q, ints(spans), ints(kv), scale)
    assert cache.device_status() == 0

    def rows(b):
        ids = torch.from_numpy(pg.table[b, :-(-kv[b] // page)]).long().cuda()
        return [x[ids].transpose(1, 2).reshape(-1, hkv, d)[:kv[b]] for x in (pg.k, pg.v)]

    wide = sum(ql) > len(ql) * (128 // (hq // hkv))      # two query tiles a unit: P in one term
    _check(out, q, rows, dt, scale, wide, spans, kv, True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,hq,hkv,ql,kl", [(128, 8, 2, [64, 64, 1], [1800, 3136, 20000]), (64, 4, 4, [300, 700], [5000, 12800]),
                                            (64, 16, 2, [1] * 30, [200 + 300 * i for i in range(30)])])
def test_cross_error(dtype, d, hq, hkv, ql, kl):
    dt, scale = DT[dtype], d ** -0.5
    at, spans = starts(kl), starts(ql)
    k, v, q = randn(1, (sum(kl), hkv, d), dt), randn(2, (sum(kl), hkv, d), dt), randn(3, (sum(ql), hq, d), dt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = skv.cross_attn(q, k, v, ints(spans), ints(at[:-1]), ints(kl), scale, status=status)
    assert status.item() == 0
    wide = sum(ql) > len(ql) * (128 // (hq // hkv))
    _check(out, q, lambda b: (k[at[b]:at[b + 1]], v[at[b]:at[b + 1]]), dt, scale, wide, spans, kl, False)


def test_bad_spans_leave_the_other_requests_right():
    """A span out of range is skipped: its rows stay as they were, the valid
    requests' rows are right, and a wrong key count makes zeros."""
    d, dt, kv, scale = 64, torch.bfloat16, [400, 200, 500], 0.125
    pg = Pages(3, kv, 16, 1, d, dt)
    q = randn(4, (400, 8, d), dt)
    dense = [[x[torch.from_numpy(pg.table[b, :-(-n // 16)]).long().cuda()].transpose(1, 2).reshape(-1, 1, d)[:n]
              for x in (pg.k, pg.v)] for b, n in enumerate(kv)]
    # spans and lengths; which requests are valid, which rows are zeros
    for spans, lens, valid, zeros in (([0, 128, 2 ** 20, 400], kv, [0], []), ([-1, 130, 260, 400], kv, [1, 2], []),
                                      ([0, 130, 100, 400], kv, [], []), ([0, 130, 300, 401], kv, [0, 1], []),
                                      ([0, 130, 300, 400], [400, 100, 500], [0, 2], range(130, 300)),
                                      ([0, 130, 300, 400], [2 ** 31 - 1, 200, 500], [1, 2], range(0, 130))):
        cache = pg.cache(skv)
        out, lse = torch.full((400, 8, d), 5.0, dtype=dt, device="cuda"), torch.full((8, 400), 5.0, device="cuda")
        skv.paged_attn(cache, q, ints(spans), ints(lens), scale, out=out, lse=lse)
        assert cache.device_status() == skv.SKV_DEV_BAD_LEN
        touched = torch.zeros(400, dtype=torch.bool)
        for b in range(3):
            lo, hi = spans[b], spans[b + 1]
            if 0 <= lo <= hi <= 400:
                touched[lo:hi] = True
            if b not in valid:
                continue
            want, var, common = S.expected(q[lo:hi].double(), dense[b][0].double(), dense[b][1].double(), kv[b] - (hi - lo), scale, dt, True)
            keys = kv[b] - (hi - lo) + 1 + torch.arange(hi - lo, device="cuda")
            row, _ = S.excess(out[lo:hi].double(), want, var, common, keys)
            assert row <= 1, (spans, lens, b, row)
        for r in zeros:
            assert (out[r] == 0).all() and torch.isneginf(lse[:, r]).all()
        assert (out[~touched] == 5).all() and (lse[:, ~touched] == 5).all(), (spans, lens)
