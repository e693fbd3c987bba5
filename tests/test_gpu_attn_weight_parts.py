"""paged_attn_weight of a step in several calls, each with a run of the
requests: their rows of the table, of q_start and of kv_len, and all of the
step's rows."""
import numpy as np
import pytest
import torch

from evict_harness import check_weights
from paged_harness import DT, Pages, f64, ints, randn, starts
from streaming_kv_cache_gb300 import skv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("q_len,kv_len,cuts,page,hq,hkv,d", [
    ([200] + [1] * 9, [700] + list(range(40, 580, 60)), [0, 1, 10], 16, 8, 2, 128), ([1, 0, 150, 300, 1], [90, 0, 400, 300, 700], [0, 2, 4, 5], 48, 14, 2, 64),
    ([130] + [0] * 40, [300] + [33] * 40, [0, 1, 41], 64, 4, 4, 64)])
def test_a_step_in_parts(q_len, kv_len, cuts, page, hq, hkv, d, dtype):
    dt, scale, st = DT[dtype], d ** -0.5, starts(q_len)
    pg, n = Pages(3, kv_len, page, hkv, d, dt), int(starts(q_len)[-1])
    cache, q = pg.cache(skv), randn(4, (n, hq, d), dt)
    _, lse = skv.paged_attn(cache, q, ints(st), ints(kv_len), scale, lse=True)
    position = torch.arange(n, dtype=torch.int32, device="cuda") + 1000
    shape = (pg.n_page, hkv, page)
    score = torch.rand(shape, generator=torch.Generator().manual_seed(5)).cuda()
    before, scores = f64(score), skv.PagedScores(score, torch.full(shape, -9, dtype=torch.int32, device="cuda"))
    ws = skv.attn_workspace()
    for lo, hi in zip(cuts, cuts[1:]):
        part = skv.PagedCache.wrap(k=cache.k, v=cache.v, block_table=cache.block_table[lo:hi], status=cache.status)
        skv.paged_attn_weight(part, scores, q, ints(st)[lo:hi + 1], ints(kv_len)[lo:hi], lse, position, scale, ws=ws)
    assert cache.device_status() == 0
    check_weights(score, pg, q, st, kv_len, lse, scale, before, before)
    want = np.full(shape, -9)
    for b, m in enumerate(kv_len):
        for i in range(q_len[b]):
            j = m - q_len[b] + i
            want[pg.table[b, j // page], :, j % page] = 1000 + st[b] + i
    assert np.array_equal(scores.pos[0].cpu().numpy(), want)
