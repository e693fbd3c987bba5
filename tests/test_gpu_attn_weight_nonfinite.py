"""paged_attn_weight where a row's lse is not finite because its scores are
not: the row gives nothing, and every other row of its tile what it gives
beside finite ones (within the bound that evict_harness.check_weights
derives)."""
import numpy as np
import pytest
import torch

from evict_harness import check_weights
from paged_harness import DT, Pages, f64, ints, randn, starts
from streaming_kv_cache_gb300 import skv

pytestmark = pytest.mark.gpu

# narrow forms of one and of several rows a tile, wide ones with whole units, and with shared ones;
# seven and three heads per kv head leave columns of a wide tile without a row
CASES = [
    ([1, 1, 1], [300, 513, 129], 16, 8, 2, 64), ([5, 3], [260, 900], 64, 4, 2, 128), ([40, 33], [700, 161], 16, 8, 2, 128),
    ([90, 1], [400, 70], 48, 14, 2, 64), ([700], [1500], 64, 8, 2, 128), ([301], [900], 96, 3, 1, 64), ([256], [1024], 64, 2, 2, 64)]


def _odd_entries(rng, n, hq):
    """(row, head) of the entries whose queries are not finite: single heads
    and whole rows, the first and the last row among them."""
    at = {(0, 0), (n - 1, hq - 1)} | {(int(rng.integers(n)), int(rng.integers(hq))) for _ in range(4)}
    whole = int(rng.integers(n))
    return sorted(at | ({(whole, h) for h in range(hq)} if n > 4 else set()))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("by_hand", [None, float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_rows_whose_scores_are_not_finite_give_nothing(case, by_hand, dtype):
    q_len, kv_len, page, hq, hkv, d = CASES[case]
    dt, scale, rng = DT[dtype], d ** -0.5, np.random.default_rng(case)
    pg, st = Pages(case, kv_len, page, hkv, d, dt), starts(q_len)
    cache, n = pg.cache(skv), int(st[-1])
    clean = randn(case + 1, (n, hq, d), dt)
    q = clean.clone()
    odd = _odd_entries(rng, n, hq)
    for i, (row, head) in enumerate(odd):
        if i % 4 == 0:
            q[row, head] = float("nan")
        else:
            q[row, head, int(rng.integers(d))] = (float("nan"), float("inf"), float("-inf"))[i % 4 - 1]
        clean[row, head] = 0
    _, lse = skv.paged_attn(cache, q, ints(st), ints(kv_len), scale, lse=True)
    finite = torch.ones((hq, n), dtype=torch.bool, device="cuda")
    for row, head in odd:
        finite[head, row] = False
        if by_hand is not None:
            lse[head, row] = by_hand
    assert torch.equal(torch.isfinite(lse), finite)
    shape = (pg.n_page, hkv, page)
    score = torch.rand(shape, generator=torch.Generator().manual_seed(case)).cuda() * 10
    before = f64(score)
    scores = skv.PagedScores(score, torch.zeros(shape, dtype=torch.int32, device="cuda"))
    skv.paged_attn_weight(cache, scores, q, ints(st), ints(kv_len), lse, torch.arange(n, dtype=torch.int32, device="cuda"), scale)
    assert cache.device_status() == 0
    check_weights(score, pg, clean, st, kv_len, lse, scale, before, before)
