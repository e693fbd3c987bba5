"""kv_evict_plan's counts of protected positions beyond 32 bits: all that a
cache may hold."""
import pytest
import torch

from paged_harness import ints
from streaming_kv_cache_gb300 import skv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sink,recent", [(2 ** 31 - 1, 0), (2 ** 32, 0), (10 ** 12, 5), (0, 2 ** 31 - 1), (0, 2 ** 32), (0, 2 ** 32 + 1), (3, 2 ** 63)])
def test_more_protected_positions_than_there_are(sink, recent):
    """Every token is protected, so the first ones stay; without protection it
    would be the last, of the largest scores."""
    cache = skv.PagedCache(4, 16, 1, 64, 1, 4, n_layer=1, evicts=True)
    cache.block_table.copy_(ints([[0, 1, 2, 3]]))
    scores = skv.PagedScores.empty(cache)
    scores.score.copy_(torch.arange(64, device="cuda", dtype=torch.float32).view(scores.score.shape))
    scores.pos.copy_(torch.arange(64, device="cuda", dtype=torch.int32).view(scores.pos.shape))
    skv.kv_evict_plan(cache, scores, ints([60]), ints([20]), sink, recent)
    assert cache.device_status() == 0 and scores.n_move.tolist() == [[[0]]]


@pytest.mark.parametrize("sink,recent", [(-1, 0), (0, -2 ** 31), (-2 ** 32, 0), (0, -2 ** 32 + 5), (-2 ** 63, 7)])
def test_negative_counts_are_refused(sink, recent):
    cache = skv.PagedCache(4, 16, 1, 64, 1, 4, n_layer=1, evicts=True)
    with pytest.raises(skv.SkvError):
        skv.kv_evict_plan(cache, skv.PagedScores.empty(cache), ints([0]), ints([0]), sink, recent)
