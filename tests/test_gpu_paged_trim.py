"""kv_paged_trim and the plan of an evicting cache on the GPU, bit for bit
against the oracle."""
import numpy as np
import pytest
import torch

from oracle import evict_oracle as EO
from paged_harness import ints
from streaming_kv_cache_gb300 import skv

pytestmark = pytest.mark.gpu


def _cache(state, table, queue, page):
    return skv.PagedCache.wrap(block_table=ints(table.tolist()), page_queue=ints(queue.tolist()), page_size=page,
                               state=ints([int(x) for x in state]))


def _trim(state, keep, table, queue, page, mode):
    cache = _cache(state, table, queue, page)
    assert cache.evicts == (mode > 0)
    want, wq, status = EO.trim(state, keep, table, queue, page, mode)
    for _ in range(2):      # repeated on the same state: the same answer
        got = skv.kv_paged_trim(cache, ints([int(x) for x in keep]), evict=mode == 2)
        np.testing.assert_array_equal(got.cpu().numpy(), want)
        np.testing.assert_array_equal(cache.page_queue.cpu().numpy(), wq)
    assert cache.device_status() == status
    assert cache.state.tolist() == [int(x) for x in state] and cache.block_table.tolist() == table.tolist()
    return want, wq, status


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("n_req,page,cols", [(1, 16, 1), (1, 16, 3000), (7, 48, 9), (513, 16, 30), (4096, 64, 5)])
def test_trim(mode, n_req, page, cols):
    rng = np.random.default_rng(n_req + mode)
    held = rng.integers(0, cols * page + 1, n_req)
    held[0] = cols * page
    used = [-(-int(x) // page) for x in held]
    n_page = sum(used) + 5
    ids = rng.permutation(n_page)
    table, at = np.full((n_req, cols), -1, dtype=np.int32), 0
    for b, n in enumerate(used):
        table[b, :n] = ids[at:at + n]
        at += n
    queue = np.full(n_page, -1, dtype=np.int32)
    head = int(rng.integers(n_page))
    for i in range(5):
        queue[(head + i) % n_page] = ids[at + i]
    state = held.tolist() + [head, 5] + (rng.integers(0, 2 ** 31, n_req).tolist() if mode else [])
    keep = np.where(rng.random(n_req) < 0.3, held, rng.integers(0, cols * page + 40, n_req))
    keep[0] = 0 if mode == 0 else 1
    _, _, status = _trim(state, keep, table, queue, page, mode)
    assert status == 0


@pytest.mark.parametrize("state,keep", [
    ([-1, 65, 5, 0, 0, 1, 2, 3], [1, 1, 1]), ([40, 40, 40, 0, 0, -5, 2 ** 31 - 1, 3], [1, -1, 1]),
    ([40, 40, 40, 9, 0, 1, 2, 3], [0, 0, 0]), ([40, 40, 40, -1, 0, 1, 2, 3], [0, 0, 0]),
    ([40, 40, 40, 0, 9, 1, 2, 3], [0, 0, 0]), ([64, 64, 64, 7, 3, 1, 2, 3], [0, 0, 20]),
    ([64, 64, 64, 2, 8, 1, 2, 3], [0, 64, 0]), ([64, 64, 64, 2, 0, 2 ** 31 - 10, -2 ** 31, 3], [1, 0, 2 ** 31 - 1])])
@pytest.mark.parametrize("mode", [0, 1, 2])
def test_trim_of_values_out_of_range(state, keep, mode):
    table = np.arange(12, dtype=np.int32).reshape(3, 4)      # some pages outside the pool of 8
    _trim(state if mode else state[:5], keep, table, np.arange(8, dtype=np.int32), 16, mode)


@pytest.mark.parametrize("n_req,page,n_page,cols,most", [(1, 16, 4, 3, 20), (33, 64, 400, 9, 200), (4096, 16, 20000, 4, 40)])
def test_plans_and_trims_over_random_steps(n_req, page, n_page, cols, most):
    """Positions go on over evictions and start anew with a new request."""
    rng = np.random.default_rng(n_req)
    table = np.full((n_req, cols), -1, dtype=np.int32)
    queue = rng.permutation(n_page).astype(np.int32)
    state = np.array([0] * n_req + [n_page - 1, n_page] + [0] * n_req, dtype=np.int32)
    for step in range(8):
        new = rng.integers(-1, most, n_req) if step % 2 == 0 else rng.integers(0, 2, n_req)
        n_tok = max(0, int(np.maximum(new, 0).sum()) + [0, 5, -3][step % 3])
        cache = _cache(state, table, queue, page)
        want, status = EO.plan_evicting(state, new, table, queue, page, n_tok)
        for _ in range(2):
            p = skv.kv_paged_plan(cache, ints(new.tolist()), n_tok)
            got = dict(q_start=p.q_start, kv_len=p.kv_len, next_state=p.next_state, position=p.position, slot=p.slot,
                       table=cache.block_table, queue=cache.page_queue)
            for name in want:
                np.testing.assert_array_equal(got[name].cpu().numpy(), want[name], err_msg=name)
        assert cache.device_status() == status
        cache.advance(p)
        assert cache.state.tolist() == want["next_state"].tolist()
        state, queue, _ = _trim(want["next_state"], rng.integers(0, cols * page, n_req), want["table"], want["queue"], page,
                                1 + step % 2)
        table = want["table"]


@pytest.mark.parametrize("words", [[-3, 5, 2 ** 31 - 1], [-1, -1, -1]])
def test_plan_of_evicted_words_out_of_range(words):
    state, table = [5, 0, 9, 0, 4] + words, np.arange(12, dtype=np.int32).reshape(3, 4) % 8
    queue = np.arange(8, dtype=np.int32)
    cache = _cache(state, table, queue, 16)
    want, status = EO.plan_evicting(state, [2, 2, 2], table, queue, 16, 8)
    p = skv.kv_paged_plan(cache, ints([2, 2, 2]), 8)
    assert p.position.tolist() == want["position"].tolist() and p.next_state.tolist() == want["next_state"].tolist()
    assert cache.device_status() == status and status & EO.BAD_LEN


def test_binding_refusals():
    cache = _cache([5, 5, 0, 4], np.zeros((2, 3), dtype=np.int32), np.arange(8, dtype=np.int32), 16)
    with pytest.raises(ValueError, match="no evicted words"):
        skv.kv_paged_trim(cache, ints([1, 1]), evict=True)
    with pytest.raises(ValueError):
        skv.kv_paged_trim(cache, ints([1, 1, 1]))
    with pytest.raises(TypeError):
        skv.kv_paged_trim(cache, ints([1, 1]).float())
    with pytest.raises(ValueError):
        skv.kv_paged_trim(cache, ints([1, 1]), next_state=ints([0] * 6))
    with pytest.raises(skv.SkvError):
        skv.kv_paged_trim(cache, ints([1, 1]), next_state=cache.state)
    with pytest.raises(ValueError, match="evicted words"):
        skv.kv_paged_plan(cache, ints([1, 1]), 2, plan=skv.PagedPlan.empty(2, 2, evicts=True))
