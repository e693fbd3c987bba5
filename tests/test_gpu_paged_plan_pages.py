"""Plans of steps that give back far more pages than they have tokens, beside
the oracle bit for bit."""
import numpy as np
import pytest

from oracle import paged_oracle as PO
from paged_harness import ints
from streaming_kv_cache_gb300 import skv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_req,page,most,finished,n_tok", [
    (1, 16, 131072, 1, 0), (8, 16, 131072, 3, 8), (8, 16, 131072, 8, 3), (300, 32, 8192, 150, 40), (4096, 16, 512, 4000, 96)])
def test_plan_that_frees_many_pages(n_req, page, most, finished, n_tok):
    rng = np.random.default_rng(n_req)
    held = rng.integers(most // 2, most + 1, n_req)
    cols = most // page + 2
    used = -(-held // page)
    n_page = int(used.sum()) + 200
    ids = rng.permutation(n_page).astype(np.int32)
    table = np.full((n_req, cols), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = ids[at:at + n]
        at += n
    head = int(rng.integers(0, n_page))
    queue = np.full(n_page, -1, dtype=np.int32)
    queue[(head + np.arange(n_page - at)) % n_page] = ids[at:]
    state = np.concatenate([held, [head, n_page - at]]).astype(np.int32)
    new = np.ones(n_req, dtype=np.int32)
    new[rng.permutation(n_req)[:finished]] = -1
    cache = skv.PagedCache.wrap(block_table=ints(table.tolist()), page_queue=ints(queue.tolist()), page_size=page,
                                state=ints(state.tolist()))
    p = skv.kv_paged_plan(cache, ints(new.tolist()), n_tok)
    want, status = PO.plan(state, new, table, queue, page, n_tok)
    got = dict(q_start=p.q_start, kv_len=p.kv_len, next_state=p.next_state, position=p.position, slot=p.slot,
               table=cache.block_table, queue=cache.page_queue)
    for name in want:
        np.testing.assert_array_equal(got[name].cpu().numpy(), want[name], err_msg=name)
    assert cache.device_status() == status
    assert int(want["next_state"][-1]) >= int(used[new < 0].sum())
