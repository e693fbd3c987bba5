"""Host-side refusals of buffers of a paged plan that overlap, without a GPU."""
import ctypes
import itertools

import pytest
import torch

from streaming_kv_cache_gb300 import build as B
from streaming_kv_cache_gb300 import skv

FAKE = 0x10000     # never dereferenced: every case fails validation or stops at the device check
NO_GPU = (skv.SKV_ERR_CUDA, skv.SKV_ERR_UNSUPPORTED)
no_gpu_here = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on the made-up pointers")


@pytest.fixture(scope="module")
def L():
    B.build()
    return skv.lib()


# ------------------------------------------------------------------- plan

N_REQ, N_TOK, N_PAGE, MAX_BLOCK = 3, 5, 8, 4
SIZE = dict(state=N_REQ + 2, new_len=N_REQ, queue=N_PAGE, q_start=N_REQ + 1, kv_len=N_REQ, next_state=N_REQ + 2,
            position=N_TOK, slot=N_TOK, block_table=N_REQ * MAX_BLOCK, status=1)   # int32 each


def _plan(L, **at):
    p = {name: FAKE * (i + 1) for i, name in enumerate(SIZE)}
    p.update(at)
    pool = skv.skv_paged(n_page=N_PAGE, page_size=16, max_block=MAX_BLOCK, block_table=p["block_table"],
                         status=p["status"])
    return L.kv_paged_plan(ctypes.byref(pool), N_REQ, N_TOK, p["state"], p["new_len"], p["queue"], p["q_start"],
                           p["kv_len"], p["next_state"], p["position"], p["slot"], None)


PAIRS = [p for p in itertools.permutations(SIZE, 2) if set(p) != {"state", "new_len"}]


@pytest.mark.parametrize("a,b", PAIRS)
def test_plan_refuses_buffers_that_overlap(L, a, b):
    """Every CTA of the plan reads the lengths, the queue and the table while
    others write already: an output over any of them would give the CTAs
    different plans."""
    base = FAKE * (list(SIZE).index(b) + 1)
    for at in (base, base + 4 * (SIZE[b] - 1), base - 4 * (SIZE[a] - 1)):
        assert _plan(L, **{a: at}) == skv.SKV_ERR_INVALID, at - base


@no_gpu_here
@pytest.mark.parametrize("a,b", PAIRS)
def test_plan_takes_buffers_that_touch(L, a, b):
    base = FAKE * (list(SIZE).index(b) + 1)
    for at in (base + 4 * SIZE[b], base - 4 * SIZE[a]):
        assert _plan(L, **{a: at}) in NO_GPU, at - base


@no_gpu_here
def test_plan_reads_one_buffer_twice(L):
    assert _plan(L, new_len=FAKE) in NO_GPU          # both only read
