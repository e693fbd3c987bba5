"""Eviction and trimming of the paged cache without a GPU: the oracle by hand
and by invariants, and the refusals of the calls."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

from oracle import evict_oracle as EO
from streaming_kv_cache_gb300 import build as B
from streaming_kv_cache_gb300 import skv

FAKE = 0x10000     # never dereferenced: every case fails validation or stops at the device check
NO_GPU = (skv.SKV_ERR_CUDA, skv.SKV_ERR_UNSUPPORTED)
no_gpu_here = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on the made-up pointers")


@pytest.fixture(scope="module")
def L():
    B.build()
    return skv.lib()


# ------------------------------------------------------------------ oracle

def test_oracle_trim_by_hand():
    """Page size 16: request 0 keeps 16 of 40 tokens (pages 5 | 3, 1), request 1
    all of its 7, request 2 none of its 20 (pages 6, 2)."""
    table = np.array([[5, 3, 1], [4, -1, -1], [6, 2, -1]], dtype=np.int32)
    queue = np.array([9, 9, 9, 9, 9, 9, 0, 7], dtype=np.int32)
    state = [40, 7, 20, 6, 2, 100, 0, 3]
    nxt, got, status = EO.trim(state, [16, 9, 0], table, queue, 16, 2)
    assert nxt.tolist() == [16, 7, 0, 6, 6, 124, 0, 0] and status == 0
    assert got.tolist() == [3, 1, 6, 2, 9, 9, 0, 7]
    nxt, _, _ = EO.trim(state, [16, 9, 0], table, queue, 16, 1)
    assert nxt.tolist() == [16, 7, 0, 6, 6, 100, 0, 0]
    nxt, _, _ = EO.trim(state[:5], [16, 9, 0], table, queue, 16, 0)
    assert nxt.tolist() == [16, 7, 0, 6, 6]


def test_oracle_steps_keep_every_page_once():
    rng = np.random.default_rng(0)
    n_req, page, n_page = 6, 16, 40
    table = np.full((n_req, 9), -1, dtype=np.int32)
    queue = rng.permutation(n_page).astype(np.int32)
    state = np.array([0] * n_req + [0, n_page] + [0] * n_req, dtype=np.int32)
    for step in range(60):
        got, status = EO.plan_evicting(state, rng.integers(-1, 40, n_req), table, queue, page, 300)
        table, queue = got["table"], got["queue"]
        before = got["next_state"]
        state, queue, more = EO.trim(before, rng.integers(0, 90, n_req), table, queue, page, 1 + step % 2)
        assert (status | more) & (EO.BAD_LEN | EO.BAD_PAGE) == 0
        held = [int(table[b, j]) for b in range(n_req) for j in range(-(-int(state[b]) // page))]
        free = [int(queue[(state[n_req] + i) % n_page]) for i in range(state[n_req + 1])]
        assert sorted(held + free) == list(range(n_page))
        if step % 2:   # evicting: the next position stays where it was
            live = state[:n_req] > 0
            nxt = lambda s: (s[:n_req] + s[n_req + 2:])[live]  # noqa: E731
            assert np.array_equal(nxt(state), nxt(before))


# ---------------------------------------------------------------- refusals

def _pool(**kw):
    base = dict(n_page=8, page_size=16, n_kv_head=2, head_dim=64, dtype=0, rope_len=0, max_block=4, reserved=0,
                k=FAKE, v=FAKE * 2, block_table=FAKE * 3, rope=0, status=FAKE * 4)
    base.update(kw)
    return skv.skv_paged(**base)


def _trim(L, pool=None, n_req=3, state=FAKE * 5, keep=FAKE * 6, evicted=2, queue=FAKE * 7, nxt=FAKE * 8):
    return L.kv_paged_trim(ctypes.byref(pool or _pool()), n_req, state, keep, evicted, queue, nxt, None)


@no_gpu_here
def test_good_trims_reach_the_device_check(L):
    for mode in (0, skv.SKV_TRIM_DRAFTS, skv.SKV_TRIM_EVICTED):
        assert _trim(L, evicted=mode) in NO_GPU
    assert _trim(L, n_req=skv.SKV_PAGED_MAX_REQUESTS, queue=FAKE * 16, nxt=FAKE * 32, pool=_pool(status=FAKE * 64)) in NO_GPU
    assert _trim(L, n_req=0, keep=None) in NO_GPU
    assert _trim(L, pool=_pool(k=0, v=0)) in NO_GPU


@pytest.mark.parametrize("bad", [
    dict(n_req=-1), dict(state=None), dict(state=FAKE + 2), dict(keep=None), dict(keep=FAKE + 1), dict(evicted=3),
    dict(evicted=-1), dict(queue=None), dict(nxt=None), dict(nxt=FAKE * 8 + 1)])
def test_bad_trims(L, bad):
    assert _trim(L, **bad) == skv.SKV_ERR_INVALID, bad


@pytest.mark.parametrize("bad", [
    dict(n_page=0), dict(page_size=24), dict(max_block=0), dict(status=0), dict(block_table=0), dict(n_page=1 << 27)])
def test_trims_of_a_bad_pool(L, bad):
    assert _trim(L, pool=_pool(**bad)) == skv.SKV_ERR_INVALID, bad
    assert L.kv_paged_plan_evicting(ctypes.byref(_pool(**bad)), 3, 5, *[FAKE * i for i in range(5, 13)], None) == skv.SKV_ERR_INVALID


def test_trims_refused_as_too_large(L):
    assert _trim(L, n_req=skv.SKV_PAGED_MAX_REQUESTS + 1) == skv.SKV_ERR_UNSUPPORTED
    assert L.kv_paged_trim(None, 3, FAKE, FAKE, 0, FAKE, FAKE, None) == skv.SKV_ERR_INVALID


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_trim_refuses_buffers_that_overlap(L, mode):
    words = 8 if mode else 5
    size = dict(state=words, keep=3, block_table=12, queue=8, nxt=words, status=1)
    at = {name: FAKE * (i + 1) for i, name in enumerate(size)}

    def call(**kw):
        p = dict(at, **kw)
        return _trim(L, pool=_pool(block_table=p["block_table"], status=p["status"]), evicted=mode, state=p["state"],
                     keep=p["keep"], queue=p["queue"], nxt=p["nxt"])

    for a, b in itertools.permutations(size, 2):
        if {a, b} <= {"state", "keep", "block_table"}:
            continue
        for x in (at[b], at[b] + 4 * (size[b] - 1), at[b] - 4 * (size[a] - 1)):
            assert call(**{a: x}) == skv.SKV_ERR_INVALID, (a, b)
        if not torch.cuda.is_available():
            for x in (at[b] + 4 * size[b], at[b] - 4 * size[a]):
                assert call(**{a: x}) in NO_GPU, (a, b)


def test_plan_evicting_counts_the_evicted_words_in_its_overlaps(L):
    """state and next_state are 2 n_req + 2 words long."""
    def call(state, nxt):
        return L.kv_paged_plan_evicting(ctypes.byref(_pool()), 3, 5, state, FAKE * 6, FAKE * 7, FAKE * 8, FAKE * 9, nxt,
                                        FAKE * 11, FAKE * 12, None)
    assert call(FAKE * 10 - 4 * 7, FAKE * 10) == skv.SKV_ERR_INVALID
    assert call(FAKE * 10 + 4 * 7, FAKE * 10) == skv.SKV_ERR_INVALID
    if not torch.cuda.is_available():
        assert call(FAKE * 10 - 4 * 8, FAKE * 10) in NO_GPU
