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


# ------------------------------------------------------ sampled verification

def test_oracle_verify_by_hand():
    p = np.array([[0.5, 0.25, 0.25, 0.0], [0.1, 0.2, 0.3, 0.4], [0.25, 0.25, 0.25, 0.25]])
    q = np.array([[0.25, 0.5, 0.25, 0.0], [0.4, 0.3, 0.2, 0.1], [9, 9, 9, 9]])
    # draft 1 has p / q = 1 / 2, draft 0 then 1 / 4
    assert EO.verify([9, 1, 0], p, q, [0.49, 0.24, 0], 0.5) == (2, 2, 0)       # all accepted: p of the last row
    assert EO.verify([9, 1, 0], p, q, [0.5, 0.24, 0], 0.9) == (0, 0, 0)        # u q < p is strict; the rest is 0.25 at 0
    assert EO.verify([9, 1, 0], p, q, [0.49, 0.25, 0], 0.24) == (1, 2, 0)      # the rest 0, 0, 0.1, 0.3
    assert EO.verify([9, 1, 0], p, q, [0.49, 0.25, 0], 0.26) == (1, 3, 0)
    assert EO.verify([9, 1], p, None, [0.3, 0], 0.7) == (0, 2, 0)              # without q: p but for the draft
    assert EO.verify([9], p, q, [0], 0.0) == (0, 0, 0)
    assert EO.verify([9, 4], p, q, [0, 0], 0.0)[2] == EO.BAD_TOKEN


def test_oracle_verify_keeps_the_target_distribution():
    """Over a fine grid of u and r and the drafter's own draws, the first token
    that comes out is distributed as the target's."""
    p, q = np.array([[0.5, 0.2, 0.2, 0.1], [0.25] * 4]), np.array([[0.1, 0.6, 0.2, 0.1], [0.25] * 4])
    grid = (np.arange(64) + 0.5) / 64
    out = np.zeros(4)
    for x in range(4):
        for u in grid:
            for r in grid:
                a, t, status = EO.verify([0, x], p, q, [u, 0], r)
                assert status == 0
                out[x if a else t] += q[0, x] / 64 ** 2
    # a threshold inside a cell of the grid is off by at most a cell
    np.testing.assert_allclose(out, p[0], atol=2 / 64)


def _sampled(L, n_req=3, n_tok=7, vocab=100, dtype=2, q_start=FAKE, token=FAKE * 2, p=FAKE * 3, ps=100, q=FAKE * 4, qs=100,
             u=FAKE * 5, r=FAKE * 6, kv_len=FAKE * 7, acc=FAKE * 8, nxt=FAKE * 9, held=FAKE * 10, status=FAKE * 11):
    return L.verify_sampled(n_req, n_tok, vocab, dtype, q_start, token, p, ps, q, qs, u, r, kv_len, acc, nxt, held, status, None)


@no_gpu_here
def test_good_verifications_reach_the_device_check(L):
    for kw in (dict(), dict(q=None, qs=0), dict(kv_len=None, held=None), dict(dtype=0, p=FAKE + 2), dict(dtype=1, q=FAKE + 2),
               dict(p=FAKE + 4), dict(ps=101, qs=1000), dict(held=FAKE * 7), dict(n_tok=0, p=None, token=None, u=None)):
        assert _sampled(L, **kw) in NO_GPU, kw


def test_a_verification_of_nothing(L):
    assert _sampled(L, n_req=0, q_start=None, r=None, acc=None, nxt=None) == skv.SKV_OK


@pytest.mark.parametrize("bad", [
    dict(n_req=-1), dict(n_tok=-1), dict(vocab=0), dict(dtype=3), dict(dtype=-1), dict(q_start=None), dict(token=None),
    dict(token=FAKE + 2), dict(p=None), dict(p=FAKE + 2), dict(dtype=0, p=FAKE + 1), dict(ps=99), dict(qs=99), dict(q=FAKE + 2),
    dict(u=None), dict(r=None), dict(r=FAKE + 1), dict(kv_len=None), dict(held=None), dict(acc=None), dict(nxt=None),
    dict(status=None), dict(status=FAKE + 2), dict(acc=FAKE * 9), dict(nxt=FAKE * 9 - 8 + FAKE), dict(held=FAKE * 7 + 4),
    dict(acc=FAKE), dict(nxt=FAKE * 2 + 24), dict(held=FAKE * 5 + 4), dict(status=FAKE * 6), dict(acc=FAKE * 7), dict(status=FAKE * 10)])
def test_bad_verifications(L, bad):
    assert _sampled(L, **bad) == skv.SKV_ERR_INVALID, bad


@pytest.mark.parametrize("big", [dict(n_req=(1 << 24) + 1), dict(n_tok=(1 << 30) + 1), dict(vocab=(1 << 30) + 1)])
def test_verifications_refused_as_too_large(L, big):
    assert _sampled(L, **big) == skv.SKV_ERR_UNSUPPORTED


# ------------------------------------------------------------------ eviction

def test_oracle_select_by_hand():
    score, pos = [5, 1, 9, 2, 2, 0.5], [0, 7, 3, 4, 5, 6]
    assert EO.select(score, pos, 6, 8, 1, 2) == []
    # protected: position 0, and 6 and 7; of the others the 9
    assert EO.select(score, pos, 4, 8, 1, 2) == [(3, 5)]
    assert EO.select(score, pos, 3, 8, 1, 2) == [(2, 5)]
    # nothing protected: 9, 5, then the first of the two 2s
    assert EO.select(score, pos, 3, 8, 0, 0) == [(1, 3)]
    assert EO.select([0.0, -0.0, float("nan"), -1.0], [0, 1, 2, 3], 2, 4, 0, 0) == []
    assert EO.select([float("nan"), -1.0, float("inf")], [0, 1, 2], 2, 3, 0, 0) == [(0, 2)]


def test_oracle_select_keeps_the_best():
    rng = np.random.default_rng(1)
    for _ in range(50):
        n = int(rng.integers(2, 60))
        keep = int(rng.integers(1, n))
        score, pos = rng.integers(0, 9, n).astype(float), rng.permutation(n)
        place = list(range(n))
        for to, src in EO.select(score, pos, keep, n, 2, 5):
            assert to < keep <= src
            place[to] = src
        got = place[:keep]
        assert len(set(got)) == keep
        best = sorted(range(n), key=lambda j: (not (pos[j] < 2 or pos[j] >= n - 5), -score[j] if 2 <= pos[j] < n - 5 else 0, j))[:keep]
        assert set(got) == set(best)


def _weight(L, pool=None, hq=4, n_req=3, n_tok=5, q=FAKE * 5, qs=256, q_start=FAKE * 6, kv_len=FAKE * 7, lse=FAKE * 8,
            position=FAKE * 9, add=FAKE * 10, score=FAKE * 10, pos=FAKE * 11, ws=FAKE * 4096, ws_bytes=None, scale=1.0):
    n = L.skv_attn_workspace_bytes() if ws_bytes is None else ws_bytes
    return L.paged_attn_weight(ctypes.byref(pool or _pool()), hq, n_req, n_tok, q, qs, q_start, kv_len, lse, position, add, score,
                               pos, ws, n, scale, None)


def _select(L, pool=None, n_layer=2, n_req=3, kv_len=FAKE * 5, keep=FAKE * 6, evicted=FAKE * 7, sink=1, recent=2, score=FAKE * 8,
            pos=FAKE * 9, move=FAKE * 10, n_move=FAKE * 11):
    return L.kv_evict_plan(ctypes.byref(pool or _pool()), n_layer, n_req, kv_len, keep, evicted, sink, recent, score, pos, move, n_move, None)


def _move(L, pool=None, n_layer=2, n_req=3, kv_len=FAKE * 5, move=FAKE * 6, n_move=FAKE * 7, score=FAKE * 8, pos=FAKE * 9):
    return L.kv_evict_move(ctypes.byref(pool or _pool()), n_layer, n_req, kv_len, move, n_move, score, pos, None)


@no_gpu_here
def test_good_evictions_reach_the_device_check(L):
    for kw in (dict(), dict(add=None), dict(add=FAKE * 12), dict(pool=_pool(v=0)), dict(hq=256, qs=256 * 64, q=FAKE * 64),
               dict(n_req=skv.SKV_PAGED_MAX_REQUESTS, q_start=FAKE * 32, kv_len=FAKE * 64, pool=_pool(block_table=FAKE * 128))):
        assert _weight(L, **kw) in NO_GPU, kw
    for kw in (dict(), dict(evicted=None), dict(pool=_pool(k=0, v=0)), dict(sink=0, recent=0), dict(sink=2 ** 31 - 1)):
        assert _select(L, **kw) in NO_GPU, kw
    assert _move(L) in NO_GPU


def test_evictions_of_nothing(L):
    assert _weight(L, n_req=0) == _weight(L, n_tok=0) == skv.SKV_OK
    for call in (_select, _move):
        assert call(L, n_layer=0) == call(L, n_req=0) == skv.SKV_OK


@pytest.mark.parametrize("bad", [
    dict(hq=0), dict(hq=3), dict(n_req=-1), dict(n_tok=-1), dict(q=None), dict(q=FAKE + 8), dict(qs=255), dict(qs=248), dict(q_start=None),
    dict(kv_len=None), dict(kv_len=FAKE + 2), dict(lse=None), dict(position=None), dict(add=FAKE * 10 + 4), dict(add=FAKE * 12 + 2),
    dict(score=None), dict(pos=None), dict(ws=None), dict(ws_bytes=16), dict(ws=FAKE * 4096 + 8), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), dict(pos=FAKE * 10 + 4), dict(score=FAKE * 5), dict(pos=FAKE * 8 + 8),
    dict(score=FAKE), dict(pos=FAKE * 3), dict(score=FAKE * 6), dict(pos=FAKE * 4), dict(ws=FAKE)])
def test_bad_weights(L, bad):
    assert _weight(L, **bad) == skv.SKV_ERR_INVALID, bad


@pytest.mark.parametrize("bad", [
    dict(n_layer=-1), dict(n_req=-1), dict(kv_len=None), dict(keep=None), dict(keep=FAKE + 1), dict(evicted=FAKE + 2), dict(sink=-1),
    dict(recent=-1), dict(score=None), dict(score=FAKE * 8 + 4), dict(pos=None), dict(pos=FAKE * 9 + 8), dict(move=None),
    dict(move=FAKE * 10 + 8), dict(n_move=None), dict(move=FAKE * 8), dict(move=FAKE * 9 + 1024), dict(n_move=FAKE * 6), dict(n_move=FAKE * 10 + 32),
    dict(move=FAKE * 5 - 32), dict(n_move=FAKE * 3), dict(n_move=FAKE * 4)])
def test_bad_evict_plans(L, bad):
    assert _select(L, **bad) == skv.SKV_ERR_INVALID, bad


@pytest.mark.parametrize("bad", [
    dict(n_layer=-1), dict(n_req=-1), dict(kv_len=None), dict(move=None), dict(move=FAKE * 6 + 8), dict(n_move=None), dict(score=None),
    dict(pos=None), dict(pos=FAKE * 9 + 4), dict(score=FAKE), dict(pos=FAKE * 2), dict(score=FAKE * 6), dict(pos=FAKE * 8 + 16),
    dict(score=FAKE * 7 - 32), dict(pos=FAKE * 5 - 16), dict(score=FAKE * 3), dict(pos=FAKE * 4 - 1024),
    dict(pool=_pool(v=FAKE + 64)), dict(pool=_pool(k=FAKE + 8)), dict(pool=_pool(head_dim=32)), dict(pool=_pool(v=0))])
def test_bad_moves(L, bad):
    assert _move(L, **bad) == skv.SKV_ERR_INVALID, bad


@pytest.mark.parametrize("bad", [
    dict(n_page=0), dict(page_size=24), dict(max_block=0), dict(status=0), dict(block_table=0), dict(n_kv_head=0), dict(n_kv_head=1 << 29)])
def test_evictions_of_a_bad_pool(L, bad):
    for call in (_weight, _select, _move):
        assert call(L, pool=_pool(**bad)) == skv.SKV_ERR_INVALID, (call, bad)
    assert L.paged_attn_weight(None, 4, 1, 1, *[FAKE] * 1, 256, *[FAKE] * 7, FAKE, 0, 1.0, None) == skv.SKV_ERR_INVALID
    assert L.kv_evict_plan(None, 1, 1, FAKE, FAKE, None, 0, 0, FAKE, FAKE, FAKE, FAKE, None) == skv.SKV_ERR_INVALID
    assert L.kv_evict_move(None, 1, 1, FAKE, FAKE, FAKE, FAKE, FAKE, None) == skv.SKV_ERR_INVALID


def test_evictions_refused_as_too_large(L):
    assert _weight(L, n_req=skv.SKV_PAGED_MAX_REQUESTS + 1) == skv.SKV_ERR_UNSUPPORTED
    assert _weight(L, hq=258) == skv.SKV_ERR_UNSUPPORTED                 # 129 query heads per kv head
    assert _weight(L, n_tok=1 << 30) == skv.SKV_ERR_UNSUPPORTED
    # 2^18 query tiles of 64 tokens (two query heads per kv head); 2^31 rows
    assert _weight(L, n_tok=(1 << 24) + 1) == skv.SKV_ERR_UNSUPPORTED
    assert _weight(L, hq=256, qs=256 * 64, n_tok=(1 << 18) + 1) == skv.SKV_ERR_UNSUPPORTED
    for call in (_select, _move):
        assert call(L, n_layer=1 << 15, n_req=1 << 11) == skv.SKV_ERR_UNSUPPORTED


def test_scores_that_are_no_tensors():
    with pytest.raises(TypeError):
        skv.PagedScores(3, 4)
