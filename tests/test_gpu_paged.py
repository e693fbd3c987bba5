"""The paged cache and cross attention on the GPU against the fp64 oracle:
plans and writes bit for bit (rotated values within half a step of their
type), attention within the bound that paged_harness.check derives."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO
from paged_harness import DT, Pages, check, f64, ints, randn, run_paged, starts
from streaming_kv_cache_gb300 import skv

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------- plan

def _run_plan(state, new_len, table, queue, page, n_tok):
    cache = skv.PagedCache.wrap(block_table=ints(table.tolist()), page_queue=ints(queue.tolist()), page_size=page,
                                state=ints(list(state)))
    want, status = PO.plan(state, new_len, table, queue, page, n_tok)
    first = None
    for _ in range(2):      # repeated on the same state: the same plan
        p = skv.kv_paged_plan(cache, ints(list(new_len)), n_tok)
        got = dict(q_start=p.q_start, kv_len=p.kv_len, next_state=p.next_state, position=p.position, slot=p.slot,
                   table=cache.block_table, queue=cache.page_queue)
        got = {k: v.cpu().numpy() for k, v in got.items()}
        for name in want:
            np.testing.assert_array_equal(got[name], want[name], err_msg=name)
        first = first or got
    assert cache.state.tolist() == [int(x) for x in state]
    assert cache.device_status() == status
    return want, status


@pytest.mark.parametrize("n_req,page,n_page,cols,most", [
    (1, 16, 4, 3, 20), (7, 16, 60, 8, 30), (33, 64, 400, 9, 200), (600, 48, 3000, 6, 150), (4096, 16, 20000, 4, 40)])
def test_plan_over_random_steps(n_req, page, n_page, cols, most):
    """Steps of mixed new, paused and finished requests, from a small queue
    that runs dry at times, advancing on the oracle's own state."""
    rng = np.random.default_rng(n_req)
    table = np.full((n_req, cols), -1, dtype=np.int32)
    queue = rng.permutation(n_page).astype(np.int32)
    state = np.array([0] * n_req + [n_page - 1, n_page], dtype=np.int32)
    seen = 0
    for step in range(8):
        new = rng.integers(-1, most, n_req) if step % 2 == 0 else rng.integers(0, 2, n_req)
        n_tok = int(np.maximum(new, 0).sum()) + [0, 5, -3][step % 3]
        want, status = _run_plan(state, new, table, queue, page, max(0, n_tok))
        table, queue, state = want["table"], want["queue"], want["next_state"]
        seen |= status
    assert n_req < 7 or seen & PO.TABLE_FULL


def test_plan_when_the_queue_runs_dry():
    table = np.array([[0, -1], [1, -1], [2, -1], [3, -1]], dtype=np.int32)
    queue = np.array([4, 5, 9, 9, 9, 9], dtype=np.int32)
    want, status = _run_plan([10, 16, 16, 3, 0, 2], [1, 17, 9, 2], table, queue, 16, 40)
    # request 1 would reach 33 tokens, a row holds 32
    assert status & PO.TABLE_FULL
    want, status = _run_plan([16, 16, 16, 16, 0, 2], [1, 1, 1, 0], table, queue, 16, 8)
    assert status == PO.NO_PAGE
    assert want["kv_len"].tolist() == [17, 17, 0, 16]
    assert want["slot"].tolist() == [64, 80, -1, -1, -1, -1, -1, -1]


@pytest.mark.parametrize("state,new", [
    ([-1, 5, 5, 0, 4], [1, 1, 1]), ([5, 5, 5, 0, 4], [1, -2, 1]), ([5, 2 ** 31 - 1, 5, 0, 4], [1, 1, -1]),
    ([5, 65, 5, 0, 4], [1, -1, 1]), ([5, 5, 5, 9, 4], [12, 1, 1]), ([5, 5, 5, -1, 4], [12, 1, 1]),
    ([5, 5, 5, 0, 9], [12, 1, 1]), ([5, 5, 5, 0, -1], [0, 0, 0]), ([5, 5, 5, 0, 4], [2 ** 31 - 1, 1, 1]),
    ([64, 64, 64, 0, 8], [-1, -1, -1])])
def test_plan_of_lengths_out_of_range(state, new):
    table = np.arange(12, dtype=np.int32).reshape(3, 4) % 8
    _run_plan(state, new, table, np.arange(8, dtype=np.int32), 16, 20)


@pytest.mark.parametrize("state,new", [
    ([2 ** 31 - 20, 2 ** 26 - 10, 2 ** 26, 5, 0, 2047], [32, 10, 1, 3]),
    ([2 ** 31 - 2 ** 20, 2 ** 26 - 10, 2 ** 26 + 1, 2 ** 26, 7, 2000], [-1, 11, 0, -1])])
def test_plan_of_rows_longer_than_a_request_may_be(state, new):
    """Table rows of 2^31 tokens: a length above the limit, or one that would
    pass it (and 2^31) with its new tokens, is left out."""
    rng = np.random.default_rng(3)
    table = rng.integers(0, 2047, (4, 2048)).astype(np.int32)
    want, status = _run_plan(state, new, table, rng.permutation(2047).astype(np.int32), 2 ** 20, 60)
    assert status & PO.BAD_LEN and status & PO.TABLE_FULL


def test_plan_without_requests_or_rows():
    cache = skv.PagedCache.wrap(block_table=torch.zeros((1, 2), dtype=torch.int32, device="cuda"),
                                page_queue=ints([0, 1]), page_size=16, state=ints([3, 0, 2]))
    p = skv.kv_paged_plan(cache, ints([0]), 0)
    assert p.q_start.tolist() == [0, 0] and p.kv_len.tolist() == [3] and p.next_state.tolist() == [3, 0, 2]


def test_plan_flags_a_page_outside_the_pool():
    cache = skv.PagedCache.wrap(block_table=ints([[77]]), page_queue=ints([0, 1]), page_size=16, state=ints([3, 0, 2]))
    p = skv.kv_paged_plan(cache, ints([2]), 2)
    assert p.slot.tolist() == [-1, -1] and cache.device_status() == skv.SKV_DEV_BAD_PAGE


# --------------------------------------------------------------------- write

def _half_step(x, dtype):
    """Half a step of the type at |x|, and the smallest normal's below it."""
    fi = torch.finfo(dtype)
    return np.maximum(np.abs(x), fi.tiny) * fi.eps / 2


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,hq,hkv,page,n,rope", [
    (128, 32, 8, 64, 37, True), (64, 14, 2, 48, 129, True), (64, 1, 1, 16, 1, True), (128, 5, 5, 16, 300, False),
    (128, 3, 1, 272, 70, True)])
def test_write(dtype, d, hq, hkv, page, n, rope):
    dt = DT[dtype]
    rng = np.random.default_rng(n)
    n_page = -(-n // page) + 4
    qkv = randn(1, (n, hq + 2 * hkv, d), dt)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    kp, vp = randn(2, (n_page, hkv, page, d), dt), randn(3, (n_page, hkv, page, d), dt)
    tab = None
    if rope:
        tab = torch.empty((5000, d // 2, 2), dtype=torch.float32, device="cuda")
        skv.skv_build_rope_table(tab, 1e6)
    cache = skv.PagedCache.wrap(k=kp, v=vp, block_table=torch.zeros((1, 1), dtype=torch.int32, device="cuda"), rope=tab)
    slot = rng.permutation(n_page * page)[:n]
    slot[rng.random(n) < 0.1] = -1
    pos = rng.integers(0, 5000, n)
    pos[0] = 4999
    before, guard = (kp.clone(), vp.clone()), torch.full((n + 2, hq, d), 7.0, dtype=dt, device="cuda")
    skv.kv_paged_write(cache, q, k, v, ints(pos.tolist()) if rope else None, ints(slot.tolist()), q_out=guard[1:-1])
    assert cache.device_status() == 0
    live = slot >= 0
    cs = f64(tab)[pos] if rope else None

    def turned(x):
        if cs is None:
            return x
        a, b = x[..., :d // 2], x[..., d // 2:]
        c, s = cs[:, None, :, 0], cs[:, None, :, 1]
        return np.concatenate([a * c - b * s, b * c + a * s], -1)

    def near(got, want):
        # one rounding of a sum of two fp32 products (each a half step of fp32 off)
        assert (np.abs(got - want) <= _half_step(want, dt) * (1 + 2.0 ** -8) + 2.0 ** -21).all()

    near(f64(guard[1:-1])[live], turned(f64(q))[live])
    assert (f64(guard[1:-1])[~live] == 7).all() and (f64(guard[0]) == 7).all() and (f64(guard[-1]) == 7).all()
    pages, rows = slot[live] // page, slot[live] % page
    near(f64(kp)[pages, :, rows], turned(f64(k))[live])
    np.testing.assert_array_equal(f64(vp)[pages, :, rows], f64(v)[live])
    for now, old in zip((kp, vp), before):   # nothing else has moved
        same = torch.ones((n_page, page), dtype=torch.bool)
        same[pages, rows] = False
        np.testing.assert_array_equal(f64(now.transpose(1, 2))[same.numpy()], f64(old.transpose(1, 2))[same.numpy()])


def test_write_in_place_and_without_queries():
    dt, n, hq, hkv, d, page = torch.bfloat16, 50, 4, 2, 128, 16
    q, k, v = (randn(i, (n, h, d), dt) for i, h in ((1, hq), (2, hkv), (3, hkv)))
    tab = torch.empty((100, d // 2, 2), dtype=torch.float32, device="cuda")
    skv.skv_build_rope_table(tab, 1e4)
    cache = skv.PagedCache.wrap(k=torch.zeros((4, hkv, page, d), dtype=dt, device="cuda"),
                                v=torch.zeros((4, hkv, page, d), dtype=dt, device="cuda"),
                                block_table=torch.zeros((1, 1), dtype=torch.int32, device="cuda"), rope=tab)
    pos, slot = ints(list(range(n))), ints(list(range(n)))
    want = skv.kv_paged_write(cache, q, k, v, pos, slot)
    pages = cache.k.clone()
    cache.k.zero_()
    assert skv.kv_paged_write(cache, None, k, v, pos, slot) is None
    assert torch.equal(cache.k, pages)
    skv.kv_paged_write(cache, q, k, v, pos, slot, q_out=q)
    assert torch.equal(q, want)
    with pytest.raises(skv.SkvError):
        wide = torch.empty((2 * n, hq, d), dtype=dt, device="cuda")
        skv.kv_paged_write(cache, wide[1:n + 1], k, v, pos, slot, q_out=wide[:n])


def test_write_flags_bad_slots_and_positions():
    dt, hkv, d, page = torch.float16, 1, 64, 16
    k = randn(1, (4, hkv, d), dt)
    tab = torch.ones((10, d // 2, 2), dtype=torch.float32, device="cuda")
    for slot, pos, bit in (([0, 32, 2, -5], [0, 1, 2, 99], skv.SKV_DEV_BAD_PAGE), ([0, 2 ** 31 - 1, 2, 3], [0] * 4, skv.SKV_DEV_BAD_PAGE),
                           ([0, 1, 2, 3], [0, 10, 9, 3], skv.SKV_DEV_BAD_POS), ([0, 1, 2, 3], [0, -1, 9, 3], skv.SKV_DEV_BAD_POS)):
        kp = torch.zeros((2, hkv, page, d), dtype=dt, device="cuda")
        cache = skv.PagedCache.wrap(k=kp, v=kp.clone(), block_table=torch.zeros((1, 1), dtype=torch.int32, device="cuda"), rope=tab)
        skv.kv_paged_write(cache, None, k, k, ints(pos), ints(slot))
        assert cache.device_status() == bit
        np.testing.assert_array_equal(f64(cache.v)[0, 0, 2], f64(k)[2, 0])
        assert (f64(cache.v)[0, 0, 1] == 0).all() and (f64(cache.v)[1] == 0).all()


# ----------------------------------------------------------------- attention

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 48, 64, 128, 272])
def test_paged_decode(dtype, d, page):
    kv = [1, 2, 15, 16, 17, 63, 64, 127, 128, 129, 255, 256, 257, 300, 700, 1111]
    run_paged(skv, d + page, [1] * len(kv), kv, page, 8, 2, d, DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 2), (3, 1), (6, 2), (10, 2), (7, 1), (8, 1), (12, 1), (40, 1), (128, 1)])
def test_paged_chunks_and_single_tokens(dtype, hq, hkv):
    """Chunk edges around the query tiles and key tiles, no context and some."""
    ql = [1, 7, 128, 129, 40, 3, 33, 260]
    kv = [1, 7, 128, 130, 500, 300, 161, 260]
    run_paged(skv, hq, ql, kv, 32, hq, hkv, 64 if hq % 2 else 128, DT[dtype])


@pytest.mark.parametrize("d", [64, 128])
def test_paged_long_context_is_split(d):
    run_paged(skv, 5, [1], [9001], 64, 8, 1, d, torch.bfloat16)
    run_paged(skv, 6, [2, 1], [20000, 130], 16, 4, 2, d, torch.float16)
    run_paged(skv, 7, [200], [5000], 128, 4, 1, d, torch.bfloat16)


def test_paged_many_requests():
    rng = np.random.default_rng(3)
    kv = rng.integers(1, 200, 700).tolist()
    run_paged(skv, 8, [1] * 700, kv, 16, 4, 4, 64, torch.bfloat16)
    ql = [min(k, int(x)) for k, x in zip(kv, rng.integers(0, 40, 700))]
    run_paged(skv, 9, ql, kv, 16, 2, 1, 64, torch.bfloat16)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_paged_sharp_scores(dtype):
    """Scores of some hundreds: late keys that dwarf the first tiles' maximum."""
    run_paged(skv, 11, [1, 100, 3], [1500, 900, 2000], 64, 4, 2, 128, DT[dtype], q_mul=40.0)


def test_paged_rows_without_keys_and_padding():
    d, hq, dt = 128, 4, torch.bfloat16
    pg = Pages(1, [40, 0, 9, 300], 16, 1, d, dt)
    cache = pg.cache(skv)
    qs = [0, 3, 8, 8, 140]
    q = randn(2, (150, hq, d), dt)
    q[3:8] = float("nan")
    out = torch.full((150, hq, d), 5.0, dtype=dt, device="cuda")
    lse = torch.full((hq, 150), 5.0, device="cuda")
    skv.paged_attn(cache, q, ints(qs), ints([40, 0, 9, 300]), d ** -0.5, out=out, lse=lse)
    assert cache.device_status() == 0
    assert (out[3:8] == 0).all() and torch.isneginf(lse[:, 3:8]).all()
    assert (out[140:] == 5).all() and (lse[:, 140:] == 5).all()
    live = torch.cat([q[:3], q[8:140]])
    want, wlse, mass = PO.paged(f64(live), f64(pg.k), f64(pg.v), pg.table, [0, 3, 3, 3, 135], [40, 0, 9, 300], d ** -0.5)
    got, gl = torch.cat([out[:3], out[8:140]]), torch.cat([lse[:, :3], lse[:, 8:140]], 1)
    check(f64(got), f64(gl), want, wlse, mass, dt, 20.0, 20.0, d ** -0.5, d, 300)


def test_paged_lengths_and_pages_out_of_range():
    d, dt = 64, torch.float16
    kv = [40, 20, 50]
    for bad_kv, bad_qs, rows in (([40, -1, 50], None, range(2, 5)), ([40, 10 ** 6, 50], None, range(2, 5)),
                                 ([40, 2, 50], None, range(2, 5)), ([40, 2 ** 31 - 1, 50], None, range(2, 5)),
                                 (None, [0, 2, 2000, 7], ()), (None, [-1, 2, 5, 7], ()), (None, [0, 2, 1, 7], ())):
        pg = Pages(3, kv, 16, 1, d, dt)
        cache = pg.cache(skv)
        qs = bad_qs or [0, 2, 5, 7]
        out = torch.full((7, 2, d), 5.0, dtype=dt, device="cuda")
        skv.paged_attn(cache, randn(4, (7, 2, d), dt), ints(qs), ints(bad_kv or kv), 0.125, out=out)
        assert cache.device_status() == skv.SKV_DEV_BAD_LEN
        assert torch.isfinite(out).all()
        for r in rows:
            assert (out[r] == 0).all()
    for entry in (-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
        pg = Pages(3, kv, 16, 2, d, dt)
        bad = int(pg.table[2, 1])
        pg.table[2, 1] = entry
        cache = pg.cache(skv)
        q = randn(4, (3, 2, d), dt)
        out = skv.paged_attn(cache, q, ints([0, 1, 2, 3]), ints(kv), 0.125)
        assert cache.device_status() == skv.SKV_DEV_BAD_PAGE
        pg.table[2, 1] = bad                      # its keys and values count as zeros
        pg.k[bad], pg.v[bad] = 0.0, 0.0
        want, _, mass = PO.paged(f64(q), f64(pg.k), f64(pg.v), pg.table, [0, 1, 2, 3], kv, 0.125)
        check(f64(out), None, want, None, mass, dt, 20.0, 20.0, 0.125, d, 50)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq", [1, 8, 12, 40])
def test_paged_after_calls_that_left_nan_on_chip(hq, d):
    """Shared memory and tensor memory hold NaN from another call's keys,
    values and queries: nothing of them may reach the outputs.  Units of one
    and of two query tiles follow each other in every share."""
    dt, page = torch.bfloat16, 32
    ql, kv = [1, 7, 128, 129, 40, 3, 33, 260], [1, 7, 128, 130, 500, 300, 161, 260]
    pg = Pages(hq, kv, page, 1, d, dt)
    cache, qs = pg.cache(skv), starts(ql)
    q = randn(hq, (int(qs[-1]), hq, d), dt)
    want, wlse, mass = PO.paged(f64(q), f64(pg.k), f64(pg.v), pg.table, qs, kv, d ** -0.5)
    ws, other = skv.attn_workspace(), skv.attn_workspace()
    ws.fill_(255)                                # of any contents
    for i in range(6):
        dd, n = (d, 192 - d)[i % 2], (600, 1)[i % 3 == 2]
        pool = torch.full((64, 1, 128, dd), float("nan"), dtype=dt, device="cuda")
        bad = skv.PagedCache.wrap(k=pool, v=pool, block_table=torch.arange(64, dtype=torch.int32, device="cuda")[None])
        skv.paged_attn(bad, torch.full((n, hq, dd), float("nan"), dtype=dt, device="cuda"), ints([0, n]), ints([64 * 128]),
                       0.1, ws=other)
        out, lse = skv.paged_attn(cache, q, ints(qs), ints(kv), d ** -0.5, lse=True, ws=ws)
        check(f64(out), f64(lse), want, wlse, mass, dt, 24.0, 24.0, d ** -0.5, d, 500, "call %d" % i)
    assert cache.device_status() == 0


@pytest.mark.parametrize("hq,hkv", [(4, 1), (5, 1), (1, 1)])
def test_paged_token_counts_around_the_choice_of_form(hq, hkv):
    """One query tile per unit up to floor(128 / G) tokens a request, two above."""
    tq = 128 // (hq // hkv)
    for ql in ([tq, tq], [tq, tq + 1], [2 * tq, 1], [2 * tq + 1], [tq]):
        run_paged(skv, sum(ql), ql, [x + 37 for x in ql], 16, hq, hkv, 64, torch.float16, what=str(ql))


def test_rows_before_the_first_request():
    d, dt = 64, torch.bfloat16
    pg = Pages(2, [70, 9], 16, 1, d, dt)
    cache, q = pg.cache(skv), randn(1, (12, 2, d), dt)
    out = torch.full((12, 2, d), 5.0, dtype=dt, device="cuda")
    skv.paged_attn(cache, q, ints([4, 9, 10]), ints([70, 9]), 0.125, out=out)
    want, _, mass = PO.paged(f64(q[4:10]), f64(pg.k), f64(pg.v), pg.table, [0, 5, 6], [70, 9], 0.125)
    check(f64(out[4:10]), None, want, None, mass, dt, 20.0, 20.0, 0.125, d, 70)
    assert (out[:4] == 5).all() and (out[10:] == 5).all()


def test_pool_past_32_bit_offsets():
    """Pages whose elements and bytes lie past 2^32: writes and reads of the last ones."""
    hkv, page, d, dt = 8, 64, 128, torch.bfloat16
    n_page = 70000                                  # 4.6e9 elements a pool
    k = torch.empty((n_page, hkv, page, d), dtype=dt, device="cuda")
    v = torch.empty_like(k)
    table = ints([[n_page - 1, 3, n_page - 2], [35000, n_page - 70, -1]])
    cache = skv.PagedCache.wrap(k=k, v=v, block_table=table)
    kv, slots = [150, 100], []
    for b, n in enumerate(kv):
        slots += [int(table[b, t // page]) * page + t % page for t in range(n)]
    kn, vn = randn(1, (250, hkv, d), dt), randn(2, (250, hkv, d), dt)
    skv.kv_paged_write(cache, None, kn, vn, None, ints(slots))
    for t in (0, 149, 200):
        assert torch.equal(k[slots[t] // page, :, slots[t] % page], kn[t])
    q = randn(3, (2, 16, d), dt)
    out, lse = skv.paged_attn(cache, q, ints([0, 1, 2]), ints(kv), d ** -0.5, lse=True)
    assert cache.device_status() == 0
    o, l, mass = PO.cross(f64(q), f64(kn), f64(vn), [0, 1, 2], [0, 150], kv, d ** -0.5)
    check(f64(out), f64(lse), o, l, mass, dt, 20.0, 20.0, d ** -0.5, d, 150)


@pytest.mark.parametrize("n_q", [1, 100])
def test_units_that_take_milliseconds(n_q):
    """More units than SMs, each of 2,500 key tiles: the scheduler and a query
    tile's warps wait a whole unit long.  All values are 1, so is the output."""
    page, d, n, n_req, dt = 64, 64, 320000, 160, torch.bfloat16
    k = torch.zeros((2, 1, page, d), dtype=dt, device="cuda")
    cache = skv.PagedCache.wrap(k=k, v=torch.ones_like(k), block_table=torch.ones((n_req, n // page), dtype=torch.int32, device="cuda"))
    q = torch.zeros((n_req * n_q, 2, d), dtype=dt, device="cuda")
    out = skv.paged_attn(cache, q, ints(starts([n_q] * n_req)), ints([n] * n_req), 1.0)
    assert cache.device_status() == 0 and (out == 1).all()


@pytest.mark.parametrize("n_q", [1, 100])
def test_fp16_keys_far_below_the_largest(n_q):
    """One key of score 0 with value 0 among 65,536 of score -26 ln 2 with value
    1: together they are worth 2^-10 of it and must not vanish.  q = e_0 and
    k = 0 or -26 ln 2 e_0 (its fp16 rounding, scale 1): the score is exact, and
    its P is off by at most an absolute half step, 2^-25 of what 2^6 stands for.  (160 requests of the same pages:
    most are one CTA's work from the first key on.)"""
    page, d, n, n_req, dt = 64, 64, 65536 + 64, 160, torch.float16
    low = float(torch.tensor(26 * np.log(2)).to(dt))
    k = torch.zeros((2, 1, page, d), dtype=dt, device="cuda")
    k[:, :, :, 0] = -low
    k[0, 0, 0, 0] = 0.0
    v = torch.ones_like(k)
    v[0, 0, 0] = 0.0
    table = torch.ones((n_req, n // page), dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    cache = skv.PagedCache.wrap(k=k, v=v, block_table=table)
    q = torch.zeros((n_req * n_q, 2, d), dtype=dt, device="cuda")
    q[:, :, 0] = 1.0
    out = skv.paged_attn(cache, q, ints(starts([n_q] * n_req)), ints([n] * n_req), 1.0).view(n_req, n_q, 2, d)
    seen = n - n_q + torch.arange(1, n_q + 1, device="cuda").double()[:, None, None]
    p = np.exp(-low) * (seen - 1)
    want = p / (1 + p)
    tol = seen * 2.0 ** -31 + want * (2.0 ** -11 + 2.0 ** -20) + 2.0 ** -25
    assert cache.device_status() == 0
    assert ((out.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("over", [0, 1])
def test_longest_request(over):
    """Equal scores over the most keys that a request may hold (one page, over
    and over): the mean of the values; one key more is refused.  Sums of ones are
    exact.  A CTA's share is less than a page, so its value sums stay below 3
    times the largest running sum s of the page, and lose at most a step of
    that per 16 keys: n / 16 2^-23 3 s over all, beside the merge's 152."""
    page, d, dt = 2 ** 20, 64, torch.bfloat16
    k = torch.zeros((1, 1, page, d), dtype=dt, device="cuda")
    v = torch.randn((1, 1, page, d), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(dt)
    cache = skv.PagedCache.wrap(k=k, v=v, block_table=torch.zeros((1, 65), dtype=torch.int32, device="cuda"))
    q = randn(1, (1, 2, d), dt)
    n = skv.SKV_MAX_KEYS + over
    out, lse = skv.paged_attn(cache, q, ints([0, 1]), ints([n]), 0.125, lse=True)
    assert cache.device_status() == (skv.SKV_DEV_BAD_LEN if over else 0)
    if over:
        assert (out == 0).all() and torch.isneginf(lse).all()
        return
    want = v[0, 0].double().mean(0)
    s = v[0, 0].double().cumsum(0).abs().amax(0)
    tol = torch.finfo(dt).eps / 2 * want.abs() + 2.0 ** -27 * 4 * s
    assert ((out.double() - want).abs() <= tol).all()
    # log2 n = 26 times ln 2 in fp32: the constant is off by at most 2^-25 of
    # itself, log2's result by a step of 2^-23 of itself, and the product is
    # rounded by half a step of 18, 2^-20
    assert (lse.double() - np.log(n)).abs().max() <= 2.0 ** -20 + np.log(n) * (2.0 ** -25 + 2.0 ** -23)


def test_paged_results_repeat():
    a = run_paged(skv, 21, [1, 90, 1, 400], [5000, 1000, 33, 1400], 64, 8, 2, 128, torch.bfloat16)
    b = run_paged(skv, 21, [1, 90, 1, 400], [5000, 1000, 33, 1400], 64, 8, 2, 128, torch.bfloat16)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_paged_strided_queries_and_lse_left_out():
    d, dt = 128, torch.bfloat16
    kv, ql = [200, 77], [30, 1]
    pg = Pages(5, kv, 64, 2, d, dt)
    cache = pg.cache(skv)
    wide = randn(6, (31, 9, d), dt)
    q = wide[:, 3:7]
    out = skv.paged_attn(cache, q, ints(starts(ql)), ints(kv), 0.1)
    assert torch.equal(out, skv.paged_attn(cache, q.contiguous(), ints(starts(ql)), ints(kv), 0.1))
    want, _, mass = PO.paged(f64(q), f64(pg.k), f64(pg.v), pg.table, starts(ql), kv, 0.1)
    check(f64(out), None, want, None, mass, dt, 20.0, 20.0, 0.1, d, 200)


# --------------------------------------------------------------------- cross

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 4), (128, 8, 2), (64, 7, 1), (128, 5, 5)])
def test_cross(dtype, d, hq, hkv):
    dt = DT[dtype]
    kl, ql = [1, 127, 128, 129, 0, 700, 5, 300], [3, 130, 1, 64, 5, 300, 0, 1]
    k_start, at = [], 4
    for n in kl:      # gaps between the requests' states
        k_start.append(at)
        at += n + 3
    kv = randn(1, (at, 2 * hkv + 1, d), dt)
    used = torch.zeros(at, dtype=torch.bool)
    for s, n in zip(k_start, kl):
        used[s:s + n] = True
    kv[~used.cuda()] = float("nan")        # what no request reads may hold anything
    k, v = kv[:, :hkv], kv[:, hkv:2 * hkv]
    qs = starts(ql)
    q = randn(2, (int(qs[-1]), hq, d), dt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = skv.cross_attn(q, k, v, ints(qs), ints(k_start), ints(kl), d ** -0.5, status=status, lse=True)
    assert status.item() == 0
    clean = torch.where(torch.isnan(kv), 0.0, kv.float())
    want, wlse, mass = PO.cross(f64(q), f64(clean[:, :hkv]), f64(clean[:, hkv:2 * hkv]), qs, k_start, kl, d ** -0.5)
    check(f64(out), f64(lse), want, wlse, mass, dt, 20.0, 20.0, d ** -0.5, d, 700)
    assert (out[int(qs[4]):int(qs[5])] == 0).all()


def test_cross_shared_and_padded_states():
    d, dt = 128, torch.bfloat16
    k, v = randn(1, (4 * 300, 2, d), dt), randn(2, (4 * 300, 2, d), dt)
    q = randn(3, (64, 4, d), dt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for ks, kl in (([0, 300, 600, 900], [300, 17, 256, 1]), ([100, 100, 0, 50], [500, 500, 1200, 7])):
        out, lse = skv.cross_attn(q, k, v, ints([0, 16, 32, 48, 64]), ints(ks), ints(kl), 0.09, status=status, lse=True)
        want, wlse, mass = PO.cross(f64(q), f64(k), f64(v), [0, 16, 32, 48, 64], ks, kl, 0.09)
        check(f64(out), f64(lse), want, wlse, mass, dt, 20.0, 20.0, 0.09, d, 1200)
    assert status.item() == 0


def test_cross_ranges_out_of_bounds_and_no_states():
    d, dt = 64, torch.bfloat16
    q = randn(3, (4, 2, d), dt)
    for n_key, ks, kl, bit in ((50, [-1, 0], [5, 50], 32), (50, [49, 0], [2, 50], 32), (50, [2 ** 31 - 1, 0], [2 ** 31 - 1, 50], 32),
                               (50, [0, 0], [-3, 50], 32), (0, [0, 0], [0, 0], 0)):
        k = randn(1, (n_key, 1, d), dt)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = skv.cross_attn(q, k, k, ints([0, 2, 4]), ints(ks), ints(kl), 0.125, status=status, lse=True)
        assert status.item() == bit
        assert (out[:2] == 0).all() and torch.isneginf(lse[:, :2]).all()
        assert torch.isfinite(lse[:, 2:]).all() == (n_key > 0)


# ------------------------------------------------------------ used together

def _serve(dtype, n_layer, steps, graph=False):
    """A small server: requests come, grow by chunks and single tokens, finish
    and give their rows to new ones; every step is plan, then per layer write
    and attend, against a dense fp64 history of each request."""
    dt, hq, hkv, d, page, n_req = DT[dtype], 6, 2, 64, 16, 5
    theta, scale = 1e4, 64 ** -0.5
    cache = skv.PagedCache(60, page, hkv, d, n_req, 12, theta=theta, dtype=dt, n_layer=n_layer)
    layers, ws = [cache.layer(i) for i in range(n_layer)], skv.attn_workspace()
    hist = [[(np.zeros((0, hkv, d)), np.zeros((0, hkv, d))) for _ in range(n_req)] for _ in range(n_layer)]
    rng = np.random.default_rng(4)
    n_tok = 96
    new_len, plan = ints([0] * n_req), skv.PagedPlan.empty(n_req, n_tok)
    qkv = [torch.zeros((n_tok, hq + 2 * hkv, d), dtype=dt, device="cuda") for _ in range(n_layer)]
    outs = [torch.zeros((n_tok, hq, d), dtype=dt, device="cuda") for _ in range(n_layer)]
    rot = torch.zeros((n_tok, hq, d), dtype=dt, device="cuda")

    def step():
        skv.kv_paged_plan(cache, new_len, n_tok, plan=plan)
        for x, c, o in zip(qkv, layers, outs):
            skv.kv_paged_write(c, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], plan.position, plan.slot, q_out=rot)
            skv.paged_attn(c, rot, plan.q_start, plan.kv_len, scale, out=o, ws=ws)
        cache.advance(plan)

    captured = None
    if graph:
        step()                       # of nothing: every length is 0
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
    held = [0] * n_req
    u = torch.finfo(dt).eps / 2
    for i in range(steps):
        lens = [int(rng.choice([-1, 0, 1, 1, 1, 9, 30])) if h else int(rng.integers(1, 40)) for h in held]
        lens = [x if x < 0 or h + x <= 12 * page else -1 for x, h in zip(lens, held)]
        while sum(max(0, x) for x in lens) > n_tok:
            lens[int(np.argmax(lens))] = 0
        new_len.copy_(ints(lens))
        for l in range(n_layer):
            qkv[l].copy_(randn(100 * i + l, (n_tok, hq + 2 * hkv, d), dt))
        captured.replay() if graph else step()
        assert cache.device_status() == 0
        at = 0
        for b, w in enumerate(lens):
            if w < 0:
                held[b] = 0
                for l in range(n_layer):
                    hist[l][b] = (np.zeros((0, hkv, d)), np.zeros((0, hkv, d)))
                continue
            for l in range(n_layer):
                x = f64(qkv[l][at:at + w])
                pos = np.arange(held[b], held[b] + w)
                kr, vr = PO.rotate(x[:, hq:hq + hkv], pos, theta), x[:, hq + hkv:]
                k, v = (np.concatenate(p) for p in zip(hist[l][b], (kr, vr)))
                hist[l][b] = (k, v)
                if w == 0:
                    continue
                q = PO.rotate(x[:, :hq], pos, theta)
                want, _, mass = PO.attend(q, k, v, held[b], scale)
                got = f64(outs[l][at:at + w])
                # as paged_harness.check, and the rotated q and k are rounded once
                # each: a score moves by at most 2 u |q| |k| scale
                e = 2 * u * np.linalg.norm(q, axis=-1).max() * np.linalg.norm(k, axis=-1).max() * scale + 1e-4
                tol = u * (np.abs(want) * (1 + u) + mass) + (np.exp(2 * e) - 1) * mass + 1e-6
                assert (np.abs(got - want) <= tol).all(), (i, l, b)
            held[b] += w
            at += w
        assert cache.state[:n_req].tolist() == held
        assert int(cache.state[-1]) == 60 - sum(-(-h // page) for h in held)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_serving_steps(dtype):
    _serve(dtype, 2, 25)


def test_serving_steps_from_a_graph():
    _serve("bf16", 2, 15, graph=True)


@pytest.mark.parametrize("ql", [[1, 1, 1], [1, 150, 60]])
def test_attention_in_place_of_its_queries(ql):
    d, dt, kv = 128, torch.bfloat16, [9000, 400, 61]
    pg = Pages(8, kv, 16, 2, d, dt)
    cache = pg.cache(skv)
    q = randn(9, (sum(ql), 12, d), dt)
    args = (ints(starts(ql)), ints(kv), 0.09)
    want = skv.paged_attn(cache, q, *args)
    for _ in range(5):
        got = q.clone()
        assert skv.paged_attn(cache, got, *args, out=got) is got
        assert torch.equal(got, want)


def test_requests_that_share_pages():
    """Two requests over the same first pages, each with a page of its own
    after them, and a third that is the first one's prefix."""
    d, dt, page = 64, torch.float16, 32
    pg = Pages(8, [300, 310, 40], page, 2, d, dt)
    pg.table[1, :8] = pg.table[0, :8]
    pg.table[2, :2] = pg.table[0, :2]
    cache, ql, kv = pg.cache(skv), [3, 1, 40], [300, 310, 40]
    q = randn(9, (44, 6, d), dt)
    out, lse = skv.paged_attn(cache, q, ints(starts(ql)), ints(kv), 0.1, lse=True)
    want, wlse, mass = PO.paged(f64(q), f64(pg.k), f64(pg.v), pg.table, starts(ql), kv, 0.1)
    check(f64(out), f64(lse), want, wlse, mass, dt, 14.0, 14.0, 0.1, d, 310)


def test_captured_on_a_forked_stream():
    """In one graph: a plan and a write on the captured stream, attention of two
    caches on streams that fork from it after a copy and join again."""
    d, dt, page, n_req = 64, torch.bfloat16, 16, 3
    caches = [skv.PagedCache(40, page, 2, d, n_req, 8, theta=1e4) for _ in range(2)]
    x, new_len = randn(1, (3 * 20, 8, d), dt), ints([20, 20, 20])
    q, plans, outs, spaces = torch.empty((60, 4, d), dtype=dt, device="cuda"), [], [], []
    for _ in range(2):
        plans.append(skv.PagedPlan.empty(n_req, 60))
        outs.append(torch.zeros((60, 4, d), dtype=dt, device="cuda"))
        spaces.append(skv.attn_workspace())
    rot = [torch.empty_like(q) for _ in range(2)]
    side = torch.cuda.Stream()

    def one(i):
        c, p = caches[i], plans[i]
        skv.kv_paged_write(c, q, x[:, 4:6], x[:, 6:], p.position, p.slot, q_out=rot[i])
        skv.paged_attn(c, rot[i], p.q_start, p.kv_len, 0.125, out=outs[i], ws=spaces[i])

    def both():
        for c, p in zip(caches, plans):
            skv.kv_paged_plan(c, new_len, 60, plan=p)
        q.copy_(x[:, :4])
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            one(1)
        one(0)
        main.wait_stream(side)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed in (5, 6):
        x.copy_(randn(seed, x.shape, dt))
        both()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        assert torch.equal(*want) and want[0].abs().sum() > 0
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[0])
    assert all(c.device_status() == 0 for c in caches)


def test_two_streams_with_their_own_workspaces():
    d, dt = 128, torch.bfloat16
    kv, ql = [4000, 900, 128], [1, 40, 1]
    pg = Pages(5, kv, 64, 2, d, dt)
    cache = pg.cache(skv)
    q = randn(6, (42, 8, d), dt)
    args = (ints(starts(ql)), ints(kv), 0.1)
    want = skv.paged_attn(cache, q, *args)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    spaces = [skv.attn_workspace() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        with torch.cuda.stream(streams[i % 2]):
            got.append(skv.paged_attn(cache, q, *args, ws=spaces[i % 2]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)
    assert cache.device_status() == 0


def test_binding_refusals():
    d, dt = 64, torch.bfloat16
    pg = Pages(1, [20, 30], 16, 2, d, dt, fill=0.0)
    cache = pg.cache(skv)
    q = randn(1, (2, 4, d), dt)
    qs, kv = ints([0, 1, 2]), ints([20, 30])
    bad = [lambda: skv.paged_attn(cache, q.half(), qs, kv, 1.0), lambda: skv.paged_attn(cache, q[..., :32], qs, kv, 1.0),
           lambda: skv.paged_attn(cache, q.transpose(0, 1), qs, kv, 1.0), lambda: skv.paged_attn(cache, q, qs[:2], kv, 1.0),
           lambda: skv.paged_attn(cache, q, qs, kv.long(), 1.0), lambda: skv.paged_attn(cache, q, qs, kv, 0.0),
           lambda: skv.paged_attn(cache, q[:, :3], qs, kv, 1.0),
           lambda: skv.paged_attn(cache, q, qs, kv, 1.0, out=q[:1]), lambda: skv.paged_attn(cache, q, qs, kv, 1.0, ws=torch.zeros(1, device="cuda")),
           lambda: skv.kv_paged_plan(cache, kv, 2), lambda: skv.kv_paged_write(cache, q, q, q, None, qs[:2]),
           lambda: skv.kv_paged_write(cache, None, q[:, :2], q[:1, :2], None, qs[:2]),
           lambda: skv.PagedCache.wrap(k=pg.k.float(), v=pg.v.float(), block_table=cache.block_table),
           lambda: skv.PagedCache.wrap(k=pg.k, v=pg.v[:1], block_table=cache.block_table),
           lambda: skv.cross_attn(q, q[:, :2], q[:1, :2], qs, kv, kv, 1.0, status=cache.status)]
    for i, f in enumerate(bad):
        with pytest.raises((TypeError, ValueError, skv.SkvError)):
            f()
            print("not refused:", i)
