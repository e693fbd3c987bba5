"""kv_evict_plan and kv_evict_move on the GPU against the oracle, and eviction
as it is used: steps of an evicting cache over several layers."""
import numpy as np
import pytest
import torch

from evict_harness import lay, moves_of, tables
from oracle import evict_oracle as EO
from paged_harness import DT, ints, randn
from streaming_kv_cache_gb300 import skv

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def _scores(rng, kind, shape):
    if kind == "ties":
        return rng.integers(0, 3, shape).astype(np.float32)
    if kind == "odd":
        x = rng.choice(np.array([0.0, -0.0, 1.0, -1.0, np.nan, -np.nan, np.inf, -np.inf, 1e-45, 3e38], dtype=np.float32), shape)
        return x
    if kind == "equal":
        return np.full(shape, 0.25, dtype=np.float32)
    x = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    x[rng.random(shape) < 0.05] = 0
    return x


def _plan(seed, held, keep, page, hkv, n_layer, sink, recent, kind, evicted=True, d=64, dtype="bf16", cols=2):
    """kv_evict_plan and kv_evict_move against the oracle."""
    rng = np.random.default_rng(seed)
    used = [-(-m // page) for m in held]
    n_page, n_req = sum(used) + 2, len(held)
    cols = max(used + [1]) + cols
    table = tables(rng, used, n_page, cols)
    gone = rng.integers(0, 1000, n_req) if evicted else np.zeros(n_req, dtype=int)
    score = [[_scores(rng, kind, (hkv, m)) for m in held] for _ in range(n_layer)]
    pos = [[np.stack([rng.permutation(m) + gone[b] * (rng.random() < 0.8) for _ in range(hkv)]) if m else np.zeros((hkv, 0), int)
            for b, m in enumerate(held)] for _ in range(n_layer)]
    sp, pp = lay(score, table, page, n_page, -7.0, np.float32), lay(pos, table, page, n_page, -8, np.int32)
    shape = sp.shape
    k, v = (randn(seed + i, shape + (d,), DT[dtype]) for i in (1, 2))
    state = ints(list(held) + [0, 0] + (gone.tolist() if evicted else []))
    cache = skv.PagedCache.wrap(k=k, v=v, block_table=ints(table.tolist()), state=state)
    scores = skv.PagedScores(torch.from_numpy(sp).cuda(), torch.from_numpy(pp).cuda(), torch.full(shape, -5, **I32),
                             torch.full((n_layer, n_req, hkv), -6, **I32))
    for _ in range(2):
        skv.kv_evict_plan(cache, scores, ints(list(held)), ints(list(keep)), sink, recent)
    assert cache.device_status() == 0
    move, n_move = scores.move.cpu().numpy(), scores.n_move.cpu().numpy()
    want_move = np.full(shape, -5, dtype=np.int32)
    bits = lambda t: t.view(torch.int16 if t.element_size() == 2 else torch.int32).cpu().numpy()  # noqa: E731
    pools = [bits(t) for t in (k, v, scores.score, scores.pos)]
    for l in range(n_layer):
        for b, m in enumerate(held):
            for h in range(hkv):
                want = EO.select(score[l][b][h], pos[l][b][h], keep[b], int(gone[b]) + m, sink, recent)
                assert moves_of(move, n_move, table, page, l, b, h) == want, (l, b, h)
                for i, pair in enumerate(want):
                    for x in (0, 1):
                        want_move[l, table[b, (2 * i + x) // page], h, (2 * i + x) % page] = pair[x]
                    to, src = ((l, table[b, j // page], h, j % page) for j in pair)
                    for pool in pools:
                        pool[to] = pool[src]
    assert np.array_equal(move, want_move)
    for _ in range(2):
        skv.kv_evict_move(cache, scores, ints(list(held)))
    assert cache.device_status() == 0
    for got, want in zip((k, v, scores.score, scores.pos), pools):
        assert np.array_equal(bits(got), want)
    assert np.array_equal(scores.move.cpu().numpy(), want_move)
    return cache, scores


@pytest.mark.parametrize("kind", ["weights", "ties", "odd", "equal"])
@pytest.mark.parametrize("held,keep,page,hkv,n_layer,sink,recent", [
    ([1], [1], 16, 1, 1, 0, 0), ([2], [1], 16, 1, 1, 0, 0), ([5, 40, 0, 17], [4, 20, 3, 17], 16, 2, 3, 2, 3), ([100], [0], 48, 3, 1, 4, 4),
    ([2049, 2049], [2048, 2048], 64, 2, 2, 4, 256), ([300, 299], [150, 298], 16, 1, 2, 0, 150), ([700], [350], 272, 2, 1, 300, 300),
    ([4097, 9000], [1000, 8999], 64, 1, 1, 4, 64), ([513, 512, 511], [1, 511, 256], 16, 1, 1, 0, 1)])
def test_evict(kind, held, keep, page, hkv, n_layer, sink, recent):
    _plan(len(held) + held[0], held, keep, page, hkv, n_layer, sink, recent, kind)


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (64, "fp16"), (128, "bf16"), (128, "fp16")])
def test_evict_types(d, dtype):
    _plan(5, [333, 150, 1000], [100, 149, 600], 16, 2, 2, 3, 20, "weights", d=d, dtype=dtype)


@pytest.mark.parametrize("held,keep", [([40000], [20000]), ([70001], [70000]), ([150000], [1000]), ([33000, 100], [32999, 50])])
def test_evict_long(held, keep):
    for kind in ("weights", "ties"):
        _plan(1, held, keep, 128, 1, 1, 4, 100, kind)


@pytest.mark.parametrize("held,keep", [([300, 9000, 20000], [299, 4000, 19999]), ([5], [2]), ([16385, 40], [1, 39])])
def test_evict_of_short_requests_in_long_table_rows(held, keep):
    """Rows that hold 144,000 tokens: CTAs of a cluster that a request does not
    need leave before the others meet."""
    _plan(6, held, keep, 16, 2, 1, 2, 30, "weights", cols=9000)


def test_evict_layer_by_layer():
    """One layer's cache and scores give what all layers at once give."""
    whole, ws = _plan(21, [333, 150], [100, 149], 16, 2, 3, 3, 20, "ties")
    again, s2 = _plan(21, [333, 150], [100, 149], 16, 2, 3, 3, 20, "ties")
    kv, keep = ints([333, 150]), ints([60, 140])
    skv.kv_evict_plan(whole, ws, kv, keep, 3, 20)
    skv.kv_evict_move(whole, ws, kv)
    for l in (-1, 0, 1):
        skv.kv_evict_plan(again.layer(l), s2.layer(l), kv, keep, 3, 20)
        skv.kv_evict_move(again.layer(l), s2.layer(l), kv)
    for x, y in ((whole._k, again._k), (whole._v, again._v), (ws.score, s2.score), (ws.pos, s2.pos), (ws.move, s2.move), (ws.n_move, s2.n_move)):
        assert torch.equal(x, y)


def test_evict_without_evicted_words():
    _plan(2, [90, 33], [40, 32], 16, 2, 1, 2, 5, "weights", evicted=False)


def test_evict_of_many_requests():
    rng = np.random.default_rng(0)
    held = rng.integers(0, 60, 700).tolist()
    _plan(3, held, [max(0, x - int(y)) for x, y in zip(held, rng.integers(0, 9, 700))], 16, 1, 2, 1, 4, "weights")


def test_values_out_of_range():
    """Positions of 100 are none of the request's, so nothing is protected.  In
    the last two cases a page of request 1 is outside the pool: its tokens come
    last, so that of 20 the ten kept are 3 to 12, and the four kept 16 to 19."""
    page, hkv, n_page = 16, 1, 4
    shape = (1, n_page, hkv, page)
    for table, held, keep, gone, status, n in (
            ([[0, 1], [2, 3]], [33, 20], [5, 20], [0, 0], skv.SKV_DEV_BAD_LEN, [0, 0]), ([[0, 1], [2, 3]], [-2, 20], [5, 19], [0, 0], skv.SKV_DEV_BAD_LEN, [0, 1]),
            ([[0, 1], [2, 3]], [20, 20], [-1, 19], [0, 0], skv.SKV_DEV_BAD_LEN, [0, 1]), ([[0, 1], [2, 3]], [20, 20], [20, 19], [0, -4], skv.SKV_DEV_BAD_LEN, [0, 1]),
            ([[0, 1], [2, 9]], [20, 20], [20, 10], [0, 0], skv.SKV_DEV_BAD_PAGE, [0, 3]), ([[0, 1], [-1, 3]], [20, 20], [20, 4], [0, 0], skv.SKV_DEV_BAD_PAGE, [0, 4])):
        k = torch.zeros(shape + (64,), dtype=torch.bfloat16, device="cuda")
        cache = skv.PagedCache.wrap(k=k, v=k.clone(), block_table=ints(table), state=ints(held + [0, 0] + gone))
        score = torch.ones(shape, device="cuda")
        score[0, table[1][0], 0, :3] = 0 if table[1][0] >= 0 else 1
        scores = skv.PagedScores(score, torch.full(shape, 100, **I32), torch.zeros(shape, **I32), torch.full((1, 2, 1), -1, **I32))
        skv.kv_evict_plan(cache, scores, ints(held), ints(keep))
        assert cache.device_status() == status
        assert scores.n_move[0, :, 0].tolist() == n
        cache.status.zero_()
        skv.kv_evict_move(cache, scores, ints(held))
        torch.cuda.synchronize()


def test_moves_out_of_range_are_left_out():
    shape = (1, 4, 1, 16)
    k = randn(0, shape + (64,), torch.bfloat16)
    before = k.clone()
    cache = skv.PagedCache.wrap(k=k, v=k.clone(), block_table=ints([[0, 7], [2, 3]]))
    scores = skv.PagedScores(torch.zeros(shape, device="cuda"), torch.zeros(shape, **I32), torch.zeros(shape, **I32), torch.zeros((1, 2, 1), **I32))
    move = lambda page, *pairs: scores.move.view(4, 16)[page, :2 * len(pairs)].copy_(ints([x for p in pairs for x in p]))  # noqa: E731
    for n, status in ((-1, skv.SKV_DEV_BAD_LEN), (11, skv.SKV_DEV_BAD_LEN), (2 ** 31 - 1, skv.SKV_DEV_BAD_LEN)):
        scores.n_move.fill_(n)
        skv.kv_evict_move(cache, scores, ints([20, 20]))
        assert cache.device_status() == status and torch.equal(k, before)
        cache.status.zero_()
    scores.n_move.copy_(ints([0, 3]).view(1, 2, 1))
    move(2, (3, 20), (-1, 19), (2, 18))
    skv.kv_evict_move(cache, scores, ints([20, 20]))
    assert cache.device_status() == skv.SKV_DEV_BAD_LEN
    want = before.clone()
    want[0, 2, 0, 2] = want[0, 3, 0, 2]
    assert torch.equal(k, want)
    cache.status.zero_()
    scores.n_move.copy_(ints([1, 0]).view(1, 2, 1))
    move(0, (2, 18))
    skv.kv_evict_move(cache, scores, ints([20, 20]))
    assert cache.device_status() == skv.SKV_DEV_BAD_PAGE and torch.equal(k, want)


def test_pools_past_32_bit_offsets():
    """Layers whose keys lie beyond 2^31 elements, places beyond 2^31 bytes."""
    n_page, page, hkv, d, n_layer = 20000, 64, 4, 128, 4         # 655 M elements a layer
    shape = (n_layer, n_page, hkv, page)
    k, v = (torch.zeros(shape + (d,), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = ints([[n_page - 1, n_page - 2, 0]])
    cache = skv.PagedCache.wrap(k=k, v=v, block_table=table)
    scores = skv.PagedScores(torch.zeros(shape, device="cuda"), torch.full(shape, 100, **I32), torch.zeros(shape, **I32),
                             torch.zeros((n_layer, 1, hkv), **I32))
    scores.score[:, n_page - 1] = torch.arange(64.0, device="cuda") + 1
    scores.score[:, n_page - 2] = 500
    k[:, n_page - 2] = torch.arange(64, device="cuda", dtype=torch.bfloat16)[:, None] + 3
    skv.kv_evict_plan(cache, scores, ints([130]), ints([64]))
    skv.kv_evict_move(cache, scores, ints([130]))
    assert cache.device_status() == 0 and (scores.n_move == 64).all()
    assert torch.equal(k[:, n_page - 1], k[:, n_page - 2]) and (k[:, 1:n_page - 2] == 0).all()


def test_graph_replay_and_two_calls_at_once():
    cache, scores = _plan(8, [900, 300], [500, 299], 16, 2, 2, 4, 40, "weights")
    other, oscores = _plan(9, [800, 350], [300, 349], 16, 2, 2, 4, 40, "weights")
    sides, graphs, wants = [torch.cuda.Stream() for _ in range(2)], [], []
    for (c, s, held, keep), side in zip(((cache, scores, [900, 300], [500, 299]), (other, oscores, [800, 350], [300, 349])), sides):
        kv, kp = ints(held), ints(keep)
        skv.kv_evict_plan(c, s, kv, kp, 4, 40)
        wants.append((s.move.clone(), s.n_move.clone()))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            skv.kv_evict_plan(c, s, kv, kp, 4, 40)
        graphs.append((g, kv, kp, s))
    for _ in range(3):
        for (g, *_, s), side in zip(graphs, sides):
            with torch.cuda.stream(side):
                s.n_move.fill_(-1)
                g.replay()
    torch.cuda.synchronize()
    for (_, _, _, s), (move, n) in zip(graphs, wants):
        assert torch.equal(s.n_move, n) and torch.equal(s.move, move)


def test_binding_refusals():
    cache = skv.PagedCache(8, 16, 2, 64, 2, 4, n_layer=2, evicts=True)
    scores = skv.PagedScores.empty(cache)
    kv, keep = ints([1, 1]), ints([1, 1])
    skv.kv_evict_plan(cache, scores, kv, keep)
    skv.kv_evict_move(cache, scores, kv)
    for bad in (dict(scores=scores.layer(0)), dict(kv_len=ints([1])), dict(keep=ints([1, 1]).float()),
                dict(scores=skv.PagedScores(scores.score, scores.pos)),
                dict(scores=skv.PagedScores(scores.score, scores.pos, scores.move, torch.zeros((2, 3, 2), **I32)))):
        with pytest.raises((ValueError, TypeError)):
            skv.kv_evict_plan(**{**dict(cache=cache, scores=scores, kv_len=kv, keep=keep), **bad})
    for n_sink, n_recent in ((-1, 0), (0, -1)):
        with pytest.raises(skv.SkvError):
            skv.kv_evict_plan(cache, scores, kv, keep, n_sink, n_recent)
    with pytest.raises(skv.SkvError):      # the keys over the values
        skv.kv_evict_move(skv.PagedCache.wrap(k=cache._k, v=cache._k, block_table=cache.block_table), scores, kv)
    for make in (lambda: skv.PagedScores(scores.score, scores.pos, scores.move), lambda: skv.PagedScores(scores.score, scores.pos[:1]),
                 lambda: skv.PagedScores(scores.score.double(), scores.pos), lambda: skv.PagedScores(scores.score[0, 0], scores.pos[0, 0])):
        with pytest.raises((ValueError, TypeError)):
            make()


# ------------------------------------------------------------ as it is used

class _Model:
    """What an evicting cache should hold, in 64 bits: per layer, request and
    kv head a list of tokens (key rotated at its position, value, score, pos)."""

    def __init__(self, n_layer, n_req, hkv):
        self.t = [[[[] for _ in range(hkv)] for _ in range(n_req)] for _ in range(n_layer)]
        self.next = [0] * n_req


@pytest.mark.parametrize("dtype,d,hq,hkv,page", [("bf16", 64, 4, 2, 16), ("fp16", 128, 6, 2, 32)])
def test_steps_of_an_evicting_cache(dtype, d, hq, hkv, page):
    """Prompts, decode steps and drafted blocks over a budget: plan, write,
    attend, weigh, verify, trim, evict, trim.  The cache's tokens are found by
    their positions; attention over them is what the model's lists give."""
    dt, rng = DT[dtype], np.random.default_rng(3)
    n_layer, n_req, n_page, cols, budget, sink, recent, vocab = 2, 3, 24, 6, 40, 2, 8, 50
    cache = skv.PagedCache(n_page, page, hkv, d, n_req, cols, theta=1e4, dtype=dt, n_layer=n_layer, evicts=True, rope_len=600)
    scores, ws, model = skv.PagedScores.empty(cache), skv.attn_workspace(), _Model(n_layer, n_req, hkv)
    scores.score.fill_(float("nan"))
    scale, grp = d ** -0.5, hq // hkv
    held = [0] * n_req
    n_evict = n_reject = 0
    for step in range(30):
        new = [50, 3, 0] if step == 0 else [int(x) for x in rng.integers(0, 7, n_req)]
        if step == 15:
            new[0] = -1                       # ends; the next step starts a new one in its slot
        span = [max(0, x) for x in new]
        n_tok = sum(span) + 2
        plan = skv.kv_paged_plan(cache, ints(new), n_tok)
        st = plan.q_start.tolist()
        if step == 15:
            held[0] = 0
            for l in range(n_layer):
                model.t[l][0] = [[] for _ in range(hkv)]
        nxt = [model.next[b] if held[b] else 0 for b in range(n_req)]
        for b in range(n_req):
            assert plan.position[st[b]:st[b + 1]].tolist() == list(range(nxt[b], nxt[b] + span[b]))
        for l in range(n_layer):
            qkv = randn(1000 * step + l, (n_tok, hq + 2 * hkv, d), dt)
            lay_c, lay_s = cache.layer(l), scores.layer(l)
            q = skv.kv_paged_write(lay_c, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], plan.position, plan.slot)
            out, lse = skv.paged_attn(lay_c, q, plan.q_start, plan.kv_len, scale, lse=True, ws=ws)
            skv.paged_attn_weight(lay_c, lay_s, q, plan.q_start, plan.kv_len, lse, plan.position, scale, ws=ws)
            qd, vd = q.double().cpu().numpy(), qkv[:, hq + hkv:].double().cpu().numpy()
            kd = lay_c.k.double().cpu().numpy()
            slot = plan.slot.tolist()
            for b in range(n_req):
                for h in range(hkv):
                    t = model.t[l][b][h]
                    for i in range(span[b]):
                        row = st[b] + i
                        t.append([kd[slot[row] // page, h, slot[row] % page], vd[row, h], 0.0, nxt[b] + i])
                        keys, vals = np.stack([x[0] for x in t]), np.stack([x[1] for x in t])
                        for g in range(grp):
                            z = keys @ qd[row, h * grp + g] * scale
                            p = np.exp(z - z.max())
                            p /= p.sum()
                            want = p @ vals
                            # the output's rounding and the probabilities' (see paged_harness.check), with room for the scores' error
                            tol = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
                            got = out[row, h * grp + g].double().cpu().numpy()
                            assert (np.abs(got - want) <= tol * (np.abs(want) + 1.01 * (p @ np.abs(vals))) + 1e-5).all()
                            for x, w in zip(t, p):
                                x[2] += w
        cache.advance(plan)
        held = [held[b] + span[b] for b in range(n_req)]
        # the drafts of this step's blocks, accepted or not
        prob = torch.softmax(torch.from_numpy(rng.standard_normal((n_tok, vocab))).float(), -1).cuda()
        token = ints(rng.integers(0, vocab, n_tok).tolist())
        u = torch.from_numpy(rng.random(n_tok)).float().cuda() * (0.02 if step else 0.0)
        acc, _, stay = skv.verify_sampled(prob, token, plan.q_start, u, torch.rand(n_req, device="cuda"), kv_len=plan.kv_len,
                                          status=cache.status)
        stay = [s if span[b] else held[b] for b, s in enumerate(stay.tolist())]
        assert stay == [held[b] - (span[b] - 1 - a if span[b] else 0) for b, a in enumerate(acc.tolist())]
        n_reject += sum(h - s for h, s in zip(held, stay))
        cache.advance(skv.kv_paged_trim(cache, ints(stay)))
        held = stay
        model.next = [n + s - r for n, s, r in zip(nxt, span, [span[b] - 1 - a if span[b] else 0 for b, a in enumerate(acc.tolist())])]
        for l in range(n_layer):
            for b in range(n_req):
                for h in range(hkv):
                    del model.t[l][b][h][held[b]:]
        # the budget
        kv, keep = ints(held), ints([budget] * n_req)
        skv.kv_evict_plan(cache, scores, kv, keep, sink, recent)
        skv.kv_evict_move(cache, scores, kv)
        cache.advance(skv.kv_paged_trim(cache, keep, evict=True))
        for b in range(n_req):
            if held[b] <= budget:
                continue
            n_evict += held[b] - budget
            for l in range(n_layer):
                for h in range(hkv):
                    t = model.t[l][b][h]
                    moves = EO.select([x[2] for x in t], [x[3] for x in t], budget, model.next[b], sink, recent)
                    for to, src in moves:
                        t[to] = t[src]
                    del t[budget:]
            held[b] = budget
        assert cache.device_status() == 0
        state = cache.state.tolist()
        assert state[:n_req] == held
        assert all(held[b] + state[n_req + 2 + b] == model.next[b] for b in range(n_req) if held[b])
        # places, positions and scores of every token
        table = cache.block_table.tolist()
        pos, score = scores.pos.tolist(), scores.score.tolist()
        for l in range(n_layer):
            for b in range(n_req):
                for h in range(hkv):
                    t = model.t[l][b][h]
                    at = [(table[b][j // page], j % page) for j in range(held[b])]
                    assert [pos[l][p][h][r] for p, r in at] == [x[3] for x in t], (step, l, b, h)
                    np.testing.assert_allclose([score[l][p][h][r] for p, r in at], [x[2] for x in t], rtol=1e-4, atol=1e-6)
        used = sum(-(-x // page) for x in held)
        assert state[n_req + 1] == n_page - used
    assert n_evict > 30 and n_reject > 20   # the steps do evict and reject
