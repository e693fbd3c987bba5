"""paged_attn_weight on the GPU against the fp64 oracle, within the bound that
evict_harness.check_weights derives."""
import numpy as np
import pytest
import torch

from evict_harness import check_weights
from paged_harness import DT, Pages, f64, ints, randn, starts
from streaming_kv_cache_gb300 import skv

pytestmark = pytest.mark.gpu


def _run(seed, q_len, kv_len, page, hq, hkv, d, dtype, add="own", scale=None, q=None, lse=None, wait_ns=0, ws=None):
    dt, scale = DT[dtype], d ** -0.5 if scale is None else scale
    pg = Pages(seed, kv_len, page, hkv, d, dt)
    cache = pg.cache(skv, wait_ns=wait_ns)
    st = starts(q_len)
    n = int(st[-1])
    q = randn(seed + 1, (n, hq, d), dt) if q is None else q
    ws = skv.attn_workspace() if ws is None else ws
    if lse is None:
        _, lse = skv.paged_attn(cache, q, ints(st), ints(kv_len), scale, lse=True, ws=ws)
        for b, m in enumerate(kv_len):      # a row without keys has lse -inf
            assert m or torch.isneginf(lse[:, st[b]:st[b + 1]]).all()
    g = torch.Generator().manual_seed(seed + 2)
    shape = (pg.n_page, hkv, page)
    # what lies at the step's own tokens and past the lengths is not to be added to
    old = torch.full(shape, float("nan"))
    for b, m in enumerate(kv_len):
        for j in range(m - q_len[b]):
            old[pg.table[b, j // page], :, j % page] = torch.rand(hkv, generator=g) * 10
    score, pos = torch.full(shape, -3.0, device="cuda"), torch.full(shape, -9, dtype=torch.int32, device="cuda")
    if add == "own":
        score = old.clone().cuda()
    before = f64(score)
    position = torch.randint(0, 1 << 30, (n,), generator=g, dtype=torch.int32).cuda()
    scores = skv.PagedScores(score, pos)
    skv.paged_attn_weight(cache, scores, q, ints(st), ints(kv_len), lse, position, scale,
                          add=True if add == "own" else old.cuda() if add == "other" else False, ws=ws)
    assert cache.device_status() == 0
    w = check_weights(score, pg, q, st, kv_len, lse, scale, None if add == "none" else f64(old), before)
    want = np.full(shape, -9)
    for b, m in enumerate(kv_len):
        if m == 0:
            continue
        for i in range(q_len[b]):
            j = m - q_len[b] + i
            want[pg.table[b, j // page], :, j % page] = int(position[st[b] + i])
    assert np.array_equal(pos.cpu().numpy(), want)
    return w, score, (cache, scores, q, ints(st), ints(kv_len), lse, position, scale)


CASES = [
    ([1], [1], 16, 1, 1, 64), ([1], [1], 64, 32, 8, 128), ([1], [3136], 64, 8, 2, 128), ([1] * 5, [1, 40, 128, 129, 1000], 16, 8, 2, 64),
    ([3, 0, 17, 130], [3, 50, 400, 300], 48, 14, 2, 64), ([200], [200], 64, 4, 4, 128), ([1, 2, 3], [500, 127, 257], 272, 6, 3, 128),
    ([5, 40], [5, 140], 32, 128, 1, 64), ([1, 1], [300, 255], 128, 128, 1, 128), ([60, 1, 33], [60, 700, 161], 16, 10, 2, 128),
    ([0, 0], [70, 5], 16, 2, 1, 64), ([300], [900], 96, 3, 1, 64), ([4, 1], [0, 9], 16, 2, 2, 64), ([128, 129], [128, 385], 128, 2, 1, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_weights(case, dtype):
    q_len, kv_len, page, hq, hkv, d = CASES[case]
    w, _, _ = _run(10 * case, q_len, kv_len, page, hq, hkv, d, dtype, add=["own", "other", "none"][case % 3])
    for b, n in enumerate(q_len):       # a row gives each of its query heads a sum of 1
        if kv_len[b]:
            np.testing.assert_allclose(w[b].sum(1), hq // hkv * n, rtol=1e-3)


@pytest.mark.parametrize("add", ["own", "other", "none"])
@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 2), (64, 7, 1)])
def test_what_is_added_to(add, d, hq, hkv):
    _run(3, [2, 0, 90, 1], [300, 40, 200, 700], 48, hq, hkv, d, "bf16", add=add)


@pytest.mark.parametrize("scale,q_mul", [(0.05, 1.0), (1.0, 3.0)])
def test_scales(scale, q_mul):
    q = randn(8, (20, 4, 64), torch.float16) * q_mul
    _run(7, [20], [333], 16, 4, 2, 64, "fp16", scale=scale, q=q)


def test_strided_queries():
    qkv = randn(5, (33, 12, 64), torch.bfloat16)
    _run(4, [1, 32], [200, 40], 16, 8, 2, 64, "bf16", q=qkv[:, 2:10])


@pytest.mark.parametrize("n", [1, 40])
def test_rows_whose_lse_is_not_finite_give_nothing(n):
    lse = torch.rand((4, n + 2)) + 5
    lse[0, :], lse[1, 0], lse[2, n // 2] = float("-inf"), float("nan"), float("inf")
    _run(6, [n, 2], [300, 50], 16, 4, 2, 64, "bf16", lse=lse.cuda())


def test_repeats_bit_for_bit():
    for q_len, kv in (([1] * 40, list(range(100, 4100, 100))), ([500, 1, 300], [2000, 900, 300])):
        _, score, args = _run(9, q_len, kv, 16, 8, 2, 128, "bf16", add="none")
        first = score.clone()
        for _ in range(3):
            skv.paged_attn_weight(*args, add=False)
            assert torch.equal(torch.nan_to_num(score), torch.nan_to_num(first))


def test_lengths_spans_and_pages_out_of_range():
    """Such requests and pages are left out, the others are right."""
    d, hkv, hq, page = 64, 2, 4, 16
    dt = torch.bfloat16
    k = randn(1, (8, hkv, page, d), dt)
    for table, st, kv, n, status, out in (
            ([[0, 1], [2, 3]], [0, 1, 2], [33, 20], 2, skv.SKV_DEV_BAD_LEN, [0]), ([[0, 1], [2, 3]], [0, 1, 2], [-1, 20], 2, skv.SKV_DEV_BAD_LEN, [0]),
            ([[0, 1], [2, 3]], [0, 3, 4], [2, 20], 4, skv.SKV_DEV_BAD_LEN, [0]), ([[0, 1], [2, 3]], [-1, 1, 2], [20, 20], 2, skv.SKV_DEV_BAD_LEN, [0]),
            ([[0, 1], [2, 3]], [0, 1, 9], [20, 20], 2, skv.SKV_DEV_BAD_LEN, [1]), ([[0, 8], [2, -1]], [0, 1, 2], [20, 20], 2, skv.SKV_DEV_BAD_PAGE, []),
            ([[0, 1], [2, 3]], [0, 1, 0], [20, 20], 2, skv.SKV_DEV_BAD_LEN, [1])):
        cache = skv.PagedCache.wrap(k=k, v=k, block_table=ints(table))
        scores = skv.PagedScores(torch.full((8, hkv, page), -1.0, device="cuda"), torch.zeros((8, hkv, page), dtype=torch.int32, device="cuda"))
        q, lse = randn(2, (n, hq, d), dt), torch.zeros((hq, n), device="cuda")
        skv.paged_attn_weight(cache, scores, q, ints(st), ints(kv), lse, ints([5] * n), 0.125, add=False)
        assert cache.device_status() == status
        score = scores.score[0]
        for b in range(2):
            for j in range(20):
                p = table[b][j // page]
                if not 0 <= p < 8:
                    continue
                got = score[p, :, j % page]
                if b in out:
                    assert (got == -1.0).all()
                    continue
                row = st[b]
                kk = k[p, :, j % page].float()
                want = torch.exp(torch.einsum("hgd,hd->hg", q[row].float().view(hkv, hq // hkv, d), kk) * 0.125).sum(1)
                torch.testing.assert_close(got, want, rtol=1e-4, atol=0)


def test_captured_and_replayed_on_another_stream():
    _, score, args = _run(12, [1] * 9 + [70], [100 * i + 5 for i in range(9)] + [600], 16, 8, 2, 128, "bf16", add="none")
    want, ws = score.clone(), skv.attn_workspace()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        skv.paged_attn_weight(*args, add=False, ws=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            skv.paged_attn_weight(*args, add=False, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    score.fill_(-3.0)
    g.replay()
    g.replay()
    assert torch.equal(score, want)


def test_binding_refusals():
    cache = skv.PagedCache(8, 16, 2, 64, 2, 4, n_layer=2)
    scores = skv.PagedScores.empty(cache)
    one, so = cache.layer(1), scores.layer(1)
    f = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    ok = lambda **kw: skv.paged_attn_weight(**{**dict(cache=one, scores=so, q=q, q_start=ints([0, 1, 3]), kv_len=ints([1, 2]),  # noqa: E731
                                                      lse=f(4, 3), position=ints([0, 0, 1]), sm_scale=0.1), **kw})
    ok()
    for kw, err in ((dict(cache=cache, scores=scores), ValueError), (dict(cache=cache), ValueError), (dict(q=q.half()), TypeError),
                    (dict(q=q[:, :, :32]), ValueError), (dict(lse=f(3, 4)), ValueError), (dict(lse=f(4, 3).double()), TypeError),
                    (dict(position=ints([0])), ValueError), (dict(kv_len=ints([1])), ValueError), (dict(add=f(8, 2, 15)), ValueError),
                    (dict(add=1.5), TypeError), (dict(ws=5), TypeError), (dict(q=q.cpu()), ValueError)):
        with pytest.raises(err):
            ok(**kw)
    for kw in (dict(sm_scale=0.0), dict(sm_scale=float("nan")), dict(ws=torch.zeros(16, dtype=torch.uint8, device="cuda")),
               dict(q=torch.zeros((3, 3, 64), dtype=torch.bfloat16, device="cuda"), lse=f(3, 3))):
        with pytest.raises(skv.SkvError):
            ok(**kw)
