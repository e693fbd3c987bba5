"""paged_attn_weight over many requests, idle slots, long caches and large
pools, against a plain sum in 64 bits on the GPU (the error terms are those of
evict_harness.check_weights)."""
import numpy as np
import pytest
import torch

from paged_harness import DT, ints, starts
from streaming_kv_cache_gb300 import skv

pytestmark = pytest.mark.gpu


def _run(q_len, kv_len, page, hq, hkv, d, dtype, n_page=None, first_page=0, cols=None, seed=0):
    dt, grp, scale = DT[dtype], hq // hkv, d ** -0.5
    g = torch.Generator(device="cuda").manual_seed(seed)
    used = [-(-n // page) for n in kv_len]
    n_page = n_page or sum(used)
    ids = (first_page + torch.randperm(sum(used), generator=g, device="cuda")).to(torch.int32)
    table = torch.zeros((len(kv_len), cols or max(used)), dtype=torch.int32, device="cuda")
    have = torch.arange(table.shape[1], device="cuda")[None, :] < ints(used)[:, None]
    table[have] = ids
    k = torch.empty((n_page, hkv, page, d), dtype=dt, device="cuda")
    k[first_page:].normal_(generator=g)
    cache = skv.PagedCache.wrap(k=k, v=k, block_table=table)
    score = torch.full((n_page, hkv, page), -1.0, device="cuda")
    scores = skv.PagedScores(score, torch.full((n_page, hkv, page), -2, dtype=torch.int32, device="cuda"))
    n_tok = sum(q_len)
    q = torch.empty((n_tok, hq, d), dtype=dt, device="cuda").normal_(generator=g)
    lse = torch.rand((hq, n_tok), generator=g, device="cuda") * 4 + 4
    position = torch.arange(n_tok, dtype=torch.int32, device="cuda")
    st = starts(q_len)
    skv.paged_attn_weight(cache, scores, q, ints(st), ints(kv_len), lse, position, scale, add=False)
    assert cache.device_status() == 0
    qn, kn = float(q.float().norm(dim=-1).max()), max(float(x.float().norm(dim=-1).max()) for x in k[first_page:].split(4096))
    e = d * 2.0 ** -24 * qn * kn * scale + 4 * 2.0 ** -24 * 1.45 * (scale * qn * kn + 8) + 2.0 ** -21
    seen = torch.zeros(score.shape, dtype=torch.bool, device="cuda")
    for b, (n, m) in enumerate(zip(q_len, kv_len)):
        if n == 0 or m == 0:
            continue
        j = torch.arange(m, device="cuda")
        pg, row = table[b].long()[j // page], j % page
        for h in range(hkv):
            kk = k[pg, h, row].double()
            x = q[st[b]:st[b + 1], h * grp:(h + 1) * grp].double().reshape(n * grp, d)
            z = torch.exp(x @ kk.T * scale - lse[h * grp:(h + 1) * grp, st[b]:st[b + 1]].double().T.reshape(-1, 1))
            vis = j[None, :] <= (m - n + torch.arange(n, device="cuda").repeat_interleave(grp))[:, None]
            want = (z * vis).sum(0)
            got = score[pg, h, row].double()
            tol = want * (np.expm1(e) + (grp * n + 2) * 2.0 ** -24) + 2.0 ** -126
            assert bool(((got - want).abs() <= tol).all()), (b, h, float(((got - want).abs() / tol).max()))
            seen[pg, h, row] = True
            assert torch.equal(scores.pos[0][pg[m - n:], h, row[m - n:]], position[st[b]:st[b + 1]])
    assert bool((score[~seen] == -1).all())


@pytest.mark.parametrize("page", [16, 64])
def test_four_thousand_requests(page):
    rng = np.random.default_rng(page)
    kv = rng.integers(1, 300, 4096).tolist()
    ql = [0 if i % 3 == 1 else 1 for i in range(4096)]
    _run(ql, kv, page, 4, 1, 64, "bf16")


@pytest.mark.parametrize("chunk", [1, 1500])
def test_a_long_request_among_thousands_of_short_ones(chunk):
    """One CTA's share holds more requests than its list of them."""
    kv = [3] * 2000 + [60000] + [5] * 2000
    ql = [1] * 2000 + [chunk] + [1] * 2000
    _run(ql, kv, 16, 2, 1, 64, "fp16")


def test_one_request_among_idle_slots():
    for at in (0, 1000, 4095):
        ql, kv = [0] * 4096, [40] * 4096
        ql[at], kv[at] = 70, 900
        _run(ql, kv, 16, 8, 2, 128, "bf16")


@pytest.mark.parametrize("q_len", [[1, 1], [3, 40]])
def test_long_caches(q_len):
    _run(q_len, [300001, 131072], 128, 4, 2, 128, "bf16")


def test_pools_past_32_bit_offsets():
    """Keys beyond 2^31 elements of the pool."""
    _run([1, 200, 1], [1000, 700, 65], 64, 8, 4, 128, "bf16", n_page=70000, first_page=69000)


def test_two_graphs_with_workspaces_of_their_own():
    args, graphs, wants = [], [], []
    for seed, (n, m) in enumerate(((300, 1500), (700, 2000))):
        g = torch.Generator(device="cuda").manual_seed(seed)
        page, hkv, hq, d = 64, 2, 8, 128
        n_page = -(-m // page)
        k = torch.empty((n_page, hkv, page, d), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        cache = skv.PagedCache.wrap(k=k, v=k, block_table=torch.arange(n_page, dtype=torch.int32, device="cuda")[None])
        scores = skv.PagedScores(torch.zeros((n_page, hkv, page), device="cuda"), torch.zeros((n_page, hkv, page), dtype=torch.int32, device="cuda"))
        q = torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        args.append((cache, scores, q, ints([0, n]), ints([m]), torch.full((hq, n), 7.0, device="cuda"), ints([0] * n), d ** -0.5))
    sides = [torch.cuda.Stream() for _ in args]
    ws = [skv.attn_workspace() for _ in args]
    for a, side, w in zip(args, sides, ws):
        skv.paged_attn_weight(*a, add=False, ws=w)
        wants.append(a[1].score.clone())
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            skv.paged_attn_weight(*a, add=False, ws=w)
        graphs.append(g)
    for _ in range(10):
        for a, side, g in zip(args, sides, graphs):
            with torch.cuda.stream(side):
                g.replay()
    torch.cuda.synchronize()
    for a, want in zip(args, wants):
        assert torch.equal(a[1].score, want)
