"""Waits of paged_attn_weight that run out, without a GPU fault: with a limit
of 1 ns each warp gives up at its first wait that is not met already.  The
call returns and sets SKV_DEV_TIMEOUT; the next one is right."""
import pytest
import torch

from paged_harness import DT, ints, randn, starts
from streaming_kv_cache_gb300 import skv

pytestmark = pytest.mark.gpu

SHAPES = [([1] * 9, [1, 40, 128, 129, 1000, 5000, 333, 128, 77]), ([1], [9000]), ([1, 150, 60, 300], [400, 400, 61, 2000]),
          ([1] * 200, [700] * 200), ([100] * 160, [2000] * 160), ([2000], [2000])]


@pytest.mark.parametrize("dtype,d,hq,hkv", [("bf16", 128, 8, 2), ("fp16", 64, 4, 4), ("bf16", 64, 7, 1), ("fp16", 128, 2, 1)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_weight_waits_that_run_out(dtype, d, hq, hkv, shape):
    ql, kv = SHAPES[shape]
    page, dt = 64, DT[dtype]
    used = [-(-n // page) for n in kv]
    table, at = torch.zeros((len(kv), max(used)), dtype=torch.int32), 0
    for b, n in enumerate(used):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    k = randn(1, (at, hkv, page, d), dt)
    cache = skv.PagedCache.wrap(k=k, v=k, block_table=table.cuda())
    n_tok = sum(ql)
    scores = skv.PagedScores(torch.zeros((at, hkv, page), device="cuda"), torch.zeros((at, hkv, page), dtype=torch.int32, device="cuda"))
    args = (cache, scores, randn(3, (n_tok, hq, d), dt), ints(starts(ql)), ints(kv), torch.full((hq, n_tok), 7.0, device="cuda"),
            torch.arange(n_tok, dtype=torch.int32, device="cuda"), d ** -0.5)
    ws = skv.attn_workspace()
    skv.paged_attn_weight(*args, add=False, ws=ws)
    want, pos = scores.score.clone(), scores.pos.clone()
    assert cache.device_status() == 0
    for ns in (1, 1000, 5000):
        cache.wait_ns = ns
        skv.paged_attn_weight(*args, add=False, ws=ws)
        torch.cuda.synchronize()
        assert cache.device_status() & ~skv.SKV_DEV_TIMEOUT == 0
        assert ns > 1 or cache.device_status() == skv.SKV_DEV_TIMEOUT
        cache.wait_ns = 0
        cache.status.zero_()
        skv.paged_attn_weight(*args, add=False, ws=ws)
        assert cache.device_status() == 0
        assert torch.equal(scores.score, want) and torch.equal(scores.pos, pos), ns


def test_a_limit_that_is_not_reached():
    k = randn(1, (40, 2, 64, 64), torch.bfloat16)
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(1, 40)
    out = []
    for ns in (0, 10 ** 9):
        cache = skv.PagedCache.wrap(k=k, v=k, block_table=table, wait_ns=ns)
        scores = skv.PagedScores(torch.zeros((40, 2, 64), device="cuda"), torch.zeros((40, 2, 64), dtype=torch.int32, device="cuda"))
        skv.paged_attn_weight(cache, scores, randn(2, (300, 4, 64), torch.bfloat16), ints([0, 300]), ints([2500]),
                              torch.full((4, 300), 8.0, device="cuda"), ints([0] * 300), 0.125)
        assert cache.device_status() == 0
        out.append(scores.score)
    assert torch.equal(*out)
