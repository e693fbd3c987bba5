"""Waits of paged_attn and cross_attn that run out, without a GPU fault: with a
limit of 1 ns each warp gives up at its first wait that is not met already.
The call returns and sets SKV_DEV_TIMEOUT; the next one, with the same
workspace, is right."""
import pytest
import torch

from paged_harness import DT, ints, randn, starts
from streaming_kv_cache_gb300 import skv

pytestmark = pytest.mark.gpu


def _paged(dt, d, hq, hkv, ql, kv, page=64, wait_ns=0):
    used = [-(-n // page) for n in kv]
    n_page, at = sum(used), 0
    table = torch.zeros((len(kv), max(used)), dtype=torch.int32)
    for b, n in enumerate(used):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    cache = skv.PagedCache.wrap(k=randn(1, (n_page, hkv, page, d), dt), v=randn(2, (n_page, hkv, page, d), dt),
                                block_table=table.cuda(), wait_ns=wait_ns)
    q = randn(3, (sum(ql), hq, d), dt)
    qs, lens = ints(starts(ql)), ints(kv)
    return cache, lambda ws: skv.paged_attn(cache, q, qs, lens, d ** -0.5, lse=True, ws=ws)


SHAPES = [([1] * 9, [1, 40, 128, 129, 1000, 5000, 333, 128, 77]), ([1], [9000]), ([1, 150, 60, 300], [400, 400, 61, 2000]),
          ([1] * 200, [700] * 200), ([100] * 160, [2000] * 160)]


@pytest.mark.parametrize("dtype,d,hq,hkv", [("bf16", 128, 8, 2), ("fp16", 64, 4, 4), ("bf16", 64, 7, 1), ("fp16", 128, 2, 1)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_paged_waits_that_run_out(dtype, d, hq, hkv, shape):
    cache, call = _paged(DT[dtype], d, hq, hkv, *SHAPES[shape])
    ws = skv.attn_workspace()
    want = call(ws)
    assert cache.device_status() == 0
    for ns in (1, 1000, 5000):
        cache.wait_ns = ns
        call(ws)
        torch.cuda.synchronize()
        assert cache.device_status() & ~skv.SKV_DEV_TIMEOUT == 0
        assert ns > 1 or cache.device_status() == skv.SKV_DEV_TIMEOUT
        cache.wait_ns = 0
        cache.status.zero_()
        out, lse = call(ws)
        assert cache.device_status() == 0
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), ns


@pytest.mark.parametrize("n_q", [1, 100])
def test_units_of_milliseconds_against_a_limit_below_and_above(n_q):
    """The scheduler waits a unit long for its queries' buffer (2,500 key
    tiles, some 3 ms): a limit of 0.1 ms runs out, one of a second does not."""
    dt, d, page, n, n_req = torch.bfloat16, 64, 64, 320000, 160
    k = torch.zeros((2, 1, page, d), dtype=dt, device="cuda")
    cache = skv.PagedCache.wrap(k=k, v=torch.ones_like(k), block_table=torch.ones((n_req, n // page), dtype=torch.int32, device="cuda"))
    q, qs, lens = torch.zeros((n_req * n_q, 2, d), dtype=dt, device="cuda"), ints(starts([n_q] * n_req)), ints([n] * n_req)
    ws = skv.attn_workspace()
    for ns, bits in ((10 ** 5, skv.SKV_DEV_TIMEOUT), (10 ** 9, 0), (2 ** 63, 0), (0, 0)):
        cache.status.zero_()
        cache.wait_ns = ns
        out = skv.paged_attn(cache, q, qs, lens, 1.0, ws=ws)
        assert cache.device_status() == bits, ns
        assert bits or (out == 1).all()


@pytest.mark.parametrize("dtype,d,hq,hkv,n_q", [("bf16", 128, 8, 2, 64), ("fp16", 64, 4, 4, 700), ("bf16", 64, 4, 1, 1)])
def test_cross_waits_that_run_out(dtype, d, hq, hkv, n_q):
    dt, kl = DT[dtype], [1500, 0, 129, 3000]
    k, v = randn(1, (sum(kl), hkv, d), dt), randn(2, (sum(kl), hkv, d), dt)
    q, status = randn(3, (4 * n_q, hq, d), dt), torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (ints(starts([n_q] * 4)), ints(starts(kl)[:-1].tolist()), ints(kl), 0.1)
    ws = skv.attn_workspace()
    want = skv.cross_attn(q, k, v, *args, status=status, ws=ws)
    assert status.item() == 0
    skv.cross_attn(q, k, v, *args, status=status, ws=ws, wait_ns=1)
    assert status.item() == skv.SKV_DEV_TIMEOUT
    status.zero_()
    assert torch.equal(skv.cross_attn(q, k, v, *args, status=status, ws=ws), want) and status.item() == 0


def test_layers_take_the_limit_of_their_cache():
    cache = skv.PagedCache(8, 16, 1, 64, 2, 4, n_layer=2, wait_ns=7)
    assert cache.wait_ns == 7 and cache.layer(1).wait_ns == 7
