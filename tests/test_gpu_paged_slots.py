"""Caches with many idle slots and calls with many padding rows: what such a
server passes to the paged calls."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO
from paged_harness import Pages, check, f64, ints, randn, starts
from streaming_kv_cache_gb300 import skv

pytestmark = pytest.mark.gpu


def _among_idle(pg, n_slot, slots):
    """The pool's requests on the given slots of a wider table; the other slots hold no page."""
    table = np.full((n_slot, pg.table.shape[1]), -1, dtype=np.int32)
    table[slots] = pg.table
    return skv.PagedCache.wrap(k=pg.k, v=pg.v, block_table=torch.from_numpy(table).cuda())


def _spread(values, n_slot, slots):
    x = np.zeros(n_slot, dtype=np.int64)
    x[slots] = values
    return x.tolist()


@pytest.mark.parametrize("kv,hkv", [([30000], 1), ([3136], 8), ([9000, 131], 2)])
def test_idle_slots_change_nothing(kv, hkv):
    """Single tokens alone and among idle slots: the same split of the keys, so
    the same bits."""
    d, dt, hq = 128, torch.bfloat16, 4 * hkv
    pg, n = Pages(1, kv, 64, hkv, d, dt), len(kv)
    q = randn(2, (n, hq, d), dt)
    want = skv.paged_attn(pg.cache(skv), q, ints(starts([1] * n)), ints(kv), d ** -0.5, lse=True)
    for n_slot in (3, 40, 256, 900):
        slots = (np.arange(n) * (n_slot - 1) // max(1, n - 1) if n > 1 else np.array([n_slot // 2])).tolist()
        cache = _among_idle(pg, n_slot, slots)
        got = skv.paged_attn(cache, q, ints(starts(_spread([1] * n, n_slot, slots))), ints(_spread(kv, n_slot, slots)),
                             d ** -0.5, lse=True)
        assert cache.device_status() == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), n_slot


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (7, 1, 64)])
def test_chunks_among_idle_slots(hq, hkv, d):
    """Chunks and single tokens on a few of many slots, paused requests among
    them (they hold keys and get no token)."""
    dt, kv, ql = torch.bfloat16, [700, 129, 300, 2000], [300, 1, 0, 41]
    pg = Pages(3, kv, 48, hkv, d, dt)
    q = randn(4, (sum(ql), hq, d), dt)
    want, wlse, mass = PO.paged(f64(q), f64(pg.k), f64(pg.v), pg.table, starts(ql), kv, 0.1)
    for n_slot in (4, 200, 1000):
        slots = [0, n_slot // 3, n_slot // 2, n_slot - 1]
        cache = _among_idle(pg, n_slot, slots)
        out, lse = skv.paged_attn(cache, q, ints(starts(_spread(ql, n_slot, slots))), ints(_spread(kv, n_slot, slots)),
                                  0.1, lse=True)
        assert cache.device_status() == 0
        check(f64(out), f64(lse), want, wlse, mass, dt, 20.0, 20.0, 0.1, d, 2000, str(n_slot))


@pytest.mark.parametrize("n_tok", [5, 64, 600, 8192])
@pytest.mark.parametrize("ql", [[1, 1, 1], [2, 0, 3]])
def test_few_tokens_among_padding_rows(n_tok, ql):
    """A step captured for long chunks that gets single tokens: padding rows are
    neither read (NaN) nor written."""
    d, dt, kv = 128, torch.float16, [3000, 129, 40]
    pg = Pages(5, kv, 16, 2, d, dt)
    n = sum(ql)
    q = torch.full((n_tok, 8, d), float("nan"), dtype=dt, device="cuda")
    q[:n] = randn(6, (n, 8, d), dt)
    out = torch.full((n_tok, 8, d), 5.0, dtype=dt, device="cuda")
    lse = torch.full((8, n_tok), 5.0, device="cuda")
    cache = pg.cache(skv)
    skv.paged_attn(cache, q, ints(starts(ql)), ints(kv), 0.09, out=out, lse=lse)
    want, wlse, mass = PO.paged(f64(q[:n]), f64(pg.k), f64(pg.v), pg.table, starts(ql), kv, 0.09)
    assert cache.device_status() == 0
    check(f64(out[:n]), f64(lse[:, :n]), want, wlse, mass, dt, 20.0, 20.0, 0.09, d, 3000)
    assert (out[n:] == 5).all() and (lse[:, n:] == 5).all()
