"""The Python side of the paged cache: what is fixed, and its indices."""
import pytest
import torch

from streaming_kv_cache_gb300 import skv

pytestmark = pytest.mark.gpu


def _cache(**kw):
    return skv.PagedCache(8, 16, 1, 64, 2, 4, theta=1e4, **kw)


@pytest.mark.parametrize("name", ["k", "v", "block_table", "page_queue", "state", "rope", "status", "page_size", "n_req"])
def test_what_the_calls_keep_cannot_be_replaced(name):
    """An assignment would be ignored: the calls go on with the first tensor."""
    cache = _cache()
    old = getattr(cache, name)
    with pytest.raises(AttributeError):
        setattr(cache, name, old.clone() if isinstance(old, torch.Tensor) else old + 1)
    assert getattr(cache, name) is old
    if isinstance(old, torch.Tensor):
        old.zero_()                         # written into, as ever
    with pytest.raises(AttributeError):
        setattr(_cache(n_layer=2).layer(1), name, old)


def test_wait_limit_may_be_set():
    cache = _cache()
    cache.wait_ns = 5
    assert cache.wait_ns == 5


def test_layers_by_index():
    cache = _cache(n_layer=3)
    for i, j in ((0, 0), (2, 2), (-1, 2), (-3, 0)):
        c = cache.layer(i)
        assert c.k.data_ptr() == cache.layer(j).k.data_ptr()
        assert c.layer(0).k.data_ptr() == c.k.data_ptr() and c.layer(-1).v.data_ptr() == c.v.data_ptr()
        with pytest.raises(IndexError):
            c.layer(1)
    for i in (3, -4):
        with pytest.raises(IndexError):
            cache.layer(i)


def test_caches_without_their_parts():
    table = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    plan_only = skv.PagedCache.wrap(block_table=table, page_queue=torch.zeros(4, dtype=torch.int32, device="cuda"), page_size=16)
    with pytest.raises(ValueError):
        plan_only.layer(0)
    with pytest.raises(ValueError):
        skv.PagedCache.wrap(page_queue=table[0], page_size=16)
