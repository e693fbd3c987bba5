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
