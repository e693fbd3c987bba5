"""The rope table of an evicting cache, without a GPU."""
import pytest

from streaming_kv_cache_gb300 import skv


def test_an_evicting_cache_with_rope_needs_the_tables_length():
    """Positions go on past max_block * page_size: a token beyond the table would
    be skipped by kv_paged_write and yet be counted as held by the plan."""
    with pytest.raises(ValueError, match="rope_len"):
        skv.PagedCache(8, 16, 2, 64, 2, 4, theta=1e4, evicts=True, device="cpu")
