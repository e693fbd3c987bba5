"""kv_evict_plan and kv_evict_move at table rows on either side of every
change of form: 4,096 and 8,192 tokens (CTAs of 128, 256 and 512 threads),
16,384 and its multiples (clusters)."""
import pytest

from test_gpu_evict import _plan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["weights", "ties", "odd", "equal"])
@pytest.mark.parametrize("held,keep,page,cols", [
    ([4096, 100], [2000, 99], 64, 0), ([4097, 4000], [4096, 1], 64, 0), ([5000, 4097, 300], [2500, 4096, 150], 64, 2), ([8192, 8191], [8191, 4000], 64, 0),
    ([2049, 2049], [2048, 2048], 64, 90), ([8193, 60], [4000, 59], 16, 0), ([16384], [16000], 64, 0), ([16385], [5], 64, 0), ([32769], [20000], 128, 0)])
def test_evict_at_table_rows_of_every_form(held, keep, page, cols, kind):
    _plan(11, held, keep, page, 2, 1, 4, 60, kind, cols=cols)
