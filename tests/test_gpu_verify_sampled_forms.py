"""verify_sampled over every form of its launch, against whole-number
arithmetic."""
import numpy as np
import pytest

from test_gpu_verify_sampled import DT, _softmax
from test_gpu_verify_sampled_exact import _check, _strided

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("n_req,vocab,pad", [
    (15, 5003, 5), (16, 5003, 5), (16, 33000, 0), (37, 33000, 0), (37, 4999, 1), (38, 33000, 0), (38, 5000, 0), (64, 33001, 7), (64, 5000, 0),
    (151, 5000, 0), (152, 5001, 7), (200, 5000, 8), (303, 2049, 7), (304, 33000, 0)])
def test_batches_of_every_launch_shape(n_req, vocab, pad, draft, dtype):
    """Requests of 1 to 3 rows: few and many of them over vocabularies that
    spread a request over one CTA, or a cluster of up to 16, of either size."""
    rng = np.random.default_rng(n_req + vocab)
    spans = rng.integers(1, 4, n_req).tolist()
    n = sum(spans)
    logits = rng.standard_normal((n, vocab), dtype=np.float32) * 2
    pn, qn = _softmax(logits), _softmax(logits + 0.4 * rng.standard_normal((n, vocab), dtype=np.float32))
    token = rng.integers(0, vocab, n)
    token[1:] = np.argmax(qn[:-1] * rng.random((n - 1, vocab), dtype=np.float32), -1)     # mostly likely ones
    p = _strided(pn, vocab + pad, DT[dtype], 0)
    q = _strided(qn, vocab + pad, DT[dtype], 0) if draft else None
    _check(p, q, token, spans, rng.random(n) * (1 if draft else 0.01), rng.random(n_req))
