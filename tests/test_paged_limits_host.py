"""Limits of scalar arguments of the paged and cross attention calls, without a
GPU."""
import ctypes

import numpy as np
import pytest
import torch

from streaming_kv_cache_gb300 import build as B
from streaming_kv_cache_gb300 import skv

FAKE = 0x10000     # never dereferenced: every case fails validation or stops at the device check


@pytest.fixture(scope="module")
def L():
    B.build()
    return skv.lib()


def _calls(L, scale=1.0, n_req=3):
    n, ws = L.skv_attn_workspace_bytes(), FAKE * 9
    pool = skv.skv_paged(8, 16, 2, 64, 0, 0, 4, 0, FAKE, FAKE * 2, FAKE * 3, None, FAKE * 4)
    st = skv.skv_states(100, 2, 64, 0, 128, 128, FAKE, FAKE * 2, FAKE * 3, FAKE * 4, FAKE * 5)
    return (L.paged_attn(ctypes.byref(pool), 4, n_req, 5, FAKE * 5, 256, FAKE * 6, FAKE * 7, FAKE * 8, None, ws, n, scale, None),
            L.cross_attn(ctypes.byref(st), 4, n_req, 5, FAKE * 6, 256, FAKE * 7, FAKE * 8, None, ws, n, scale, None))


def test_scale_whose_base_two_form_overflows(L):
    """Scores are taken to base two: scale / ln 2 has to be finite too, or a
    score of 0 becomes NaN."""
    big = float(np.finfo(np.float32).max)
    for scale in (big, big * 0.7):                     # 0.7 > ln 2
        assert _calls(L, scale) == (skv.SKV_ERR_INVALID,) * 2, scale


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on the made-up pointers")
def test_largest_and_smallest_scales(L):
    big = float(np.finfo(np.float32).max)
    for scale in (big * 0.69, 1e-45, 1.0):             # 0.69 < ln 2
        assert all(rc in (skv.SKV_ERR_CUDA, skv.SKV_ERR_UNSUPPORTED) for rc in _calls(L, scale)), scale


def test_requests_whose_indices_pass_32_bits(L):
    """A thread's first request is its number times the requests per thread."""
    for n in (2 ** 30 + 1, 2 ** 31 - 1):
        assert _calls(L, n_req=n) == (skv.SKV_ERR_UNSUPPORTED,) * 2, n
