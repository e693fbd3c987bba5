"""What the statistical check of the attention tests can see, without a GPU:
results with the kernel's roundings pass it; a lost value, a page in the wrong
place, a probability in one term where two are promised do not."""
import numpy as np
import pytest
import torch

import paged_stats as S

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(dtype, n_q, n_key, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    q = torch.randn((n_q, 4, d), generator=g).to(dt).double()
    k, v = (torch.randn((n_key, 2, d), generator=g).to(dt).double() for _ in range(2))
    return q, k, v, d ** -0.5, dt


def _round(x, dt):
    return x.to(dt).double()


def _restated(q, k, v, first, scale, dt, terms, sign=1.0, chop=False):
    """The kernel's roundings: P relative to its row's maximum in `terms` terms
    of the type, sums exact, the output once."""
    n, hq, d = q.shape
    m, hkv, _ = k.shape
    out = torch.zeros_like(q)
    for h in range(hq):
        hk = h // (hq // hkv)
        z = q[:, h] @ k[:, hk].T * scale
        if first is not None:
            z = torch.where(torch.arange(m)[None, :] <= first + torch.arange(n)[:, None], z, float("-inf"))
        p = torch.exp(z - z.amax(-1, keepdim=True))
        if terms == 0:
            r = p
        elif chop:
            step = 2 * S.half_step(p, dt)
            r = torch.floor(p / step) * step
        else:
            r = _round(p, dt)
        if terms == 2:
            r = r + sign * _round(p - r, dt)
        out[:, h] = r @ v[:, hk] / p.sum(-1, keepdim=True)
    return _round(out, dt)


CASES = [("bf16", 64, 9001, 64), ("fp16", 64, 20000, 64), ("bf16", 40, 1500, 128), ("fp16", 33, 700, 64)]


def _keys(q, k, first):
    return torch.full((q.shape[0],), k.shape[0]) if first is None else first + 1 + torch.arange(q.shape[0])


@pytest.mark.parametrize("dtype,n_q,n_key,d", CASES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("terms", [1, 2])
def test_the_kernels_roundings_pass(dtype, n_q, n_key, d, causal, terms):
    q, k, v, scale, dt = _case(dtype, n_q, n_key, d)
    first = n_key - n_q if causal else None
    want = S.expected(q, k, v, first, scale, dt, terms == 1)
    row, total = S.excess(_restated(q, k, v, first, scale, dt, terms), *want, _keys(q, k, first))
    assert row <= 1 and total <= 1, (row, total)


@pytest.mark.parametrize("dtype,n_q,n_key,d", CASES)
@pytest.mark.parametrize("rounded_p", [False, True])
@pytest.mark.parametrize("slip", ["row", "page", "rows swapped", "key"])
def test_lost_and_misplaced_keys_fail(dtype, n_q, n_key, d, rounded_p, slip):
    q, k, v, scale, dt = _case(dtype, n_q, n_key, d, 1)
    want = S.expected(q, k, v, None, scale, dt, rounded_p)
    k2, v2 = k.clone(), v.clone()
    at = n_key // 2 // 16 * 16
    if slip == "row":
        v2[at + 3] = 0                                       # one value row lost
    elif slip == "page":
        v2[at:at + 16] = v[at + 16:at + 32]                  # a page of 16 read in place of another
    elif slip == "rows swapped":
        v2[at], v2[at + 1] = v[at + 1], v[at]
    else:
        k2, v2 = torch.cat([k[:at], k[at + 1:]]), torch.cat([v[:at], v[at + 1:]])   # one key skipped
    got = _restated(q, k2, v2, None, scale, dt, 1 if rounded_p else 2)
    row, total = S.excess(got, *want, _keys(q, k, None))
    assert row > 1 or total > 1, (row, total)


# (at 20,000 keys the fp32 sums' own allowance is above fp16's second term)
@pytest.mark.parametrize("dtype,n_q,n_key,d", [c for c in CASES if c[2] < 20000])
@pytest.mark.parametrize("slip", ["dropped", "flipped", "cut off"])
def test_coarser_probabilities_fail_where_two_terms_are_promised(dtype, n_q, n_key, d, slip):
    q, k, v, scale, dt = _case(dtype, n_q, n_key, d, 2)
    want = S.expected(q, k, v, None, scale, dt, False)
    got = {"dropped": lambda: _restated(q, k, v, None, scale, dt, 1),
           "flipped": lambda: _restated(q, k, v, None, scale, dt, 2, sign=-1.0),
           "cut off": lambda: _restated(q, k, v, None, scale, dt, 1, chop=True)}[slip]()
    row, total = S.excess(got, *want, _keys(q, k, None))
    assert total > 1, (row, total)


def test_half_step_is_the_types():
    for dt in DT.values():
        x = torch.tensor([1.0, 1.5, 3.99, 0.3, 1e-3, 100.0])
        for a in x.to(dt):
            up = torch.nextafter(a.float(), torch.tensor(np.inf)).to(dt)   # same value again
            assert up == a
        bits = x.to(dt).view(torch.int16)
        step = (bits + 1).view(dt).double() - x.to(dt).double()
        assert torch.equal(S.half_step(x.to(dt).double(), dt), step / 2)
