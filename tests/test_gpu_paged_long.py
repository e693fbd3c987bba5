"""Long runs of keys in one CTA: values of one sign, whose sums drift if they
are cut off at every step, and lengths around the parts that a run is summed
in.  Many requests share the same pages, so that few or no units are split
over CTAs."""
import numpy as np
import pytest
import torch

from paged_harness import DT, ints, starts
from streaming_kv_cache_gb300 import skv

pytestmark = pytest.mark.gpu

PART = 256 * 128        # keys of a part


def _inputs(seed, rows, hq, d, n_pool, dt):
    """Normal queries and keys; values of one sign, each dimension around a size of its own."""
    g = torch.Generator("cuda").manual_seed(seed)
    q = torch.randn((rows, hq, d), generator=g, device="cuda").to(dt)
    k = torch.randn((n_pool, 1, d), generator=g, device="cuda").to(dt)
    v = torch.rand((n_pool, 1, d), generator=g, device="cuda") + 0.5
    return q, k, (v * (1 + torch.rand((d,), generator=g, device="cuda"))).to(dt)


def _want(q, k, v, weight, scale):
    """fp64: out, lse, mass of rows q [n, hq, d] over k, v [m, 1, d], key j
    there weight [n, m] times (0: not at all)."""
    n, hq, d = q.shape
    z = torch.einsum("nhd,md->nhm", q.double(), k[:, 0].double()) * scale + torch.log(weight.double())[:, None, :]
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - lse[..., None])
    return p @ v[:, 0].double(), lse, p @ v[:, 0].double().abs()


def _check(out, lse, want, wlse, mass, dt, q, k, scale, n_key, n_q, what):
    """As paged_harness.check (a rounded output, probabilities rounded once,
    scores and row sums in fp32, the row sums of a part and one step a part),
    and the value sums: a part's MMAs, 8 a key tile, 16 for single tokens (two
    terms of a probability), cut off less than a step (2^-23) of the sum each;
    its addition rounds by half a step.
    The drift of the mean over all outputs is bounded too: a rounding is
    uniform within u, so the mean over d dimensions of different sizes is
    within 6 u / sqrt(3 d) (six deviations, rows counted once); a cut is half a
    step on average."""
    d = q.shape[-1]
    u = torch.finfo(dt).eps / 2
    parts = -(-n_key // PART)
    tiles = min(PART, n_key) / 128
    q_norm, k_norm = float(q.float().norm(dim=-1).max()), float(k.float().norm(dim=-1).max())
    e = d * 2.0 ** -24 * q_norm * k_norm * scale + 2.0 ** -22 + (128 + tiles + parts) * 2.0 ** -24
    cut = (16 if n_q == 1 else 8) * tiles * 2.0 ** -23 + 4 * parts * 2.0 ** -24
    tol = u * (want.abs() * (1 + u) + mass) + (2 * e + cut) * mass + 2.0 ** -24
    err = out.double() - want
    worst = float((err.abs() / tol).max())
    assert worst <= 1, "%s: %.3g times the bound" % (what, worst)
    drift = float((err / want).mean().abs())
    assert drift <= 6 * u / (3 * d) ** 0.5 + cut / 2 + e, "%s: mean off by %.3g" % (what, drift)
    ltol = e + 2.0 ** -22 * (1 + wlse.abs())
    assert ((lse.double() - wlse).abs() <= ltol).all(), what


@pytest.mark.parametrize("dtype,d,repeat", [("fp16", 64, 40), ("fp16", 128, 128), ("bf16", 64, 512), ("bf16", 128, 40)])
@pytest.mark.parametrize("n_q", [1, 70])
def test_values_of_one_sign_over_long_contexts(dtype, d, repeat, n_q):
    """One page of 8,192 keys over and over (to 4 million keys): the softmax of
    one page, a key that a row sees c times having weight c."""
    dt, page, n_req, scale = DT[dtype], 8192, 160, 0.5 * d ** -0.5
    n = page * repeat
    q, k, v = _inputs(repeat + d, n_req * n_q, 2, d, page, dt)
    pool = [x.transpose(0, 1)[None].contiguous() for x in (k, v)]
    cache = skv.PagedCache.wrap(k=pool[0], v=pool[1], block_table=torch.zeros((n_req, repeat), dtype=torch.int32, device="cuda"))
    out, lse = skv.paged_attn(cache, q, ints(starts([n_q] * n_req)), ints([n] * n_req), scale, lse=True)
    assert cache.device_status() == 0
    seen = page - n_q + 1 + torch.arange(n_q, device="cuda")        # of the last page
    weight = repeat - 1 + (torch.arange(page, device="cuda")[None] < seen[:, None]).double()
    for b in range(0, n_req, 40):
        rows = slice(b * n_q, (b + 1) * n_q)
        want, wlse, mass = _want(q[rows], k, v, weight, scale)
        _check(out[rows], lse[:, rows].t(), want, wlse, mass, dt, q, k, scale, n, n_q, "request %d" % b)


@pytest.mark.parametrize("dtype,d", [("fp16", 64), ("bf16", 128)])
@pytest.mark.parametrize("n_q", [1, 70])
def test_lengths_around_the_parts(dtype, d, n_q):
    dt, page, scale = DT[dtype], 128, d ** -0.5
    lens = [PART - 1, PART, PART + 1, PART + 128, 2 * PART, 2 * PART + 1, 50001, 130, 70, 3 * PART + 70] * 18
    most = max(lens)
    n_req, n_page = len(lens), -(-most // page)
    q, k, v = _inputs(d, n_req * n_q, 2, d, n_page * page, dt)
    pool = [x.view(n_page, page, 1, d).transpose(1, 2).contiguous() for x in (k, v)]
    table = torch.arange(n_page, dtype=torch.int32, device="cuda").expand(n_req, n_page).contiguous()
    cache = skv.PagedCache.wrap(k=pool[0], v=pool[1], block_table=table)
    out, lse = skv.paged_attn(cache, q, ints(starts([n_q] * n_req)), ints(lens), scale, lse=True)
    again = skv.paged_attn(cache, q.clone(), ints(starts([n_q] * n_req)), ints(lens), scale)
    in_place = q.clone()
    skv.paged_attn(cache, in_place, ints(starts([n_q] * n_req)), ints(lens), scale, out=in_place)
    assert cache.device_status() == 0
    assert torch.equal(out, again) and torch.equal(out, in_place)
    for b in list(range(20)) + list(range(170, 180)):
        rows, n = slice(b * n_q, (b + 1) * n_q), lens[b]
        seen = n - n_q + 1 + torch.arange(n_q, device="cuda")
        weight = (torch.arange(n, device="cuda")[None] < seen[:, None]).double()
        want, wlse, mass = _want(q[rows], k[:n], v[:n], weight, scale)
        _check(out[rows], lse[:, rows].t(), want, wlse, mass, dt, q, k, scale, n, n_q, "request %d of %d keys" % (b, n))


@pytest.mark.parametrize("n_q", [1, 70])
def test_long_states_that_requests_share(n_q):
    """cross_attn, 262,221 states read by every request, and a part of them."""
    dt, d, n_key, n_req, scale = torch.float16, 64, 2 ** 18 + 77, 160, 0.06
    q, k, v = _inputs(9, n_req * n_q, 2, d, n_key, dt)
    start, length = [0, 5, 77] * 53 + [0], [n_key, PART * 3, 2 ** 18] * 53 + [n_key]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = skv.cross_attn(q, k, v, ints(starts([n_q] * n_req)), ints(start), ints(length), scale, status=status, lse=True)
    assert status.item() == 0
    for b in (0, 1, 2, 80, 158, 159):
        rows, s = slice(b * n_q, (b + 1) * n_q), slice(start[b], start[b] + length[b])
        want, wlse, mass = _want(q[rows], k[s], v[s], torch.ones((1, length[b]), device="cuda"), scale)
        _check(out[rows], lse[:, rows].t(), want, wlse, mass, dt, q, k, scale, length[b], n_q, "request %d" % b)


def test_a_late_key_that_outweighs_the_parts_before_it():
    """The largest score comes in the last part, and in the first: the other
    parts' sums shrink to nothing, or add nothing."""
    dt, d, page, n_req = torch.bfloat16, 64, 128, 160
    n = 3 * PART
    for at in (5, n - 3, PART + 1):
        k = torch.zeros((n // page, 1, page, d), dtype=dt, device="cuda")
        v = torch.ones_like(k)
        k[at // page, 0, at % page, 0] = 200.0
        v[at // page, 0, at % page] = 3.0
        table = torch.arange(n // page, dtype=torch.int32, device="cuda").expand(n_req, n // page).contiguous()
        cache = skv.PagedCache.wrap(k=k, v=v, block_table=table)
        for n_q in (1, 70):
            q = torch.zeros((n_req * n_q, 2, d), dtype=dt, device="cuda")
            q[..., 0] = 1.0
            out, lse = skv.paged_attn(cache, q, ints(starts([n_q] * n_req)), ints([n] * n_req), 1.0, lse=True)
            assert cache.device_status() == 0
            out, lse = out.view(n_req, n_q, 2, d), lse.view(2, n_req, n_q)
            sees = (n - n_q + torch.arange(n_q, device="cuda")) >= at
            assert (out[:, sees] == 3).all() and (out[:, ~sees] == 1).all()
            # exp(-200) of the others is nothing; without the key all scores are 0
            assert (lse[..., sees] == 200).all() or (lse[..., sees] - 200).abs().max() <= 2.0 ** -15
            if (~sees).any():
                left = np.log((n - n_q + 1 + torch.arange(n_q)[~sees.cpu()]).double().numpy())
                assert np.abs(lse[0, 0, ~sees].double().cpu().numpy() - left).max() <= 2.0 ** -20 + 2.0 ** -20 * 11
