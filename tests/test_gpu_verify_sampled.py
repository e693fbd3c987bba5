"""verify_sampled on the GPU against the oracle: whole numbers, so every one is
equal.  The oracle's sums are in 64 bits, the call's whole numbers of 2^-55:
they part where a draw lies within some 2^-50 of a border between tokens, which
the seeded draws below do not."""
import numpy as np
import pytest
import torch

from oracle import evict_oracle as EO
from paged_harness import ints, starts
from streaming_kv_cache_gb300 import skv

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _strided(x, stride, dtype, offset=0):
    n, v = x.shape
    buf = torch.full((offset + max(n, 1) * stride + 8,), float("nan"), dtype=dtype, device="cuda")
    view = torch.as_strided(buf, (n, v), (stride, 1), offset)
    view.copy_(torch.from_numpy(x))
    return view


def _run(p, q, token, spans, u, r, kv_len, n_tok=None):
    """Both on the same values; p, q device tensors."""
    st = starts(spans)
    status = ints([0])
    f = lambda x: torch.tensor(np.asarray(x), dtype=torch.float32, device="cuda")  # noqa: E731
    n_tok = p.shape[0]
    acc, nxt, held = skv.verify_sampled(p, ints(list(token) + [-5] * (n_tok - len(token))), ints(st), f(list(u) + [0.5] * (n_tok - len(u))),
                                        f(r), q=q, kv_len=ints(kv_len), status=status)
    hp, hq = p.double().cpu().numpy(), q.double().cpu().numpy() if q is not None else None
    u, r = np.asarray(u, dtype=np.float32), np.asarray(r, dtype=np.float32)
    want_status = 0
    for b, n in enumerate(spans):
        lo, hi = int(st[b]), int(st[b + 1])
        if n == 0:
            a, t = 0, -1
        else:
            a, t, s = EO.verify(token[lo:hi], hp[lo:hi], hq[lo:hi] if q is not None else None, u[lo:hi], r[b])
            want_status |= s
        assert (int(acc[b]), int(nxt[b])) == (a, t), (b, n)
        assert int(held[b]) == kv_len[b] - n + a + (n > 0)
    assert int(status) == want_status
    return acc, nxt, held


def _softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab,spans,pad", [
    (1, [1, 3], 0), (2, [2, 0, 5], 1), (31, [1, 4, 9, 0], 0), (100, [7] * 9, 4), (513, [3, 17, 1], 7), (4096, [9] * 5, 0),
    (32003, [5, 40, 2], 5), (151936, [9, 4], 0)])
@pytest.mark.parametrize("draft", [True, False])
def test_verify_sampled(dtype, vocab, spans, pad, draft):
    rng = np.random.default_rng(vocab + len(spans))
    n = sum(spans)
    logits = rng.standard_normal((n + 2, vocab)) * 2
    pn, qn = _softmax(logits), _softmax(logits + 0.4 * rng.standard_normal((n + 2, vocab)))
    token = np.zeros(n, dtype=np.int64)
    for i in range(1, n):
        token[i] = rng.choice(vocab, p=qn[i - 1])
    p = _strided(pn, vocab + pad, DT[dtype], offset=pad % 3)
    q = _strided(qn, vocab + 2 * pad, DT[dtype], offset=pad % 2) if draft else None
    for r in (rng.random(len(spans)), np.zeros(len(spans)), np.full(len(spans), 1 - 2.0 ** -24)):
        _run(p, q, token, spans, rng.random(n) * (1 if draft else 0.2), r, [100 + s for s in spans])


def test_borders_are_exact():
    """Probabilities that are multiples of 2^-10: draws on a border take the
    next token, thresholds are strict."""
    v = 64
    pn, qn = np.full((3, v), 1 / 64), np.full((3, v), 1 / 64)
    pn[0, ::2], pn[0, 1::2] = 3 / 128, 1 / 128
    p, q = (torch.tensor(x, dtype=torch.float32, device="cuda") for x in (pn, qn))
    for k in range(64):
        acc, nxt, _ = _run(p, q, [0, 1], [2], [0.5, 0], [k / 32 if k < 32 else (k + 0.5) / 64], [2])
        assert int(acc) == 0 and (k >= 32 or int(nxt) == 2 * k)     # u q = p: rejected; the rest is 1/128 at the even ones
        _run(p, q, [0, 1], [2], [0.5 - 2 ** -20, 0], [k / 64], [2])
        assert int(_run(p, None, [0], [1], [0], [0.0], [1])[1]) == 0


@pytest.mark.parametrize("r", [-1.0, 0.0, 1.0, 5.0, float("nan"), float("inf"), float("-inf")])
def test_draws_outside_their_range(r):
    pn = np.array([[0, 0, 0.25, 0.5, 0.25, 0, 0, 0]])
    p = torch.tensor(pn, dtype=torch.float32, device="cuda")
    _, nxt, _ = _run(p, None, [0], [1], [0], [r], [1])
    assert int(nxt) == (4 if r >= 1 else 2)


def test_thresholds_outside_their_range():
    p = torch.full((4, 4), 0.25, device="cuda")
    for u in (float("nan"), -1.0, float("inf"), 2.0):
        _run(p, p, [0, 1, 2, 3], [4], [u] * 4, [0.3], [4])


def test_rows_that_leave_nothing():
    v = 700
    pn = _softmax(np.random.default_rng(0).standard_normal((6, v)))
    p = torch.tensor(pn, dtype=torch.float32, device="cuda")
    # q = p: nothing rejected but by u = 1, and then nothing is left of p - q
    acc, nxt, _ = _run(p, p.clone(), [0, 5, 6], [3], [0.3, 1.0, 0], [0.7], [3])
    assert int(acc) == 1
    # the draft has all of p's mass and is rejected: without q nothing is left either
    one = torch.zeros((2, v), device="cuda")
    one[:, 3] = 1
    _run(one, None, [0, 3], [2], [1.0, 0], [0.5], [2])
    # no mass at all
    acc, nxt, _ = _run(torch.zeros((1, v), device="cuda"), None, [0], [1], [0], [0.5], [1])
    assert int(nxt) == -1


@pytest.mark.parametrize("bad", [float("nan"), -0.5, 3.0, float("inf")])
@pytest.mark.parametrize("where", ["p", "q"])
def test_entries_that_are_no_probabilities(bad, where):
    rng = np.random.default_rng(5)
    v = 3000
    p, q = (torch.tensor(_softmax(rng.standard_normal((4, v))), dtype=torch.float32, device="cuda") for _ in range(2))
    (p if where == "p" else q)[:, 1234] = bad
    _run(p, q, [0, 1234, 7, 8], [4], [0.5] * 4, [0.4], [4])
    _run(p, q, [0, 7, 1234, 8], [4], [1e-9, 0.9, 0.5, 0], [0.4], [4])


def test_rows_whose_sum_is_too_large():
    p = torch.ones((1, 50000), device="cuda")
    status = ints([0])
    acc, nxt, held = skv.verify_sampled(p, ints([0]), ints([0, 1]), torch.zeros(1, device="cuda"), torch.full((1,), 0.5, device="cuda"),
                                        status=status)
    assert int(nxt) == -1 and held is None and int(status) == skv.SKV_DEV_BAD_PROB
    p[0, 8:] = 0            # 8: the largest sum there may be
    _, nxt, _ = skv.verify_sampled(p, ints([0]), ints([0, 1]), torch.zeros(1, device="cuda"), torch.full((1,), 0.5, device="cuda"),
                                   status=ints([0]))
    assert int(nxt) == 4


def test_drafts_outside_the_vocabulary():
    p = torch.full((4, 10), 0.1, device="cuda")
    for t in (-1, 10, 2 ** 31 - 1, -2 ** 31):
        for q in (p, None):
            _run(p, q, [0, 3, t, 4], [4], [0.01] * 4, [0.5], [4])
    _run(p, p, [0, 3, 99, 4], [4], [1.0] * 4, [0.5], [4])      # behind a rejected one it is not looked at


def test_spans_out_of_range():
    p = torch.full((4, 10), 0.1, device="cuda")
    status = ints([0])
    acc, nxt, held = skv.verify_sampled(p, ints([0] * 4), ints([0, 2, 1, 9]), torch.zeros(4, device="cuda"),
                                        torch.full((3,), 0.55, device="cuda"), kv_len=ints([2, 5, 7]), status=status)
    assert acc.tolist() == [1, 0, 0] and nxt.tolist() == [5, -1, -1] and held.tolist() == [2, 5, 7]
    assert int(status) == skv.SKV_DEV_BAD_LEN


def test_no_rows_at_all_and_held_in_place():
    p = torch.empty((0, 10), device="cuda")
    kv = ints([4, 5])
    acc, nxt, held = skv.verify_sampled(p, ints([]), ints([0, 0, 0]), torch.empty(0, device="cuda"), torch.zeros(2, device="cuda"),
                                        kv_len=kv, held=kv, status=ints([0]))
    assert acc.tolist() == [0, 0] and nxt.tolist() == [-1, -1] and held.tolist() == [4, 5] and held.data_ptr() == kv.data_ptr()


def test_many_requests_and_graph_replay():
    rng = np.random.default_rng(9)
    spans = rng.integers(0, 4, 1500).tolist()
    n, v = sum(spans), 37
    p, q = (torch.tensor(_softmax(rng.standard_normal((n, v))), dtype=torch.float32, device="cuda") for _ in range(2))
    token, u, r = rng.integers(0, v, n), rng.random(n), rng.random(len(spans))
    want = _run(p, q, token, spans, u, r, [50] * len(spans))
    args = [p, ints(token.tolist()), ints(starts(spans)), torch.tensor(u, dtype=torch.float32, device="cuda"),
            torch.tensor(r, dtype=torch.float32, device="cuda")]
    out = [torch.zeros(len(spans), dtype=torch.int32, device="cuda") for _ in range(3)]
    kw = dict(q=q, kv_len=ints([50] * len(spans)), status=ints([0]), accept_len=out[0], next_token=out[1], held=out[2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        skv.verify_sampled(*args, **kw)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        skv.verify_sampled(*args, **kw)
    for x in out:
        x.fill_(-7)
    g.replay()
    g.replay()
    for got, w in zip(out, want):
        assert torch.equal(got, w)


def test_binding_refusals():
    p, f = torch.full((4, 10), 0.1, device="cuda"), lambda n: torch.zeros(n, device="cuda")
    ok = lambda **kw: skv.verify_sampled(**{**dict(p=p, token=ints([0] * 4), q_start=ints([0, 4]), u=f(4), r=f(1),  # noqa: E731
                                                   status=ints([0])), **kw})
    ok()
    for kw, err in ((dict(p=p.double()), ValueError), (dict(p=p[0]), ValueError), (dict(p=p.t()), ValueError), (dict(q=p[:3]), ValueError),
                    (dict(q=p.half()), TypeError), (dict(q=p.cpu()), ValueError), (dict(token=ints([0] * 3)), ValueError),
                    (dict(token=ints([0] * 4).long()), TypeError), (dict(u=f(3)), ValueError), (dict(r=f(2)), ValueError),
                    (dict(r=0.5), TypeError), (dict(held=ints([0])), ValueError), (dict(kv_len=ints([0, 0])), ValueError),
                    (dict(status=f(1)), TypeError), (dict(p=p.cpu()), ValueError), (dict(accept_len=ints([0, 0])), ValueError)):
        with pytest.raises(err):
            ok(**kw)
    with pytest.raises(skv.SkvError):
        x = ints([0])
        ok(accept_len=x, next_token=x)
