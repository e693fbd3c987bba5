"""The paged cache and cross attention without a GPU: the oracle against
plain torch, the host-side refusals of the C calls, the struct layouts and the
binding's checks."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO
from streaming_kv_cache_gb300 import build as B
from streaming_kv_cache_gb300 import skv

FAKE = 0x10000     # never dereferenced: every case fails validation first
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    B.build()
    return skv.lib()


# ------------------------------------------------------------------ oracle

def test_oracle_attention_is_sdpa_over_the_pages():
    rng = np.random.default_rng(0)
    page, hkv, hq, d = 16, 2, 6, 64
    kv, ql = [37, 5, 64], [5, 5, 1]
    table = np.array([[4, 1, 6, -1], [0, -1, -1, -1], [2, 7, 3, 5]], dtype=np.int32)
    k, v = rng.standard_normal((8, hkv, page, d)), rng.standard_normal((8, hkv, page, d))
    q = rng.standard_normal((11, hq, d))
    qs = np.concatenate([[0], np.cumsum(ql)])
    out, lse, mass = PO.paged(q, k, v, table, qs, kv, 0.3)
    for b in range(3):
        lo, hi, n = qs[b], qs[b + 1], kv[b]
        rows = [torch.from_numpy(x[table[b, :-(-n // page)]]).transpose(0, 1).reshape(hkv, -1, d)[:, :n]
                .repeat_interleave(3, 0) for x in (k, v)]
        keep = torch.arange(n)[None, :] <= (n - (hi - lo) + torch.arange(hi - lo))[:, None]
        x = torch.from_numpy(q[lo:hi]).transpose(0, 1)
        ref = torch.nn.functional.scaled_dot_product_attention(x, rows[0], rows[1], attn_mask=keep, scale=0.3)
        np.testing.assert_allclose(out[lo:hi], ref.transpose(0, 1).numpy(), atol=1e-12)
    # the last token sees all keys: its lse is that of cross attention over them
    ks = np.moveaxis(k[table[2]], 1, 2).reshape(-1, hkv, d)
    vs = np.moveaxis(v[table[2]], 1, 2).reshape(-1, hkv, d)
    o2, l2, _ = PO.cross(q[10:], ks, vs, [0, 1], [0], [64], 0.3)
    np.testing.assert_allclose(o2, out[10:], atol=1e-12)
    np.testing.assert_allclose(l2, lse[:, 10:], atol=1e-12)
    assert (mass >= np.abs(out) - 1e-12).all()


def test_oracle_plan_keeps_every_page_in_one_place():
    """Random steps: a page is on one request or in the queue, never both, and
    slots of live tokens are distinct."""
    rng = np.random.default_rng(1)
    n_req, page, n_page, cols = 6, 16, 40, 8
    table = np.full((n_req, cols), -1, dtype=np.int32)
    queue = rng.permutation(n_page).astype(np.int32)
    state = np.array([0] * n_req + [0, n_page], dtype=np.int32)
    for _ in range(60):
        new = rng.integers(-1, 30, n_req)
        got, status = PO.plan(state, new, table, queue, page, 128)
        table, queue, state = got["table"], got["queue"], got["next_state"]
        held = [int(table[b, j]) for b in range(n_req) for j in range(-(-int(state[b]) // page))]
        free = [int(queue[(state[n_req] + i) % n_page]) for i in range(state[n_req + 1])]
        assert sorted(held + free) == list(range(n_page))
        live = got["slot"][got["slot"] >= 0]
        assert len(set(live.tolist())) == len(live)
        assert status & ~(PO.NO_PAGE | PO.TABLE_FULL) == 0


def test_oracle_plan_by_hand():
    """Page size 16; request 0 holds 15 tokens on page 5 and gets 3, request 1
    has finished with 17 tokens on pages 2 and 7, request 2 starts with 16."""
    table = np.array([[5, -1], [2, 7], [-1, -1]], dtype=np.int32)
    queue = np.array([9, 9, 1, 3, 4, 6, 0, 9], dtype=np.int32)
    got, status = PO.plan([15, 17, 0, 6, 3], [3, -1, 16], table, queue, 16, 20)
    # free entries: positions 6, 7, 0 -> pages 0, 9, 9
    assert status == 0
    assert got["q_start"].tolist() == [0, 3, 3, 19]
    assert got["kv_len"].tolist() == [18, 0, 16]
    assert got["next_state"].tolist() == [18, 0, 16, 0, 3]
    assert got["table"].tolist() == [[5, 0], [2, 7], [9, -1]]
    assert got["queue"].tolist() == [9, 2, 7, 3, 4, 6, 0, 9]
    assert got["position"].tolist() == [15, 16, 17] + list(range(16)) + [0]
    assert got["slot"].tolist() == [95, 0, 1] + [9 * 16 + i for i in range(16)] + [-1]


def test_oracle_rotation_is_a_complex_product():
    x = np.random.default_rng(2).standard_normal((3, 2, 8))
    pos = [0, 5, 1000003]
    y = PO.rotate(x, pos, 1e4)
    z = x[..., :4] + 1j * x[..., 4:]
    w = z * np.exp(1j * np.array(pos)[:, None, None] * 1e4 ** (-2 * np.arange(4) / 8))
    np.testing.assert_allclose(y, np.concatenate([w.real, w.imag], -1), atol=1e-9)


# ---------------------------------------------------------------- refusals

def _pool(**kw):
    base = dict(n_page=8, page_size=16, n_kv_head=2, head_dim=64, dtype=0, rope_len=0, max_block=4, reserved=0,
                k=FAKE, v=FAKE * 2, block_table=FAKE * 3, rope=0, status=FAKE * 4)
    base.update(kw)
    return skv.skv_paged(**base)


def _states(**kw):
    base = dict(n_key=100, n_kv_head=2, head_dim=64, dtype=0, k_stride=128, v_stride=128, k=FAKE, v=FAKE * 2,
                k_start=FAKE * 3, k_len=FAKE * 4, status=FAKE * 5)
    base.update(kw)
    return skv.skv_states(**base)


def _plan(L, pool=None, n_req=3, n_tok=5, state=FAKE * 5, new_len=FAKE * 6, queue=FAKE * 7, q_start=FAKE * 8,
          kv_len=FAKE * 9, nxt=FAKE * 10, position=FAKE * 11, slot=FAKE * 12):
    return L.kv_paged_plan(ctypes.byref(pool or _pool()), n_req, n_tok, state, new_len, queue, q_start, kv_len, nxt,
                           position, slot, None)


def _write(L, pool=None, hq=4, n=5, q=FAKE * 5, qs=256, k=FAKE * 6, ks=128, v=FAKE * 7, vs=128, position=FAKE * 8,
           slot=FAKE * 9, q_out=FAKE * 10):
    return L.kv_paged_write(ctypes.byref(pool or _pool()), hq, n, q, qs, k, ks, v, vs, position, slot, q_out, None)


def _attn(L, pool=None, hq=4, n_req=3, n_tok=5, q=FAKE * 5, qs=256, q_start=FAKE * 6, kv_len=FAKE * 7, out=FAKE * 8,
          lse=None, ws=FAKE * 9, ws_bytes=None, scale=1.0):
    n = L.skv_attn_workspace_bytes() if ws_bytes is None else ws_bytes
    return L.paged_attn(ctypes.byref(pool or _pool()), hq, n_req, n_tok, q, qs, q_start, kv_len, out, lse, ws, n, scale,
                        None)


def _cross(L, st=None, hq=4, n_req=3, n_tok=5, q=FAKE * 6, qs=256, q_start=FAKE * 7, out=FAKE * 8, lse=None,
           ws=FAKE * 9, ws_bytes=None, scale=1.0):
    n = L.skv_attn_workspace_bytes() if ws_bytes is None else ws_bytes
    return L.cross_attn(ctypes.byref(st or _states()), hq, n_req, n_tok, q, qs, q_start, out, lse, ws, n, scale, None)


NO_GPU = (skv.SKV_ERR_CUDA, skv.SKV_ERR_UNSUPPORTED)
no_gpu_here = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on the made-up pointers")


@no_gpu_here
def test_good_arguments_reach_the_device_check(L):
    for call in (_plan, _write, _attn, _cross):
        assert call(L) in NO_GPU, call
    assert _write(L, q=None, q_out=None, hq=0) in NO_GPU
    assert _write(L, q_out=FAKE * 5) in NO_GPU                          # q in place
    assert _write(L, pool=_pool(rope=FAKE, rope_len=9)) in NO_GPU
    assert _attn(L, lse=FAKE) in NO_GPU and _cross(L, lse=FAKE) in NO_GPU
    assert _attn(L, hq=256, qs=256 * 64) in NO_GPU                      # 128 query heads per kv head
    assert _cross(L, st=_states(k_stride=136, v_stride=1024)) in NO_GPU


@pytest.mark.parametrize("bad", [
    dict(n_page=0), dict(page_size=0), dict(page_size=24), dict(page_size=8), dict(max_block=0), dict(status=0),
    dict(block_table=0), dict(block_table=FAKE + 2), dict(n_page=1 << 27), dict(status=FAKE + 1)])
def test_bad_pool(L, bad):
    for call in (_plan, _write, _attn):
        assert call(L, pool=_pool(**bad)) == skv.SKV_ERR_INVALID, (call, bad)


@pytest.mark.parametrize("bad", [
    dict(n_kv_head=0), dict(head_dim=96), dict(head_dim=0), dict(dtype=2), dict(dtype=-1), dict(k=0), dict(v=0),
    dict(k=FAKE + 8), dict(v=FAKE + 2), dict(n_kv_head=1 << 29)])
def test_bad_pages(L, bad):
    for call in (_write, _attn):
        assert call(L, pool=_pool(**bad)) == skv.SKV_ERR_INVALID, (call, bad)


def test_null_descriptors(L):
    ws = L.skv_attn_workspace_bytes()
    assert L.kv_paged_plan(None, 1, 1, *[FAKE] * 8, None) == skv.SKV_ERR_INVALID
    assert L.kv_paged_write(None, 4, 1, FAKE, 256, FAKE, 128, FAKE, 128, FAKE, FAKE, FAKE, None) == skv.SKV_ERR_INVALID
    assert L.paged_attn(None, 4, 1, 1, FAKE, 256, FAKE, FAKE, FAKE, None, FAKE, ws, 1.0, None) == skv.SKV_ERR_INVALID
    assert L.cross_attn(None, 4, 1, 1, FAKE, 256, FAKE, FAKE, None, FAKE, ws, 1.0, None) == skv.SKV_ERR_INVALID


@pytest.mark.parametrize("bad", [
    dict(n_req=-1), dict(n_tok=-1), dict(n_tok=(1 << 30) + 1), dict(state=0), dict(state=FAKE + 2), dict(new_len=0),
    dict(queue=0), dict(q_start=0), dict(kv_len=0), dict(nxt=0), dict(position=0), dict(slot=0), dict(slot=FAKE + 1),
    dict(nxt=FAKE * 5), dict(nxt=FAKE * 5 + 8), dict(nxt=FAKE * 5 - 8)])
def test_bad_plan_arguments(L, bad):
    assert _plan(L, **bad) == skv.SKV_ERR_INVALID


def test_plan_request_limit(L):
    assert _plan(L, n_req=skv.SKV_PAGED_MAX_REQUESTS + 1) == skv.SKV_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(hq=-1), dict(hq=0), dict(q=0), dict(q_out=0), dict(k=0), dict(v=0), dict(slot=0), dict(k=FAKE + 2),
    dict(q=FAKE + 8), dict(q_out=FAKE + 8), dict(ks=120), dict(ks=132), dict(vs=0), dict(qs=248), dict(qs=260),
    dict(pool=_pool(rope=FAKE, rope_len=0)), dict(pool=_pool(rope=0, rope_len=4)), dict(pool=_pool(rope=FAKE + 4, rope_len=4)),
    dict(pool=_pool(rope=FAKE, rope_len=4), position=0),
    dict(q_out=FAKE * 5 + 64),                    # overlaps q without being q
    dict(q_out=FAKE * 5, qs=264)])                # q itself, but not contiguous
def test_bad_write_arguments(L, bad):
    assert _write(L, **bad) == skv.SKV_ERR_INVALID


@pytest.mark.parametrize("bad", [
    dict(hq=0), dict(hq=3), dict(n_req=-1), dict(n_tok=-1), dict(q=0), dict(q=FAKE + 8), dict(qs=248), dict(qs=260),
    dict(q_start=0), dict(out=0), dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf"))])
def test_bad_attention_arguments(L, bad):
    assert _attn(L, **bad) == skv.SKV_ERR_INVALID
    assert _cross(L, **bad) == skv.SKV_ERR_INVALID


def test_outputs_that_overlap_inputs(L):
    row = 5 * 256 * 2                                                   # bytes of q, and of out
    for call, q in ((_attn, FAKE * 5), (_cross, FAKE * 6)):
        for out in (q + 512, q + row - 16, q - 16, q - row + 16):
            assert call(L, out=out) == skv.SKV_ERR_INVALID, out
        assert call(L, out=q, qs=264) == skv.SKV_ERR_INVALID            # q itself, but not contiguous
    kv = 5 * 128 * 2
    for what in (dict(k=FAKE * 6), dict(v=FAKE * 7)):
        x, = what.values()
        for out in (x, x + kv - 16, x - row + 16):
            assert _write(L, q_out=out, **what) == skv.SKV_ERR_INVALID, (what, out)


@no_gpu_here
def test_outputs_in_place_or_apart(L):
    row = 5 * 256 * 2
    for call, q in ((_attn, FAKE * 5), (_cross, FAKE * 6)):
        for out in (q, q + row, q - row):
            assert call(L, out=out) in NO_GPU, out
        assert call(L, out=q, n_tok=1, qs=768) in NO_GPU                # one token has no stride
    assert _write(L, q_out=FAKE * 5, n=1, qs=768) in NO_GPU
    # parts of one projection, its queries rotated to another place
    assert _write(L, q=FAKE * 5, qs=512, k=FAKE * 5 + 512, ks=512, v=FAKE * 5 + 768, vs=512) in NO_GPU


def test_attention_limits(L):
    for call in (_attn, _cross):
        assert call(L, hq=258, qs=258 * 64) == skv.SKV_ERR_UNSUPPORTED     # 129 query heads per kv head
        assert call(L, n_tok=1 << 30, hq=4) == skv.SKV_ERR_UNSUPPORTED
    assert _attn(L, kv_len=0) == skv.SKV_ERR_INVALID
    assert _cross(L, st=_states(n_key=(1 << 30) + 1)) == skv.SKV_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [
    dict(n_key=-1), dict(n_kv_head=0), dict(head_dim=80), dict(dtype=7), dict(k_stride=120), dict(k_stride=132),
    dict(v_stride=64), dict(k=0), dict(v=FAKE + 4), dict(k_start=0), dict(k_len=0), dict(k_len=FAKE + 2), dict(status=0)])
def test_bad_states(L, bad):
    assert _cross(L, st=_states(**bad)) == skv.SKV_ERR_INVALID


def test_empty_calls_touch_nothing(L):
    assert _write(L, n=0) == skv.SKV_OK
    for call in (_attn, _cross):
        assert call(L, n_req=0) == skv.SKV_OK
        assert call(L, n_tok=0) == skv.SKV_OK


def test_small_workspace(L):
    need = L.skv_attn_workspace_bytes()
    if need:
        for call in (_attn, _cross):
            assert call(L, ws_bytes=need - 1) == skv.SKV_ERR_INVALID
            assert call(L, ws=0) == skv.SKV_ERR_INVALID
            assert call(L, ws=FAKE + 8) == skv.SKV_ERR_INVALID


def test_status_texts(L):
    seen = {skv.status_string(c) for c in (16, 32, 64, 128, 256)}
    assert len(seen) == 5 and all(s.startswith("device: ") for s in seen)


def test_struct_layouts_match_the_header(L, tmp_path):
    src = tmp_path / "layout.c"
    lines = []
    for st in (skv.skv_paged, skv.skv_states):
        lines.append('printf("%s.size %%zu\\n", sizeof(%s));' % (st.__name__, st.__name__))
        for f, _ in st._fields_:
            lines.append('printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (st.__name__, f, st.__name__, f))
    lines.append('printf("max %d\\n", SKV_PAGED_MAX_REQUESTS);')
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "skv.h"\nint main(void) {\n%s\nreturn 0; }\n'
                   % "\n".join(lines))
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(B.ROOT, "include"), str(src),
                    "-o", exe], check=True)
    out = dict(line.split() for line in subprocess.run([exe], capture_output=True, text=True).stdout.splitlines())
    for st in (skv.skv_paged, skv.skv_states):
        assert int(out[st.__name__ + ".size"]) == ctypes.sizeof(st)
        for f, _ in st._fields_:
            assert int(out["%s.%s" % (st.__name__, f)]) == getattr(st, f).offset, f
    assert int(out["max"]) == skv.SKV_PAGED_MAX_REQUESTS


def test_binding_refuses_tensors_that_are_not_on_a_gpu(L):
    t = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(ValueError):
        skv.PagedCache.wrap(block_table=t, page_queue=torch.zeros(8, dtype=torch.int32), page_size=16,
                            state=torch.zeros(4, dtype=torch.int32), status=torch.zeros(1, dtype=torch.int32))
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        skv.cross_attn(x, x, x, torch.zeros(2, dtype=torch.int32), one, one, 1.0, status=one)
    with pytest.raises(ValueError):
        skv.PagedCache.wrap(block_table=t)
    with pytest.raises(TypeError):
        skv.cross_attn(x, [x], x, one, one, one, 1.0, status=one)
