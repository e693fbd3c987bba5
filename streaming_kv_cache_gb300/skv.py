"""Python binding of libskv (ctypes).

Argument marshalling only: every step of the streaming-attention path runs in
the library's CUDA kernels.  PyTorch provides device memory and the current
stream.  The functions carry the C entry points' names; see include/skv.h for
the full contract.
"""
from __future__ import annotations

import ctypes
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libskv.so")

SKV_OK, SKV_ERR_INVALID, SKV_ERR_UNSUPPORTED, SKV_ERR_CUDA, SKV_ERR_TOO_LARGE = 0, -1, -2, -3, -4
SKV_NOALLOC_MAX_CACHE_VIEWS = 16384
SKV_DEV_TIMEOUT, SKV_DEV_BAD_HEAD, SKV_DEV_TAIL_OVERFLOW, SKV_DEV_BAD_TAIL = 1, 2, 4, 8
SKV_DEV_NO_PAGE, SKV_DEV_BAD_LEN, SKV_DEV_BAD_PAGE, SKV_DEV_BAD_POS, SKV_DEV_TABLE_FULL = 16, 32, 64, 128, 256
SKV_PAGED_MAX_REQUESTS, SKV_MAX_KEYS = 4096, 1 << 26
_Tensor = torch.Tensor                                 # looked up several times a call
_DTYPE_CODE = {torch.bfloat16: 0, torch.float16: 1}   # SKV_BF16, SKV_FP16

# every function the C header declares
EXPORTS = ("skv_version", "skv_status_string", "skv_last_cuda_error", "skv_row_cap",
           "skv_build_rope_table", "skv_build_mrope_table", "kv_write_rows", "kv_stream_insert", "kv_stream_insert_noalloc",
           "stream_attn_prefill", "stream_attn_prefill_insert", "stream_attn_prefill_tail",
           "stream_attn_window",
           "skv_verify_workspace_bytes", "stream_attn_verify",
           "kv_paged_plan", "kv_paged_write", "skv_attn_workspace_bytes", "paged_attn", "cross_attn")


class SkvError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        msg = "%s: %s" % (what, status_string(code)) if what else status_string(code)
        if code == SKV_ERR_CUDA:
            msg += " (cudaError %d)" % lib().skv_last_cuda_error()
        super().__init__(msg)


class skv_cache(ctypes.Structure):
    _fields_ = [("n_cache", ctypes.c_int32), ("n_view", ctypes.c_int32),
                ("n_frame", ctypes.c_int32), ("frame_len", ctypes.c_int32),
                ("prefix_len", ctypes.c_int32), ("tail_cap", ctypes.c_int32),
                ("n_kv_head", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("row_cap", ctypes.c_int32), ("rope_len", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("vt", ctypes.c_void_p),
                ("head", ctypes.c_void_p), ("sync", ctypes.c_void_p),
                ("rope", ctypes.c_void_p), ("status", ctypes.c_void_p),
                ("wait_ns", ctypes.c_uint64), ("rope_mode", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class skv_paged(ctypes.Structure):
    _fields_ = [("n_page", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_kv_head", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("rope_len", ctypes.c_int32),
                ("max_block", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("rope", ctypes.c_void_p),
                ("status", ctypes.c_void_p), ("wait_ns", ctypes.c_uint64)]


class skv_states(ctypes.Structure):
    _fields_ = [("n_key", ctypes.c_int32), ("n_kv_head", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_start", ctypes.c_void_p), ("k_len", ctypes.c_void_p),
                ("status", ctypes.c_void_p), ("wait_ns", ctypes.c_uint64)]


_lib_handle = None


def lib():
    """Load libskv.so (built in-tree by streaming_kv_cache_gb300.build)."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError("libskv.so is not built (%s); run streaming_kv_cache_gb300.build.build()"
                              % _LIB_PATH)
        L = ctypes.CDLL(_LIB_PATH)
        P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        cp, pp, I64 = ctypes.POINTER(skv_cache), ctypes.POINTER(skv_paged), ctypes.c_int64
        sig = {
            "skv_version": ([], ctypes.c_int),
            "skv_status_string": ([ctypes.c_int], ctypes.c_char_p),
            "skv_last_cuda_error": ([], ctypes.c_int),
            "skv_row_cap": ([I32, I32, I32, I32, I32], I32),
            "skv_build_rope_table": ([P, I32, I32, ctypes.c_double, P], ctypes.c_int),
            "skv_build_mrope_table": ([P, I32, I32, ctypes.c_double, I32, I32, I32, I32, I32,
                                       ctypes.c_uint64, ctypes.c_uint64, P], ctypes.c_int),
            "kv_write_rows": ([cp, I32, I32, P, P, P], ctypes.c_int),
            "kv_stream_insert": ([cp, P, P, P], ctypes.c_int),
            "kv_stream_insert_noalloc": ([cp, P, P, P], ctypes.c_int),
            "stream_attn_prefill": ([cp, I32, P, P, P, ctypes.c_float, P], ctypes.c_int),
            "stream_attn_prefill_insert": ([cp, I32, P, P, P, P, P, ctypes.c_float, P], ctypes.c_int),
            "stream_attn_prefill_tail": ([cp, I32, I32, P, P, P, P, P, P, ctypes.c_float, P],
                                         ctypes.c_int),
            "stream_attn_window": ([cp, I32, P, P, P, ctypes.c_float, P], ctypes.c_int),
            "skv_verify_workspace_bytes": ([cp, I32, I32], SZ),
            "stream_attn_verify": ([cp, I32, I32, P, P, P, P, P, P, P, P, P, P, SZ,
                                    ctypes.c_float, P], ctypes.c_int),
            "kv_paged_plan": ([pp, I32, I32, P, P, P, P, P, P, P, P, P], ctypes.c_int),
            "kv_paged_write": ([pp, I32, I32, P, I64, P, I64, P, I64, P, P, P, P], ctypes.c_int),
            "skv_attn_workspace_bytes": ([], SZ),
            "paged_attn": ([pp, I32, I32, I32, P, I64, P, P, P, P, P, SZ, ctypes.c_float, P],
                           ctypes.c_int),
            "cross_attn": ([ctypes.POINTER(skv_states), I32, I32, I32, P, I64, P, P, P, P, SZ,
                            ctypes.c_float, P], ctypes.c_int),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, res
        _lib_handle = L
    return _lib_handle


def status_string(code: int) -> str:
    return lib().skv_status_string(int(code)).decode()


def _check(rc: int, what: str):
    if rc != SKV_OK:
        raise SkvError(rc, what)


def _stream():
    """The current torch stream of the current device: the library launches
    on the current device, so the tensors of a call must live there."""
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _need(t, shape, dtype, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device.type != "cuda":
        raise ValueError("%s must be on a CUDA device" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def skv_row_cap(P, V, F, T, tail_cap) -> int:
    r = lib().skv_row_cap(P, V, F, T, tail_cap)
    if r < 0:
        raise SkvError(SKV_ERR_INVALID, "skv_row_cap")
    return r


def skv_build_rope_table(tab: torch.Tensor, theta: float):
    n_pos, half, two = tab.shape
    _need(tab, (n_pos, half, 2), torch.float32, "rope table")
    _check(lib().skv_build_rope_table(_ptr(tab), n_pos, 2 * half, float(theta), _stream()),
           "skv_build_rope_table")


def section_masks(sec) -> tuple:
    """(h_mask, w_mask) of a frequency -> component map (0 = t, 1 = h, 2 = w)."""
    h = sum(1 << i for i, c in enumerate(sec) if int(c) == 1)
    w = sum(1 << i for i, c in enumerate(sec) if int(c) == 2)
    return h, w


def skv_build_mrope_table(tab: torch.Tensor, theta: float, P: int, V: int, F: int, T: int,
                          grid_w: int, sec):
    """The multi-section rotary table (see include/skv.h): row n holds the
    angles of the token at logical index n; sec maps frequency i to its
    component (0 = temporal, 1 = height, 2 = width)."""
    n_pos, half, two = tab.shape
    _need(tab, (n_pos, half, 2), torch.float32, "rope table")
    if len(sec) != half:
        raise ValueError("sec must give a component for each of the %d frequencies" % half)
    h, w = section_masks(sec)
    _check(lib().skv_build_mrope_table(_ptr(tab), n_pos, 2 * half, float(theta), P, V, F, T, grid_w,
                                       h, w, _stream()), "skv_build_mrope_table")


class StreamCache:
    """C independent streaming caches of one geometry, in device memory.

    Tensors (all zero-initialised, owned by this object):
      k      bf16 [C][Hkv][row_cap][d]   pre-RoPE keys
      vt     bf16 [C][Hkv][d][row_cap]   values, dimension-major
      head   int32 [C][V]                ring heads
      sync   int32 [C][V]                insert counters
      rope   fp32 [rope_len][d/2][2]     (cos, sin) table
      status int32 [1]                   device status bits

    mrope=(grid_w, sec) selects the multi-section rotary reading (rope_mode 1):
    frames are rows of grid_w tokens and sec maps each of the d/2
    frequencies to its component (0 = temporal, 1 = height, 2 = width).
    """

    def __init__(self, C, P, V, F, T, Hkv, d, theta, tail_cap=128, device="cuda", wait_ns=0,
                 mrope=None):
        self.C, self.P, self.V, self.F, self.T = C, P, V, F, T
        self.Hkv, self.d, self.theta, self.tail_cap = Hkv, d, float(theta), tail_cap
        self.row_cap = skv_row_cap(P, V, F, T, tail_cap)
        self.rope_len = P + V * F * T + tail_cap
        dev = torch.device(device)
        self.k = torch.zeros((C, Hkv, self.row_cap, d), dtype=torch.bfloat16, device=dev)
        self.vt = torch.zeros((C, Hkv, d, self.row_cap), dtype=torch.bfloat16, device=dev)
        self.head = torch.zeros((C, V), dtype=torch.int32, device=dev)
        self.sync = torch.zeros((C, V), dtype=torch.int32, device=dev)
        self.rope = torch.empty((self.rope_len, d // 2, 2), dtype=torch.float32, device=dev)
        self.status = torch.zeros((1,), dtype=torch.int32, device=dev)
        self.wait_ns = int(wait_ns)
        self.rope_mode = 0 if mrope is None else 1
        with torch.cuda.device(dev):
            if mrope is None:
                skv_build_rope_table(self.rope, self.theta)
            else:
                skv_build_mrope_table(self.rope, self.theta, P, V, F, T, mrope[0], mrope[1])

    @property
    def n_visual(self):
        return self.P + self.V * self.F * self.T

    def desc(self) -> skv_cache:
        return skv_cache(self.C, self.V, self.F, self.T, self.P, self.tail_cap, self.Hkv, self.d,
                         self.row_cap, self.rope_len, self.k.data_ptr(), self.vt.data_ptr(),
                         self.head.data_ptr(), self.sync.data_ptr(), self.rope.data_ptr(),
                         self.status.data_ptr(), self.wait_ns, self.rope_mode, 0)

    def device_status(self) -> int:
        return int(self.status.item())


def kv_write_rows(cache: StreamCache, row0: int, k_src: torch.Tensor, v_src: torch.Tensor):
    n = k_src.shape[1]
    shp = (cache.C, n, cache.Hkv, cache.d)
    _need(k_src, shp, torch.bfloat16, "k_src")
    _need(v_src, shp, torch.bfloat16, "v_src")
    d = cache.desc()
    _check(lib().kv_write_rows(ctypes.byref(d), row0, n, _ptr(k_src), _ptr(v_src), _stream()),
           "kv_write_rows")


def kv_stream_insert(cache: StreamCache, k_new: torch.Tensor, v_new: torch.Tensor):
    shp = (cache.C, cache.V, cache.T, cache.Hkv, cache.d)
    _need(k_new, shp, torch.bfloat16, "k_new")
    _need(v_new, shp, torch.bfloat16, "v_new")
    d = cache.desc()
    _check(lib().kv_stream_insert(ctypes.byref(d), _ptr(k_new), _ptr(v_new), _stream()),
           "kv_stream_insert")


def kv_stream_insert_noalloc(cache: StreamCache, k_new: torch.Tensor, v_new: torch.Tensor):
    """kv_stream_insert without caller scratch: for callers that may not
    allocate device memory, the insert's counters live in a fixed static
    device array inside the library (cache.sync is not used)."""
    shp = (cache.C, cache.V, cache.T, cache.Hkv, cache.d)
    _need(k_new, shp, torch.bfloat16, "k_new")
    _need(v_new, shp, torch.bfloat16, "v_new")
    d = cache.desc()
    d.sync = None
    _check(lib().kv_stream_insert_noalloc(ctypes.byref(d), _ptr(k_new), _ptr(v_new), _stream()),
           "kv_stream_insert_noalloc")


def stream_attn_prefill(cache: StreamCache, q_new: torch.Tensor, sm_scale: float,
                        out: torch.Tensor | None = None, lse: torch.Tensor | bool | None = None):
    """Returns out (and lse when asked for) for the new-frame queries."""
    C, nq, Hq, d = q_new.shape
    _need(q_new, (cache.C, cache.V * cache.T, Hq, cache.d), torch.bfloat16, "q_new")
    if out is None:
        out = torch.empty_like(q_new)
    _need(out, q_new.shape, torch.bfloat16, "out")
    if lse is True:
        lse = torch.empty((C, Hq, nq), dtype=torch.float32, device=q_new.device)
    if isinstance(lse, torch.Tensor):
        _need(lse, (C, Hq, nq), torch.float32, "lse")
    else:
        lse = None
    dd = cache.desc()
    _check(lib().stream_attn_prefill(ctypes.byref(dd), Hq, _ptr(q_new), _ptr(out), _ptr(lse),
                                     float(sm_scale), _stream()), "stream_attn_prefill")
    return (out, lse) if lse is not None else out


def stream_attn_prefill_insert(cache: StreamCache, k_new: torch.Tensor, v_new: torch.Tensor,
                               q_new: torch.Tensor, sm_scale: float, out: torch.Tensor | None = None,
                               lse: torch.Tensor | bool | None = None):
    """kv_stream_insert(k_new, v_new) then stream_attn_prefill(q_new) as one
    call (one kernel where the geometry allows).  Returns out (and lse when
    asked for)."""
    shp = (cache.C, cache.V, cache.T, cache.Hkv, cache.d)
    _need(k_new, shp, torch.bfloat16, "k_new")
    _need(v_new, shp, torch.bfloat16, "v_new")
    C, nq, Hq, d = q_new.shape
    _need(q_new, (cache.C, cache.V * cache.T, Hq, cache.d), torch.bfloat16, "q_new")
    if out is None:
        out = torch.empty_like(q_new)
    _need(out, q_new.shape, torch.bfloat16, "out")
    lse = _lse_arg(lse, C, Hq, nq, q_new.device)
    dd = cache.desc()
    _check(lib().stream_attn_prefill_insert(ctypes.byref(dd), Hq, _ptr(k_new), _ptr(v_new), _ptr(q_new),
                                            _ptr(out), _ptr(lse), float(sm_scale), _stream()),
           "stream_attn_prefill_insert")
    return (out, lse) if lse is not None else out


def _lse_arg(lse, C, Hq, n, device):
    if lse is True:
        lse = torch.empty((C, Hq, n), dtype=torch.float32, device=device)
    if isinstance(lse, torch.Tensor):
        _need(lse, (C, Hq, n), torch.float32, "lse")
        return lse
    return None


def stream_attn_prefill_tail(cache: StreamCache, tail_len: torch.Tensor, q_tail: torch.Tensor,
                             k_tail: torch.Tensor, v_tail: torch.Tensor, sm_scale: float,
                             out: torch.Tensor | None = None,
                             lse: torch.Tensor | bool | None = None):
    """Writes the tokens' K/V after tail_len[c] tail rows and returns their
    attention output (and lse when asked for).  The caller advances
    tail_len by the number of tokens."""
    C, n, Hq, d = q_tail.shape
    _need(q_tail, (cache.C, n, Hq, cache.d), torch.bfloat16, "q_tail")
    _need(k_tail, (cache.C, n, cache.Hkv, cache.d), torch.bfloat16, "k_tail")
    _need(v_tail, (cache.C, n, cache.Hkv, cache.d), torch.bfloat16, "v_tail")
    _need(tail_len, (cache.C,), torch.int32, "tail_len")
    if out is None:
        out = torch.empty_like(q_tail)
    _need(out, q_tail.shape, torch.bfloat16, "out")
    lse = _lse_arg(lse, C, Hq, n, q_tail.device)
    dd = cache.desc()
    _check(lib().stream_attn_prefill_tail(ctypes.byref(dd), Hq, n, _ptr(tail_len), _ptr(q_tail),
                                          _ptr(k_tail), _ptr(v_tail), _ptr(out), _ptr(lse),
                                          float(sm_scale), _stream()), "stream_attn_prefill_tail")
    return (out, lse) if lse is not None else out


def stream_attn_window(cache: StreamCache, q_win: torch.Tensor, sm_scale: float,
                       out: torch.Tensor | None = None, lse: torch.Tensor | bool | None = None):
    """Every window token as a query (logical order: prefix, then each view's
    frames oldest to newest).  Returns out (and lse when asked for)."""
    C, n, Hq, d = q_win.shape
    _need(q_win, (cache.C, cache.n_visual, Hq, cache.d), torch.bfloat16, "q_win")
    if out is None:
        out = torch.empty_like(q_win)
    _need(out, q_win.shape, torch.bfloat16, "out")
    lse = _lse_arg(lse, C, Hq, n, q_win.device)
    dd = cache.desc()
    _check(lib().stream_attn_window(ctypes.byref(dd), Hq, _ptr(q_win), _ptr(out), _ptr(lse),
                                    float(sm_scale), _stream()), "stream_attn_window")
    return (out, lse) if lse is not None else out


def skv_verify_workspace_bytes(cache: StreamCache, n_q_head: int, blk: int) -> int:
    d = cache.desc()
    return int(lib().skv_verify_workspace_bytes(ctypes.byref(d), n_q_head, blk))


def verify_workspace(cache: StreamCache, n_q_head: int, blk: int) -> torch.Tensor:
    """A zero-filled workspace for stream_attn_verify."""
    n = max(16, skv_verify_workspace_bytes(cache, n_q_head, blk))
    return torch.zeros((n,), dtype=torch.uint8, device=cache.k.device)


def stream_attn_verify(cache: StreamCache, tail_len: torch.Tensor, q_blk: torch.Tensor,
                       k_blk: torch.Tensor, v_blk: torch.Tensor, sm_scale: float,
                       target_ids: torch.Tensor | None = None, draft_ids: torch.Tensor | None = None,
                       ws: torch.Tensor | None = None, out: torch.Tensor | None = None,
                       accept_len: torch.Tensor | None = None, next_token: torch.Tensor | None = None):
    """One verify pass.  Returns (out, accept_len, next_token); the last two
    are None when no ids are given."""
    C, blk, Hq, d = q_blk.shape
    _need(q_blk, (cache.C, blk, Hq, cache.d), torch.bfloat16, "q_blk")
    _need(k_blk, (cache.C, blk, cache.Hkv, cache.d), torch.bfloat16, "k_blk")
    _need(v_blk, (cache.C, blk, cache.Hkv, cache.d), torch.bfloat16, "v_blk")
    _need(tail_len, (cache.C,), torch.int32, "tail_len")
    if out is None:
        out = torch.empty_like(q_blk)
    _need(out, q_blk.shape, torch.bfloat16, "out")
    ids = target_ids is not None and draft_ids is not None
    if ids:
        _need(target_ids, (cache.C, blk), torch.int32, "target_ids")
        _need(draft_ids, (cache.C, blk), torch.int32, "draft_ids")
        if accept_len is None:
            accept_len = torch.empty((cache.C,), dtype=torch.int32, device=q_blk.device)
        if next_token is None:
            next_token = torch.empty((cache.C,), dtype=torch.int32, device=q_blk.device)
        _need(accept_len, (cache.C,), torch.int32, "accept_len")
        _need(next_token, (cache.C,), torch.int32, "next_token")
    if ws is None:
        ws = verify_workspace(cache, Hq, blk)
    dd = cache.desc()
    _check(lib().stream_attn_verify(
        ctypes.byref(dd), Hq, blk, _ptr(tail_len), _ptr(q_blk), _ptr(k_blk), _ptr(v_blk), _ptr(out),
        _ptr(target_ids) if ids else None, _ptr(draft_ids) if ids else None,
        _ptr(accept_len) if ids else None, _ptr(next_token) if ids else None,
        _ptr(ws), ws.numel(), float(sm_scale), _stream()), "stream_attn_verify")
    return out, (accept_len if ids else None), (next_token if ids else None)


# --------------------------------------------- paged cache, cross attention


def _on(t, shape, dtype, name, dev):
    """_need, and the tensor lives on device dev, where the call launches.
    A decode step makes many small calls, so what a good tensor has to pass
    is one short expression."""
    if not (type(t) is _Tensor and t.dtype is dtype and t.shape == shape and t.get_device() == dev
            and t.is_contiguous()):
        _need(t, shape, dtype, name)
        _on_dev(t.get_device(), name, dev)


def _on_dev(index, name, dev):
    if index != dev:
        raise ValueError("%s is on cuda:%d, but the current device is cuda:%d" % (name, index, dev))


def _call_device(t, name):
    """The device that a call on t launches on: t's, and the current one."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be on a CUDA device" % name)
    dev = torch._C._cuda_getDevice()   # torch.cuda.current_device() once CUDA is up, as t shows
    _on_dev(t.get_device(), name, dev)
    return dev


def _raw_stream(dev):
    """The current torch stream of device dev, without making a Stream object."""
    return torch._C._cuda_getCurrentRawStream(dev)


def _rows(t, heads, d, dtype, name, dev):
    """(tokens, heads, token stride) of a token-major tensor [tokens][heads][d]
    whose heads of a token are adjacent (a part of a wider projection's rows,
    say); heads None: any number."""
    if type(t) is not _Tensor and not isinstance(t, _Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    stride = t.stride()
    if len(stride) == 3:
        n, h, width = t.shape
    if len(stride) != 3 or width != d or (heads is not None and h != heads):
        raise ValueError("%s must have shape (tokens, %s, %d), got %s" % (name, "heads" if heads is None else heads, d, tuple(t.shape)))
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError("%s must be on a CUDA device" % name)
        _on_dev(t.get_device(), name, dev)
    s0, s1, s2 = stride
    if n and (s2 != 1 or (s1 != d and h > 1)):
        raise ValueError("%s must have its heads adjacent within a token" % name)
    return n, h, s0 if n > 1 else h * d


class PagedPlan:
    """The plan of one step (see kv_paged_plan in include/skv.h): int32
    tensors q_start [n_req + 1], kv_len [n_req], next_state [n_req + 2],
    position [n_tok] and slot [n_tok], which stay where they are."""

    __slots__ = ("_t", "_args", "n_req", "n_tok", "_dev")

    def __init__(self, q_start, kv_len, next_state, position, slot):
        self._t = (q_start, kv_len, next_state, position, slot)
        n_req, n_tok = kv_len.numel(), slot.numel()
        for t, n, name in zip(self._t, (n_req + 1, n_req, n_req + 2, n_tok, n_tok),
                              ("q_start", "kv_len", "next_state", "position", "slot")):
            _need(t, (n,), torch.int32, name)
            _on_dev(t.get_device(), name, q_start.get_device())
        self.n_req, self.n_tok, self._dev = n_req, n_tok, q_start.get_device()
        self._args = tuple(ctypes.c_void_p(t.data_ptr()) for t in self._t)

    q_start = property(lambda self: self._t[0])
    kv_len = property(lambda self: self._t[1])
    next_state = property(lambda self: self._t[2])
    position = property(lambda self: self._t[3])
    slot = property(lambda self: self._t[4])

    @classmethod
    def empty(cls, n_req, n_tok, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.empty(n_req + 1, **i32), torch.empty(n_req, **i32), torch.empty(n_req + 2, **i32),
                   torch.empty(n_tok, **i32), torch.empty(n_tok, **i32))


class PagedCache:
    """A pool of pages for requests of different lengths, in device memory.

    Tensors (owned by this object; they stay where they are for its life):
      k, v         bf16 or fp16 [n_page][Hkv][page_size][d], per layer
      block_table  int32 [n_req][max_block]  pages of each request
      page_queue   int32 [n_page]            ring of free pages
      state        int32 [n_req + 2]         tokens held per request, queue head and count
      rope         fp32 [rope_len][d/2][2]   (cos, sin) table, or None
      status       int32 [1]                 device status bits

    theta gives the rope table of positions below max_block * page_size
    (None: keys and queries are not rotated).  The layers of a model share
    everything but k and v: layer(i) is the cache of one of them.  wait_ns
    limits every wait inside paged_attn (0: two seconds) and may be set later;
    everything else is fixed, because the calls keep its addresses.
    """

    def __setattr__(self, name, value):
        if "_made" in self.__dict__ and name in self.__dict__:
            raise AttributeError("%s of a PagedCache is fixed: write into it, or make another cache" % name)
        object.__setattr__(self, name, value)

    def __init__(self, n_page, page_size, Hkv, d, n_req, max_block, theta=None, dtype=torch.bfloat16,
                 n_layer=1, device="cuda", wait_ns=0):
        dev = torch.device(device)
        shape = (n_layer, n_page, Hkv, page_size, d)
        i32 = dict(dtype=torch.int32, device=dev)
        rope = None
        if theta is not None:
            rope = torch.empty((max_block * page_size, d // 2, 2), dtype=torch.float32, device=dev)
            with torch.cuda.device(dev):
                skv_build_rope_table(rope, theta)
        state = torch.zeros((n_req + 2,), **i32)
        state[-1] = n_page
        self._k, self._v = (torch.empty(shape, dtype=dtype, device=dev) for _ in range(2))
        self._set(self._k[0], self._v[0], torch.zeros((n_req, max_block), **i32),
                  torch.arange(n_page, **i32), state, rope, torch.zeros((1,), **i32), page_size)
        self.wait_ns = wait_ns

    @classmethod
    def wrap(cls, k=None, v=None, block_table=None, page_queue=None, state=None, rope=None, status=None,
             page_size=None, wait_ns=0):
        """A cache over tensors that the caller owns.  k and v may be left
        out where only kv_paged_plan is called, page_queue and state where it
        is not; status is made where it is not given."""
        self = cls.__new__(cls)
        if block_table is None:
            raise ValueError("block_table must be a (requests, max_block) tensor")
        if status is None:
            status = torch.zeros((1,), dtype=torch.int32, device=block_table.device)
        self._k = k[None] if k is not None else None
        self._v = v[None] if v is not None else None
        self._set(k, v, block_table, page_queue, state, rope, status, page_size)
        self.wait_ns = wait_ns
        return self

    def _set(self, k, v, block_table, page_queue, state, rope, status, page_size):
        if (k is None) != (v is None):
            raise ValueError("k and v come together")
        if k is None and (page_queue is None or page_size is None):
            raise ValueError("a cache without k and v needs page_queue and page_size")
        if block_table is None or block_table.dim() != 2:
            raise ValueError("block_table must be a (requests, max_block) tensor")
        _need(block_table, block_table.shape, torch.int32, "block_table")
        _need(status, (1,), torch.int32, "status")
        hkv = d = code = 0
        if k is not None:
            if k.dim() != 4:
                raise ValueError("k must have shape (pages, kv heads, page_size, d), got %s" % (tuple(k.shape),))
            if k.dtype not in _DTYPE_CODE:
                raise TypeError("k must be bfloat16 or float16, got %s" % k.dtype)
            if page_size is not None and page_size != k.shape[2]:
                raise ValueError("page_size %d, but k has pages of %d" % (page_size, k.shape[2]))
            _need(k, k.shape, k.dtype, "k")
            _need(v, k.shape, k.dtype, "v")
            (n_page, hkv, page_size, d), code = k.shape, _DTYPE_CODE[k.dtype]
        else:
            n_page = page_queue.numel()
        if page_queue is not None:
            _need(page_queue, (n_page,), torch.int32, "page_queue")
        if state is not None:
            _need(state, (block_table.shape[0] + 2,), torch.int32, "state")
        if rope is not None:
            _need(rope, (rope.shape[0], d // 2, 2), torch.float32, "rope table")
        for name, t in (("k", k), ("v", v), ("page_queue", page_queue), ("state", state), ("rope", rope),
                        ("status", status)):
            if t is not None and t.device != block_table.device:
                raise ValueError("%s is on %s, block_table on %s" % (name, t.device, block_table.device))
        n_req, max_block = block_table.shape
        ptr = lambda t: t.data_ptr() if t is not None else None  # noqa: E731
        desc = skv_paged(n_page, page_size, hkv, d, code, rope.shape[0] if rope is not None else 0, max_block, 0,
                         ptr(k), ptr(v), ptr(block_table), ptr(rope), ptr(status))
        # all at once, past __setattr__: a step may make a cache per layer
        self.__dict__.update(
            k=k, v=v, block_table=block_table, page_queue=page_queue, state=state, rope=rope, status=status,
            n_page=n_page, page_size=page_size, Hkv=hkv, d=d, n_req=n_req, max_block=max_block,
            _state_arg=ctypes.c_void_p(ptr(state)), _queue_arg=ctypes.c_void_p(ptr(page_queue)),
            _desc=desc, _ref=ctypes.byref(desc), _dev=block_table.get_device(),
            _dtype=k.dtype if k is not None else None, _made=True)

    def layer(self, i: int) -> "PagedCache":
        """The cache of layer i: its own k and v, everything else shared."""
        if self._k is None:
            raise ValueError("the cache has no k and v")
        if i < 0:
            i = range(len(self._k))[i]
        c = PagedCache.__new__(PagedCache)
        c.__dict__.update(_k=self._k[i:i + 1], _v=self._v[i:i + 1])
        c._set(self._k[i], self._v[i], self.block_table, self.page_queue, self.state, self.rope, self.status,
               self.page_size)
        c._desc.wait_ns = self._desc.wait_ns
        return c

    @property
    def wait_ns(self) -> int:
        return self._desc.wait_ns

    @wait_ns.setter
    def wait_ns(self, ns):
        self._desc.wait_ns = int(ns)

    def advance(self, plan: PagedPlan):
        """Take the state that a plan leads to as the cache's state."""
        self.state.copy_(plan.next_state)

    def device_status(self) -> int:
        return int(self.status.item())


def kv_paged_plan(cache: PagedCache, new_len: torch.Tensor, n_tok: int,
                  plan: PagedPlan | None = None) -> PagedPlan:
    """The pages, tables and slot maps of one step: new_len[b] new tokens for
    request b (-1: it has finished), packed into n_tok token rows.  The
    cache's state stays until cache.advance(plan)."""
    if cache.state is None or cache.page_queue is None:
        raise ValueError("the cache has no state and page_queue to plan with")
    n_req, dev = cache.n_req, _call_device(new_len, "new_len")
    _on_dev(cache._dev, "the cache", dev)
    _on(new_len, (n_req,), torch.int32, "new_len", dev)
    if plan is None:
        plan = PagedPlan.empty(n_req, n_tok, new_len.device)
    if plan.n_req != n_req or plan.n_tok != n_tok:
        raise ValueError("the plan is for %d requests and %d tokens, not %d and %d" % (plan.n_req, plan.n_tok, n_req, n_tok))
    _on_dev(plan._dev, "the plan", dev)
    rc = lib().kv_paged_plan(cache._ref, n_req, n_tok, cache._state_arg, new_len.data_ptr(), cache._queue_arg,
                             *plan._args, _raw_stream(dev))
    if rc:
        _check(rc, "kv_paged_plan")
    return plan


def _need_pages(cache, dev):
    if cache.k is None:
        raise ValueError("the cache has no k and v")
    _on_dev(cache._dev, "the cache", dev)


def kv_paged_write(cache: PagedCache, q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor,
                   position: torch.Tensor | None, slot: torch.Tensor,
                   q_out: torch.Tensor | None = None) -> torch.Tensor | None:
    """A step's k (rotated) and v into the cache's pages; returns q rotated
    (None for q None).  q, k and v are token-major and may be parts of one
    projection's output."""
    dev = _call_device(k, "k")
    _need_pages(cache, dev)
    hkv, d, dt = cache.Hkv, cache.d, cache._dtype
    n, _, ks = _rows(k, hkv, d, dt, "k", dev)
    nv, _, vs = _rows(v, hkv, d, dt, "v", dev)
    if nv != n:
        raise ValueError("k has %d tokens, v %d" % (n, nv))
    _on(slot, (n,), torch.int32, "slot", dev)
    if cache.rope is not None or position is not None:
        _on(position, (n,), torch.int32, "position", dev)
    hq = qs = 0
    if q is not None:
        nq, hq, qs = _rows(q, None, d, dt, "q", dev)
        if nq != n:
            raise ValueError("k has %d tokens, q %d" % (n, nq))
        if q_out is None:
            q_out = torch.empty((n, hq, d), dtype=dt, device=q.device)
        else:
            _on(q_out, (n, hq, d), dt, "q_out", dev)
    elif q_out is not None:
        raise ValueError("q_out without q")
    rc = lib().kv_paged_write(cache._ref, hq, n, q.data_ptr() if q is not None else None, qs, k.data_ptr(), ks,
                              v.data_ptr(), vs, position.data_ptr() if position is not None else None,
                              slot.data_ptr(), q_out.data_ptr() if q is not None else None, _raw_stream(dev))
    if rc:
        _check(rc, "kv_paged_write")
    return q_out


def attn_workspace(device="cuda") -> torch.Tensor:
    """A workspace for paged_attn and cross_attn (any shape)."""
    with torch.cuda.device(torch.device(device)):
        return torch.empty((int(lib().skv_attn_workspace_bytes()),), dtype=torch.uint8, device=device)


def _attn_args(q, n_req, q_start, out, lse, ws, dev):
    n, hq, d = q.shape
    _on(q_start, (n_req + 1,), torch.int32, "q_start", dev)
    if out is None:
        out = torch.empty((n, hq, d), dtype=q.dtype, device=q.device)
    else:
        _on(out, (n, hq, d), q.dtype, "out", dev)
    if lse is True:
        lse = torch.empty((hq, n), dtype=torch.float32, device=q.device)
    elif isinstance(lse, torch.Tensor):
        _on(lse, (hq, n), torch.float32, "lse", dev)
    elif lse is not None and lse is not False:
        raise TypeError("lse must be a torch.Tensor, a bool or None")
    else:
        lse = None
    if ws is None:
        ws = attn_workspace(q.device)
    elif not isinstance(ws, torch.Tensor):
        raise TypeError("ws must be a torch.Tensor")
    else:
        _on(ws, (ws.numel(),), torch.uint8, "ws", dev)
    return out, lse, ws


def paged_attn(cache: PagedCache, q: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor,
               sm_scale: float, out: torch.Tensor | None = None, lse: torch.Tensor | bool | None = None,
               ws: torch.Tensor | None = None):
    """Attention of each request's new tokens over its pages (chunks and
    single tokens together).  q is rotated already (kv_paged_write).  Returns
    out (and lse [Hq][tokens] when asked for)."""
    dev = _call_device(q, "q")
    _need_pages(cache, dev)
    n_req = cache.n_req
    n, hq, qs = _rows(q, None, cache.d, cache._dtype, "q", dev)
    _on(kv_len, (n_req,), torch.int32, "kv_len", dev)
    out, lse, ws = _attn_args(q, n_req, q_start, out, lse, ws, dev)
    rc = lib().paged_attn(cache._ref, hq, n_req, n, q.data_ptr(), qs, q_start.data_ptr(), kv_len.data_ptr(),
                          out.data_ptr(), lse.data_ptr() if lse is not None else None, ws.data_ptr(), ws.numel(),
                          sm_scale, _raw_stream(dev))
    if rc:
        _check(rc, "paged_attn")
    return (out, lse) if lse is not None else out


def cross_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_start: torch.Tensor, k_start: torch.Tensor,
               k_len: torch.Tensor, sm_scale: float, *, status: torch.Tensor, out: torch.Tensor | None = None,
               lse: torch.Tensor | bool | None = None, ws: torch.Tensor | None = None, wait_ns: int = 0):
    """Attention of packed queries to each request's packed states k, v
    [tokens][Hkv][d]: request b reads rows [k_start[b], k_start[b] + k_len[b]).
    status collects device status bits; wait_ns limits every wait inside the
    kernel (0: two seconds).  Returns out (and lse when asked for)."""
    dev = _call_device(k, "k")
    if k.dim() != 3 or k.dtype not in _DTYPE_CODE:
        raise ValueError("k must be a bfloat16 or float16 tensor (tokens, kv heads, d), got %s %s" % (k.dtype, tuple(k.shape)))
    dt, d = k.dtype, k.shape[2]
    n_key, hkv, ks = _rows(k, None, d, dt, "k", dev)
    nv, _, vs = _rows(v, hkv, d, dt, "v", dev)
    if nv != n_key:
        raise ValueError("k has %d tokens, v %d" % (n_key, nv))
    n, hq, qs = _rows(q, None, d, dt, "q", dev)
    if not isinstance(k_start, torch.Tensor):
        raise TypeError("k_start must be a torch.Tensor")
    n_req = k_start.numel()
    _on(k_start, (n_req,), torch.int32, "k_start", dev)
    _on(k_len, (n_req,), torch.int32, "k_len", dev)
    _on(status, (1,), torch.int32, "status", dev)
    out, lse, ws = _attn_args(q, n_req, q_start, out, lse, ws, dev)
    desc = skv_states(n_key, hkv, d, _DTYPE_CODE[dt], ks, vs, k.data_ptr(), v.data_ptr(), k_start.data_ptr(),
                      k_len.data_ptr(), status.data_ptr(), wait_ns)
    rc = lib().cross_attn(ctypes.byref(desc), hq, n_req, n, q.data_ptr(), qs, q_start.data_ptr(),
                          out.data_ptr(), lse.data_ptr() if lse is not None else None, ws.data_ptr(), ws.numel(),
                          sm_scale, _raw_stream(dev))
    if rc:
        _check(rc, "cross_attn")
    return (out, lse) if lse is not None else out
