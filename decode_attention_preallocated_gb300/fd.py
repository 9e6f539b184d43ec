"""Python binding of libfd.so (the C ABI in include/fd.h): ctypes, and for the
4-bit cache and page calls the extension in csrc/fd_torch.cpp.

Argument marshalling only: every step of the computation runs in the CUDA
kernels inside libfd.so.  PyTorch supplies device memory and the current
stream.  There is no fallback: if libfd.so (or
the extension) is missing or cannot be loaded, every call raises.

Low-level names mirror the C ABI (``fd_decode``, ``fd_decode_int8``,
``fd_decode_append``, ``fd_decode_paged``, ``fd_decode_masked``,
``fd_decode_gather``, ``fd_decode_gather_int8``, ``fd_decode_gather_bias``,
``fd_topk_blocks``, ``fd_decode_fp4``, ``fd_append_fp4``, ``fd_read_fp4``,
``fd_pages_reserve`` / ``_fork`` / ``_free`` / ``_compact`` / ``_copy``,
``fd_workspace_create`` ...) and take ``FdTensor`` / ``FdOpts`` structures;
``decode``, ``decode_int8``, ``decode_append``, ``decode_paged``,
``decode_masked``, ``decode_gather``, ``topk_blocks``, ``decode_fp4``,
``append_fp4``, ``read_fp4``, ``pages_reserve``, ``pages_fork``,
``pages_free``, ``pages_compact`` and ``pages_copy`` take
torch tensors, allocate ``out`` with torch when it is not given, and keep one
workspace per (device, stream).
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os
import struct
import threading
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfd.so")
NATIVE_PATH = os.path.join(_HERE, "_fd_torch.so")

# constants from include/fd.h
FD_OK, FD_ERR_ARG, FD_ERR_UNSUPPORTED, FD_ERR_ALIGN, FD_ERR_WORKSPACE, FD_ERR_CUDA = 0, -1, -2, -3, -4, -5
FD_ERR_SCRATCH = -6
FD_BF16, FD_F32, FD_I8, FD_I32, FD_U8, FD_E4M3 = 0, 1, 2, 3, 4, 5
FD_DEV_BAD_LENGTH, FD_DEV_BAD_INDEX, FD_DEV_INTERNAL, FD_DEV_NO_PAGES = 1, 2, 4, 8
FD_KERNEL_AUTO, FD_KERNEL_SIMT, FD_KERNEL_TC = 0, 1, 2
FD_MAX_ROWS = 64

_DTYPES = {torch.bfloat16: FD_BF16, torch.float32: FD_F32, torch.int8: FD_I8,
           torch.int32: FD_I32, torch.uint8: FD_U8, torch.float8_e4m3fn: FD_E4M3}


class FdTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("ndim", ctypes.c_int32), ("shape", ctypes.c_int64 * 4),
                ("stride", ctypes.c_int64 * 4)]


class FdOpts(ctypes.Structure):
    _fields_ = [("stream", ctypes.c_void_p), ("ws", ctypes.c_void_p),
                ("num_ctas", ctypes.c_int32), ("kernel", ctypes.c_int32),
                ("scale", ctypes.c_float), ("wait_limit_us", ctypes.c_int32),
                ("reserved", ctypes.c_int32 * 2)]


class FdError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__("%s failed: %s (%d)" % (what, status_string(code), code))


_lib = None
_lib_lock = threading.Lock()

# (name, restype, argtypes) for every symbol declared in include/fd.h
_P = ctypes.POINTER
_SIGNATURES = [
    ("fd_decode", ctypes.c_int,
     [_P(FdTensor), _P(FdTensor), _P(FdTensor), ctypes.c_void_p, ctypes.c_int32,
      ctypes.c_int32, ctypes.c_float, _P(FdTensor), _P(FdOpts)]),
    ("fd_decode_int8", ctypes.c_int,
     [_P(FdTensor), _P(FdTensor), _P(FdTensor), _P(FdTensor), _P(FdTensor),
      ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_float,
      _P(FdTensor), _P(FdOpts)]),
    ("fd_decode_gather", ctypes.c_int,
     [_P(FdTensor), _P(FdTensor), _P(FdTensor), ctypes.c_void_p, ctypes.c_int32,
      _P(FdTensor), _P(FdOpts)]),
    ("fd_decode_gather_int8", ctypes.c_int,
     [_P(FdTensor), _P(FdTensor), _P(FdTensor), _P(FdTensor), _P(FdTensor), ctypes.c_void_p,
      ctypes.c_int32, _P(FdTensor), _P(FdOpts)]),
    ("fd_topk_blocks", ctypes.c_int,
     [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
      ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]),
    ("fd_decode_gather_bias", ctypes.c_int,
     [_P(FdTensor), _P(FdTensor), _P(FdTensor), ctypes.c_void_p, ctypes.c_void_p,
      ctypes.c_int32, _P(FdTensor), _P(FdOpts)]),
    ("fd_decode_masked", ctypes.c_int,
     [_P(FdTensor), _P(FdTensor), _P(FdTensor), ctypes.c_void_p, _P(FdTensor), ctypes.c_int32,
      ctypes.c_int32, ctypes.c_float, _P(FdTensor), _P(FdOpts)]),
    ("fd_decode_append", ctypes.c_int,
     [_P(FdTensor), _P(FdTensor), _P(FdTensor), _P(FdTensor), _P(FdTensor),
      ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_float, _P(FdTensor),
      _P(FdOpts)]),
    ("fd_decode_paged", ctypes.c_int,
     [_P(FdTensor), _P(FdTensor), _P(FdTensor), _P(FdTensor), _P(FdTensor),
      ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
      ctypes.c_float, _P(FdTensor), _P(FdOpts)]),
    ("fd_decode_noalloc", ctypes.c_int,
     [_P(FdTensor), _P(FdTensor), _P(FdTensor), ctypes.c_void_p, ctypes.c_int32,
      ctypes.c_int32, ctypes.c_float, _P(FdTensor), ctypes.c_void_p, ctypes.c_int32]),
    # the 4-bit cache and the page calls are called through the marshalling
    # extension; here they take descriptors as bytes or any pointer
    ("fd_decode_fp4", ctypes.c_int,
     [ctypes.c_void_p] * 5 + [ctypes.c_float, ctypes.c_float, ctypes.c_void_p, ctypes.c_int32,
                              ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_float,
                              ctypes.c_void_p, ctypes.c_void_p]),
    ("fd_append_fp4", ctypes.c_int,
     [ctypes.c_void_p] * 7 + [ctypes.c_float, ctypes.c_float, ctypes.c_void_p, ctypes.c_int32,
                              ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    ("fd_read_fp4", ctypes.c_int,
     [ctypes.c_void_p] * 4 + [ctypes.c_float, ctypes.c_float, ctypes.c_void_p, ctypes.c_int32]
     + [ctypes.c_void_p] * 5),
    ("fd_pages_scratch_bytes", ctypes.c_size_t, [ctypes.c_int64]),
    ("fd_pages_reserve", ctypes.c_int,
     [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
      ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
      ctypes.c_void_p, ctypes.c_void_p]),
    ("fd_pages_fork", ctypes.c_int,
     [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
      ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
      ctypes.c_int32, ctypes.c_void_p]),
    ("fd_pages_free", ctypes.c_int,
     [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
      ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
      ctypes.c_void_p]),
    ("fd_pages_compact", ctypes.c_int,
     [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    ("fd_pages_copy", ctypes.c_int,
     [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
      ctypes.c_void_p]),
    ("fd_workspace_bytes", ctypes.c_size_t,
     [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]),
    ("fd_workspace_create", ctypes.c_int,
     [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
      ctypes.c_void_p, _P(ctypes.c_void_p)]),
    ("fd_workspace_reset", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    ("fd_workspace_fill_counters", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]),
    ("fd_workspace_destroy", ctypes.c_int, [ctypes.c_void_p]),
    ("fd_get_device_status", ctypes.c_int, [ctypes.c_void_p, _P(ctypes.c_int32)]),
    ("fd_get_device_diagnostics", ctypes.c_int, [ctypes.c_void_p, _P(ctypes.c_int32)]),
    ("fd_auto_num_ctas", ctypes.c_int32,
     [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int64]),
    ("fd_tile_tokens", ctypes.c_int32, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]),
    ("fd_masked_list_bytes", ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    ("fd_plan", ctypes.c_int64,
     [_P(ctypes.c_int64), ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
      _P(ctypes.c_int32), _P(ctypes.c_int32)]),
    ("fd_seg_units", ctypes.c_int32, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]),
    ("fd_status_string", ctypes.c_char_p, [ctypes.c_int]),
    ("fd_version", ctypes.c_int32, []),
]


def lib() -> ctypes.CDLL:
    """Load libfd.so (raises if it has not been built)."""
    global _lib
    with _lib_lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    "libfd.so is not built (%s); run "
                    "decode_attention_preallocated_gb300.build.build()" % LIB_PATH)
            h = ctypes.CDLL(LIB_PATH)
            for name, res, args in _SIGNATURES:
                fn = getattr(h, name)
                fn.restype = res
                fn.argtypes = args
            _lib = h
    return _lib


def status_string(code: int) -> str:
    return lib().fd_status_string(int(code)).decode()


# ------------------------------------------------------------- marshalling
def as_fd_tensor(t: torch.Tensor) -> FdTensor:
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError("unsupported dtype %s" % t.dtype)
    shape = t.shape
    n = len(shape)
    if n > 4:
        raise ValueError("at most 4 dimensions")
    ft = FdTensor()
    ft.data = t.data_ptr()
    ft.dtype = dt
    ft.ndim = n
    ft.shape[:n] = shape
    ft.stride[:n] = t.stride()
    return ft


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream, device) -> int:
    """Handle of a stream; an int is one already, None the current stream."""
    if isinstance(stream, int):
        return stream
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


class _on_device:
    """Makes `device` current for the C call, unless it already is."""

    __slots__ = ("device", "prev")

    def __init__(self, device):
        self.device = device
        self.prev = None

    def __enter__(self):
        cur = torch.cuda.current_device()
        if cur != self.device.index:
            self.prev = cur
            torch.cuda.set_device(self.device)

    def __exit__(self, *exc):
        if self.prev is not None:
            torch.cuda.set_device(self.prev)
        return False


def _check(code: int, what: str):
    if code != FD_OK:
        raise FdError(code, what)


# -------------------------------------------------------------- workspace
class Workspace:
    """Owns one fd_workspace (device memory allocated by libfd.so).

    Size it for the largest call it will serve; a call that needs more fails
    with FD_ERR_WORKSPACE.  Create it before capturing a CUDA graph.
    """

    def __init__(self, max_segments: int, max_rows: int, head_dim: int,
                 max_ctas: int, stream: Optional[torch.cuda.Stream] = None,
                 device=None):
        self.max_segments, self.max_rows = int(max_segments), int(max_rows)
        self.head_dim, self.max_ctas = int(head_dim), int(max_ctas)
        self.device = torch.device("cuda", torch.cuda.current_device()) \
            if device is None else torch.device(device)
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(lib().fd_workspace_create(self.max_segments, self.max_rows,
                                             self.head_dim, self.max_ctas,
                                             _stream_handle(stream, self.device),
                                             ctypes.byref(h)),
                   "fd_workspace_create")
        self.handle = h

    def fits(self, segments, rows, head_dim, ctas) -> bool:
        return (segments <= self.max_segments and rows <= self.max_rows
                and head_dim <= self.head_dim and ctas <= self.max_ctas)

    def reset(self, stream=None):
        _check(lib().fd_workspace_reset(self.handle, _stream_handle(stream, self.device)),
               "fd_workspace_reset")

    def fill_counters(self, value: int, stream=None):
        """Test hook: every completion counter set to `value` (a negative one
        stands for counters an aborted launch left behind)."""
        _check(lib().fd_workspace_fill_counters(self.handle, int(value),
                                                _stream_handle(stream, self.device)),
               "fd_workspace_fill_counters")

    def device_status(self) -> int:
        st = ctypes.c_int32(0)
        with torch.cuda.device(self.device):
            _check(lib().fd_get_device_status(self.handle, ctypes.byref(st)),
                   "fd_get_device_status")
        return int(st.value)

    def diagnostics(self):
        w = (ctypes.c_int32 * 13)()
        with torch.cuda.device(self.device):
            _check(lib().fd_get_device_diagnostics(self.handle, w), "fd_get_device_diagnostics")
        return list(w)

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            with torch.cuda.device(self.device):
                torch.cuda.synchronize(self.device)
                lib().fd_workspace_destroy(self.handle)
            self.handle = None

    def __del__(self):  # pragma: no cover - best effort at interpreter exit
        try:
            self.close()
        except Exception:
            pass


_ws_cache = {}
_ws_replaced = []
_ws_lock = threading.Lock()


def workspace_for(device, stream_handle, segments, rows, head_dim, ctas) -> Workspace:
    """Workspace shared by calls on one (device, stream); a larger one takes its
    place when needed (making it allocates, so size it up front for graph
    capture).  The smaller one is never destroyed: another thread's call may
    hold it, and a graph captured with it may still be replayed.  What was too
    small at least doubles, so that few of them pile up."""
    key = (torch.device(device).index, int(stream_handle))

    def grown(need, have, most):
        return have if need <= have else max(need, min(2 * have, most))

    with _ws_lock:
        ws = _ws_cache.get(key)
        if ws is None:
            want = dict(max_segments=max(segments, 64), max_rows=max(rows, 16),
                        head_dim=max(head_dim, 256), max_ctas=max(ctas, 1024))
        elif ws.fits(segments, rows, head_dim, ctas):
            return ws
        else:
            want = dict(max_segments=grown(segments, ws.max_segments, 1 << 62),
                        max_rows=grown(rows, ws.max_rows, FD_MAX_ROWS),
                        head_dim=max(head_dim, ws.head_dim),
                        max_ctas=grown(ctas, ws.max_ctas, (1 << 31) - 1))
        # (zeroed on the stream that its calls run on, which may not be the current)
        new = Workspace(device=device, stream=int(stream_handle), **want)
        if ws is not None:
            _ws_replaced.append(ws)
        _ws_cache[key] = new
        return new


def auto_num_ctas(kernel=FD_KERNEL_AUTO, head_dim=128, kv_dtype=FD_BF16, rows=1,
                  max_tiles=0) -> int:
    return int(lib().fd_auto_num_ctas(kernel, head_dim, kv_dtype, rows, max_tiles))


def tile_tokens(kernel=FD_KERNEL_AUTO, head_dim=128, kv_dtype=FD_BF16) -> int:
    return int(lib().fd_tile_tokens(kernel, head_dim, kv_dtype))


def masked_list_bytes(B, cap) -> int:
    """Workspace bytes, past a masked call's split partials, that let the
    tensor-core kernel list the visible chunks before it decodes."""
    return int(lib().fd_masked_list_bytes(int(B), int(cap)))


def slot_floats(rows, head_dim) -> int:
    """Floats of one workspace slot of split partials (O, m and l of rows)."""
    return rows * head_dim + ((2 * rows + 3) // 4) * 4


def plan(seg_len, tile, num_ctas, seg_units=0):
    """Host mirror of the device partitioner: (total work units, first block
    of each segment, number of blocks sharing each segment).  Each non-empty
    segment is charged `seg_units` units before its tiles."""
    n = len(seg_len)
    arr = (ctypes.c_int64 * max(n, 1))(*[int(x) for x in seg_len])
    first = (ctypes.c_int32 * max(n, 1))()
    pieces = (ctypes.c_int32 * max(n, 1))()
    total = lib().fd_plan(arr, n, int(tile), int(num_ctas), int(seg_units), first, pieces)
    if total < 0:
        raise FdError(int(total), "fd_plan")
    return int(total), list(first)[:n], list(pieces)[:n]


def seg_units(kernel, head_dim, kv_dtype=FD_BF16):
    """Work units a launch of `kernel` charges per segment start."""
    return int(lib().fd_seg_units(int(kernel), int(head_dim), int(kv_dtype)))


# ---------------------------------------------------------- torch wrappers
def _opts(stream_handle, ws, num_ctas, kernel, scale=0.0, wait_limit_us=0) -> FdOpts:
    o = FdOpts()
    o.stream = stream_handle
    o.ws = ws.handle
    o.num_ctas = int(num_ctas)
    o.kernel = int(kernel)
    o.scale = float(scale)
    o.wait_limit_us = int(wait_limit_us)
    return o


def _prepare(q, k, out, out_dtype, segments, rows, num_ctas, kernel, stream, ws):
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    device = q.device
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=device)
    sh = _stream_handle(stream, device)
    if ws is None:
        ctas = num_ctas
        if ctas == 0:
            # an upper bound on what either kernel picks for an auto launch
            with torch.cuda.device(device):
                ctas = max(auto_num_ctas(FD_KERNEL_SIMT, q.shape[-1], FD_BF16, rows, 0),
                           auto_num_ctas(FD_KERNEL_TC, q.shape[-1], FD_BF16, rows, 0))
        ws = workspace_for(device, sh, segments, rows, q.shape[-1], max(ctas, 1))
    return out, sh, ws


def decode(q, k_cache, v_cache, kv_lengths, n_q=None, causal=False, scale=None,
           out=None, out_dtype=torch.bfloat16, num_ctas=0, kernel=FD_KERNEL_AUTO,
           stream=None, workspace: Optional[Workspace] = None, wait_limit_us=0):
    """Attention of q [B, n_q, Hq, d] over the first kv_lengths[b] positions of
    k_cache / v_cache [B, Hkv, cap, d] (bf16).  kv_lengths: int32 [B] on the
    device.  Returns out [B, n_q, Hq, d].  wait_limit_us bounds each internal
    wait of the tensor-core kernel (0: 2 s)."""
    B, nq, Hq, d = q.shape
    n_q = nq if n_q is None else n_q
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    Hkv = k_cache.shape[1]
    rows = (Hq // max(Hkv, 1)) * nq
    out, sh, ws = _prepare(q, k_cache, out, out_dtype, B * Hkv, rows, num_ctas,
                           kernel, stream, workspace)
    tq, tk, tv, to = map(as_fd_tensor, (q, k_cache, v_cache, out))
    o = _opts(sh, ws, num_ctas, kernel, wait_limit_us=wait_limit_us)
    with _on_device(q.device):
        rc = lib().fd_decode(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv),
                             kv_lengths.data_ptr(), int(n_q), int(bool(causal)),
                             float(scale), ctypes.byref(to), ctypes.byref(o))
    _check(rc, "fd_decode")
    return out


def decode_int8(q, k_cache, v_cache, k_scale, v_scale, kv_lengths, n_q=None,
                causal=False, scale=None, out=None, out_dtype=torch.bfloat16,
                num_ctas=0, kernel=FD_KERNEL_AUTO, stream=None,
                workspace: Optional[Workspace] = None):
    """As ``decode`` for an int8 cache with fp32 scales [B, Hkv, cap]."""
    B, nq, Hq, d = q.shape
    n_q = nq if n_q is None else n_q
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    Hkv = k_cache.shape[1]
    rows = (Hq // max(Hkv, 1)) * nq
    # more than 32 rows: the tensor-core kernel serves each kv head's query
    # heads in parts, a segment each (at most one per query head)
    segments = B * Hq if rows > 32 else B * Hkv
    out, sh, ws = _prepare(q, k_cache, out, out_dtype, segments, rows, num_ctas,
                           kernel, stream, workspace)
    tq, tk, tv, tks, tvs, to = map(as_fd_tensor, (q, k_cache, v_cache, k_scale, v_scale, out))
    o = _opts(sh, ws, num_ctas, kernel)
    with _on_device(q.device):
        rc = lib().fd_decode_int8(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv),
                                  ctypes.byref(tks), ctypes.byref(tvs),
                                  kv_lengths.data_ptr(), int(n_q), int(bool(causal)),
                                  float(scale), ctypes.byref(to), ctypes.byref(o))
    _check(rc, "fd_decode_int8")
    return out


def topk_blocks(scores, kv_lengths, block_size, top_k, out=None, stream=None):
    """Gather lists from block scores: scores fp32 [B, n_q, n_blocks]
    (contiguous, on the device), kv_lengths int32 [B].  Returns (or fills)
    idx int32 [B, n_q, top_k*block_size]: the top_k blocks of each row in
    increasing order, expanded to cells, -1 past the length or unused."""
    if not scores.is_cuda or scores.dtype != torch.float32 or scores.dim() != 3 \
            or not scores.is_contiguous():
        raise ValueError("scores must be a contiguous CUDA float32 [B, n_q, n_blocks] tensor")
    B, n_q, nb = scores.shape
    W = int(top_k) * int(block_size)
    if out is None:
        out = torch.empty((B, n_q, W), dtype=torch.int32, device=scores.device)
    sh = _stream_handle(stream, scores.device)
    with _on_device(scores.device):
        rc = lib().fd_topk_blocks(scores.data_ptr(), B, n_q, nb, kv_lengths.data_ptr(),
                                  int(block_size), int(top_k), out.data_ptr(), sh)
    _check(rc, "fd_topk_blocks")
    return out


def decode_masked(q, k_cache, v_cache, kv_lengths, mask, n_q=None, causal=False, scale=None,
                  out=None, out_dtype=torch.bfloat16, num_ctas=0, kernel=FD_KERNEL_AUTO,
                  stream=None, workspace: Optional[Workspace] = None):
    """As ``decode`` with an additive fp32 mask [B, n_q, cap] (positions
    contiguous; -inf hides a position); 32-position chunks the mask hides for
    every query row are not read.  The default workspace leaves room for the
    tensor-core kernel's chunk list (its time then follows the visible
    chunks)."""
    B, nq, Hq, d = q.shape
    n_q = nq if n_q is None else n_q
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    Hkv = k_cache.shape[1]
    rows = (Hq // max(Hkv, 1)) * nq
    # room for the chunk list, counted in slots of the call's partials
    extra = -(-masked_list_bytes(B, k_cache.shape[2]) // (4 * slot_floats(rows, d)))
    out, sh, ws = _prepare(q, k_cache, out, out_dtype, B * Hkv + extra, rows, num_ctas,
                           kernel, stream, workspace)
    tq, tk, tv, tm, to = map(as_fd_tensor, (q, k_cache, v_cache, mask, out))
    o = _opts(sh, ws, num_ctas, kernel)
    with _on_device(q.device):
        rc = lib().fd_decode_masked(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv),
                                    kv_lengths.data_ptr(), ctypes.byref(tm), int(n_q),
                                    int(bool(causal)), float(scale), ctypes.byref(to),
                                    ctypes.byref(o))
    _check(rc, "fd_decode_masked")
    return out


def decode_append(q, k_cache, v_cache, k_new, v_new, kv_lengths, causal=True, scale=None,
                  update_lengths=True, out=None, out_dtype=torch.bfloat16, num_ctas=0,
                  kernel=FD_KERNEL_AUTO, stream=None, workspace: Optional[Workspace] = None):
    """One decode step with a fused append: writes k_new / v_new
    [B, n_q, Hkv, d] (bf16) into k_cache / v_cache [B, Hkv, cap, d] at
    positions kv_lengths[b] .. kv_lengths[b] + n_q - 1, attends q
    [B, n_q, Hq, d] over the prefix including them (row i sees up to
    kv_lengths[b] + i when causal) and, with update_lengths, advances
    kv_lengths (int32 [B], on the device) by n_q when the launch ends."""
    B, nq, Hq, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    Hkv = k_cache.shape[1]
    rows = (Hq // max(Hkv, 1)) * nq
    out, sh, ws = _prepare(q, k_cache, out, out_dtype, B * Hkv, rows, num_ctas,
                           kernel, stream, workspace)
    tq, tk, tv, tkn, tvn, to = map(as_fd_tensor, (q, k_cache, v_cache, k_new, v_new, out))
    o = _opts(sh, ws, num_ctas, kernel)
    with _on_device(q.device):
        rc = lib().fd_decode_append(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv),
                                    ctypes.byref(tkn), ctypes.byref(tvn), kv_lengths.data_ptr(),
                                    int(bool(update_lengths)), int(bool(causal)), float(scale),
                                    ctypes.byref(to), ctypes.byref(o))
    _check(rc, "fd_decode_append")
    return out


def decode_paged(q, k_pages, v_pages, block_table, kv_lengths, n_q=None,
                 causal=False, scale=None, k_scale=None, v_scale=None, out=None,
                 out_dtype=torch.bfloat16, num_ctas=0, kernel=FD_KERNEL_AUTO,
                 stream=None, workspace: Optional[Workspace] = None):
    """As ``decode`` (or ``decode_int8``) over a paged cache: pools
    k_pages / v_pages [num_pages, Hkv, page_size, d] (bf16, or int8 with fp32
    scales [num_pages, Hkv, page_size]) and block_table [B, max_pages] (int32,
    contiguous, on the device): position j of sequence b is row
    j % page_size of page block_table[b, j // page_size]."""
    B, nq, Hq, d = q.shape
    n_q = nq if n_q is None else n_q
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if (not block_table.is_contiguous() or block_table.dtype != torch.int32
            or block_table.dim() != 2 or block_table.shape[0] != B):
        raise ValueError("block_table must be a contiguous int32 [B, max_pages] tensor")
    Hkv = k_pages.shape[1]
    rows = (Hq // max(Hkv, 1)) * nq
    out, sh, ws = _prepare(q, k_pages, out, out_dtype, B * Hkv, rows, num_ctas,
                           kernel, stream, workspace)
    tq, tk, tv, to = map(as_fd_tensor, (q, k_pages, v_pages, out))
    pks = pvs = None
    if k_scale is not None or v_scale is not None:
        tks, tvs = as_fd_tensor(k_scale), as_fd_tensor(v_scale)
        pks, pvs = ctypes.byref(tks), ctypes.byref(tvs)
    o = _opts(sh, ws, num_ctas, kernel)
    with _on_device(q.device):
        rc = lib().fd_decode_paged(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv),
                                   pks, pvs, block_table.data_ptr(), int(block_table.shape[1]),
                                   kv_lengths.data_ptr(), int(n_q), int(bool(causal)),
                                   float(scale), ctypes.byref(to), ctypes.byref(o))
    _check(rc, "fd_decode_paged")
    return out


def decode_gather(q, k_cache, v_cache, idx, scale=None, out=None,
                  out_dtype=torch.bfloat16, num_ctas=0, kernel=FD_KERNEL_AUTO,
                  stream=None, workspace: Optional[Workspace] = None, bias=None,
                  k_scale=None, v_scale=None):
    """Attention of q [B, n_q, Hq, d] over the cache cells listed in
    idx [B, n_q, K] (int32, contiguous, on the device; < 0 = padding).
    bias (optional, bf16 caches): fp32 [B, n_q, K] contiguous, added to each
    entry's score (-inf drops the entry).  int8 caches take fp32 k_scale /
    v_scale [B, Hkv, cap] (fd_decode_gather_int8)."""
    B, nq, Hq, d = q.shape
    Hkv = k_cache.shape[1]
    if not idx.is_contiguous() or idx.dtype != torch.int32 or idx.dim() != 3:
        raise ValueError("idx must be a contiguous int32 [B, n_q, K] tensor")
    rows = Hq // max(Hkv, 1)
    out, sh, ws = _prepare(q, k_cache, out, out_dtype, B * nq * Hkv, rows, num_ctas,
                           kernel, stream, workspace)
    tq, tk, tv, to = map(as_fd_tensor, (q, k_cache, v_cache, out))
    o = _opts(sh, ws, num_ctas, kernel, 0.0 if scale is None else scale)
    if k_cache.dtype == torch.int8:
        if bias is not None or k_scale is None or v_scale is None:
            raise ValueError("int8 caches take k_scale and v_scale, and no bias")
        tks, tvs = as_fd_tensor(k_scale), as_fd_tensor(v_scale)
        with _on_device(q.device):
            rc = lib().fd_decode_gather_int8(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv),
                                             ctypes.byref(tks), ctypes.byref(tvs), idx.data_ptr(),
                                             int(idx.shape[2]), ctypes.byref(to), ctypes.byref(o))
        _check(rc, "fd_decode_gather_int8")
        return out
    if bias is not None:
        if (not bias.is_contiguous() or bias.dtype != torch.float32
                or tuple(bias.shape) != tuple(idx.shape)):
            raise ValueError("bias must be a contiguous float32 tensor shaped like idx")
        with _on_device(q.device):
            rc = lib().fd_decode_gather_bias(ctypes.byref(tq), ctypes.byref(tk),
                                             ctypes.byref(tv), idx.data_ptr(), bias.data_ptr(),
                                             int(idx.shape[2]), ctypes.byref(to),
                                             ctypes.byref(o))
        _check(rc, "fd_decode_gather_bias")
        return out
    with _on_device(q.device):
        rc = lib().fd_decode_gather(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv),
                                    idx.data_ptr(), int(idx.shape[2]), ctypes.byref(to),
                                    ctypes.byref(o))
    _check(rc, "fd_decode_gather")
    return out


# ------------------------------------------- 4-bit caches and their pages
_TENSOR = struct.Struct("Pii4q4q")     # fd_tensor
_OPTS = struct.Struct("PPiifi2i")      # fd_opts
_PAD = ((), (0, 0, 0), (0, 0), (0,), ())


# what stands for a dtype where only its size matters
_SIZES = {1: FD_U8, 2: FD_BF16, 4: FD_F32}


def _pack(t: torch.Tensor) -> bytes:
    """fd_tensor of a pool, as bytes."""
    shape = t.shape
    kind = _DTYPES.get(t.dtype, _SIZES.get(t.element_size()))
    if kind is None:
        raise TypeError("unsupported dtype %s" % t.dtype)
    n = len(shape)
    if not 1 <= n <= 4:
        raise ValueError("1 to 4 dimensions")
    pad = _PAD[n]
    return _TENSOR.pack(t.data_ptr(), kind, n, *shape, *pad, *t.stride(), *pad)


def _empty(shape, dtype, index, stream):
    """New memory that belongs to the given stream."""
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", index))


def _opts_for(workspace, index, stream, segments, rows, ctas, num_ctas) -> bytes:
    """fd_opts of a call: its stream, and the given workspace or the stream's,
    which has room for 1024 blocks and grows with the segments."""
    device = torch.device("cuda", index)
    sh = _stream_handle(stream, device)
    if workspace is None:
        workspace = workspace_for(device, sh, segments, rows, 256, ctas)
    return _OPTS.pack(sh, workspace.handle.value, num_ctas, FD_KERNEL_AUTO, 0.0, 0, 0, 0)


class _Unloaded:
    """Stands for the marshalling extension (csrc/fd_torch.cpp) until the first
    call, which loads it and libfd.so."""

    def __getattr__(self, name):
        global _native
        with _native_lock:
            if _native is self:
                _native = self.load()
        return getattr(_native, name)

    @staticmethod
    def load():
        if not os.path.exists(NATIVE_PATH):
            raise ImportError("%s is missing: build it first" % NATIVE_PATH)
        loader = importlib.machinery.ExtensionFileLoader("_fd_torch", NATIVE_PATH)
        m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_fd_torch", loader))
        loader.exec_module(m)
        calls = ("fd_decode_fp4", "fd_append_fp4", "fd_read_fp4", "fd_pages_reserve", "fd_pages_fork",
                 "fd_pages_free", "fd_pages_compact", "fd_pages_copy")
        m.bind(tuple(ctypes.cast(getattr(lib(), c), ctypes.c_void_p).value for c in calls),
               _ws_cache, _opts_for, _empty, FdError)
        return m


_native = _Unloaded()
_native_lock = threading.Lock()


def decode_fp4(q, k_cache, v_cache, k_scale, v_scale, kv_lengths, n_q=None, causal=False,
               scale=None, k_global=1.0, v_global=1.0, block_table=None, out=None,
               out_dtype=torch.bfloat16, num_ctas=0, stream=None,
               workspace: Optional[Workspace] = None):
    """As ``decode`` over a cache held in 4 bits: k_cache / v_cache
    [B, Hkv, cap, d/2] (uint8, two e2m1 codes a byte, the even value in the low
    nibble), k_scale / v_scale [B, Hkv, cap, d/16] (float8_e4m3fn, one per 16
    values); a value is code * scale * k_global (v_global).  With block_table
    [B, max_pages] (int32, contiguous) the four are pools
    [num_pages, Hkv, page_size, ...], as in ``decode_paged``."""
    return _native.decode_fp4(q, k_cache, v_cache, k_scale, v_scale, kv_lengths, n_q, causal, scale,
                              k_global, v_global, block_table, out, out_dtype, num_ctas, stream,
                              workspace)


def append_fp4(k_new, v_new, k_cache, v_cache, k_scale, v_scale, kv_lengths, new_lengths=None,
               lengths_out=None, k_global=1.0, v_global=1.0, block_table=None, stream=None,
               workspace: Optional[Workspace] = None):
    """Quantises new rows k_new / v_new [B, n, Hkv, d] (bf16) into a 4-bit
    cache (see ``decode_fp4``) at positions kv_lengths[b] .. kv_lengths[b] +
    new_lengths[b] - 1 (int32 [B]; None: n for every sequence; rows past it
    are padding).  lengths_out (int32 [B], may be kv_lengths) receives the
    lengths with the new rows."""
    _native.append_fp4(k_new, v_new, k_cache, v_cache, k_scale, v_scale, kv_lengths, new_lengths,
                       lengths_out, k_global, v_global, block_table, stream, workspace)


def read_fp4(k_cache, v_cache, k_scale, v_scale, kv_lengths, n, start=None, k_global=1.0,
             v_global=1.0, block_table=None, out=None, out_dtype=torch.bfloat16, stream=None,
             workspace: Optional[Workspace] = None):
    """Positions start[b] .. start[b] + n - 1 (int32 [B]; None: from 0) of a
    4-bit cache (see ``decode_fp4``) as numbers: returns (k, v)
    [B, n, Hkv, d], zeros at or past kv_lengths[b].  out: such a pair to fill."""
    return _native.read_fp4(k_cache, v_cache, k_scale, v_scale, kv_lengths, n, start, k_global,
                            v_global, block_table, out, out_dtype, stream, workspace)


def pages_reserve(block_table, kv_lengths, refs, page_size, n_new, pairs=None, count=None,
                  stream=None, workspace: Optional[Workspace] = None):
    """Pages of its own for each sequence's next n_new positions (an int for
    all of them, or int32 [B]): free pages where block_table [B, max_pages]
    has none, and pages to copy shared ones into.  Returns (pairs, count):
    pairs int32 [B, 2] (old, new) pages for ``pages_copy``, count int32 [1] of
    them, or minus the pages that are missing (nothing is then reserved).
    refs int32 [num_pages] counts the entries that name each page."""
    return _native.pages_reserve(block_table, kv_lengths, refs, page_size, n_new, pairs, count, stream,
                                 workspace)


def pages_fork(block_table, kv_lengths, refs, page_size, src, dst, lengths=None, stream=None,
               workspace: Optional[Workspace] = None):
    """Row dst[i] of the block table lets go of its pages and shares those of
    row src[i] (int32 [n]), the first lengths[i] positions of them where
    lengths is given; kv_lengths[dst[i]] follows."""
    _native.pages_fork(block_table, kv_lengths, refs, page_size, src, dst, lengths, stream, workspace)


def pages_free(block_table, kv_lengths, refs, page_size, seqs=None, lengths=None, stream=None,
               workspace: Optional[Workspace] = None):
    """Sequences seqs (int32 [n]; None: every one) shrink to lengths (int32
    [n]; None: 0) where that is less, and let go of the pages past it."""
    _native.pages_free(block_table, kv_lengths, refs, page_size, seqs, lengths, stream, workspace)


def pages_compact(block_table, refs, pairs=None, count=None, stream=None,
                  workspace: Optional[Workspace] = None):
    """Renumbers the pages in use to 0 .. used - 1 in block_table and refs.
    Returns (pairs, count): int32 [num_pages // 2, 2] (from, to) pages for
    ``pages_copy`` and int32 [1], how many."""
    return _native.pages_compact(block_table, refs, pairs, count, stream, workspace)


class PagePools:
    """The pools of a paged cache ([num_pages, ...] CUDA tensors of 1 to 4
    dimensions and of any dtype of 1, 2 or 4 bytes: codes, scales, of K and V, of
    every layer) as ``pages_copy`` wants them; made once, kept with the pools,
    whose memory it holds on to."""

    def __init__(self, pools):
        self.pools = list(pools)
        if not self.pools:
            raise ValueError("no pools")
        self.device = self.pools[0].device
        for t in self.pools:
            if not t.is_cuda or t.device != self.device:
                raise ValueError("pools must be CUDA tensors on one device")
        self.packed = b"".join(_pack(t) for t in self.pools)


def pages_copy(pools, pairs, count, stream=None, workspace: Optional[Workspace] = None):
    """Copies pages pairs[i] = (from, to) in every pool (a ``PagePools``, or
    up to 256 tensors) for i < count, both as ``pages_reserve`` and
    ``pages_compact`` return them."""
    if not isinstance(pools, PagePools):
        pools = PagePools(pools)
    _native.pages_copy(pools.packed, pools.device.index, pairs, count, stream, workspace)
