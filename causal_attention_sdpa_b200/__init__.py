"""Python binding of the gpt_attn C ABI (libgpt_attn.so, built in-tree for sm_100a).

Argument marshalling only: every step of the attention computation runs in the
CUDA kernels behind the C ABI.  PyTorch supplies device memory and streams.
There is no CPU or library fallback: if the shared library is missing or
cannot be loaded, importing the functions raises.

Entry points (same names as the C ABI, see include/gpt_attn.h):
  gpt_attn_fwd(q, k, v, scale=None, window=0, o=None, lse=None, stream=None) -> (o, lse)
  gpt_attn_bwd(q, k, v, o, lse, dO, scale=None, window=0, dq=None, dk=None, dv=None,
               workspace=None, stream=None) -> (dq, dk, dv)
  gpt_attn_bwd_workspace_bytes(B, H, T, D) -> int
  gpt_attn_fwd_sinks / gpt_attn_bwd_sinks: a sliding window with first tokens that stay visible
  gpt_attn_paged_append / _decode / _accept: new or drafted tokens over a paged key/value cache
  gpt_attn_pages_reserve / _fork / _free / _compact / _copy: the pages themselves
  gpt_attn_check(stream=None) -> int
  gpt_attn_status_string(status) -> str
Tensors are bf16 contiguous [B, H, T, D] on the GPU; lse is fp32 [B, H, T].
`stream` (a torch stream or a raw handle) is where a call runs instead of on the current stream.  What the
call allocates is taken there, and may be used on the current stream too once that waits for the other.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgpt_attn.so")

GPT_ATTN_OK = 0
GPT_ATTN_ERR_NULL = 1
GPT_ATTN_ERR_SHAPE = 2
GPT_ATTN_ERR_UNSUPPORTED_D = 3
GPT_ATTN_ERR_ALIGN = 4
GPT_ATTN_ERR_CUDA = 5
GPT_ATTN_ERR_TIMEOUT = 6
GPT_ATTN_ERR_WORKSPACE = 7
GPT_ATTN_ERR_UNAVAILABLE = 8
GPT_ATTN_ERR_BOUNDS = 9

EXPORTED = ("gpt_attn_fwd", "gpt_attn_bwd", "gpt_attn_bwd_workspace_bytes", "gpt_attn_bwd_delta",
            "gpt_attn_bwd_grads", "gpt_attn_bwd_dq_convert", "gpt_attn_check", "gpt_attn_status_string",
            "gpt_attn_debug_wait_timeout", "gpt_attn_bwd_noalloc", "gpt_attn_tmap_cache_stats",
            "gpt_attn_fwd_ex", "gpt_attn_bwd_ex", "gpt_attn_decode", "gpt_attn_decode_workspace_bytes",
            "gpt_attn_debug_skip_load", "gpt_attn_qk_prologue_fwd", "gpt_attn_qk_prologue_bwd",
            "gpt_attn_fwd_sinks", "gpt_attn_bwd_sinks", "gpt_attn_bwd_sinks_workspace_bytes",
            "gpt_attn_paged_append", "gpt_attn_paged_decode", "gpt_attn_paged_decode_workspace_bytes",
            "gpt_attn_paged_accept", "gpt_attn_pages_reserve", "gpt_attn_pages_fork", "gpt_attn_pages_free",
            "gpt_attn_pages_compact", "gpt_attn_pages_copy", "gpt_attn_pages_workspace_bytes")


class GptAttnStrides(ctypes.Structure):
    """The C ABI's gpt_attn_strides: element strides (batch, head, token) of a [b, h, t, d] tensor."""
    _fields_ = [("batch", ctypes.c_longlong), ("head", ctypes.c_longlong), ("token", ctypes.c_longlong)]


class GptAttnLayout(ctypes.Structure):
    """The C ABI's gpt_attn_layout: strides of q, k, v, o, dO, dq, dk, dv."""
    _fields_ = [(n, GptAttnStrides) for n in ("q", "k", "v", "o", "dO", "dq", "dk", "dv")]


class GptAttnMask(ctypes.Structure):
    """The C ABI's gpt_attn_mask: a window for every head, or per-head windows (host ints), and
    optional document starts (device int32 [B, T])."""
    _fields_ = [("window", ctypes.c_int), ("head_windows", ctypes.POINTER(ctypes.c_int)),
                ("doc_start", ctypes.c_void_p)]


class GptAttnPagedCache(ctypes.Structure):
    """The C ABI's gpt_attn_paged_cache: pools, table and lengths of a paged key/value cache."""
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("lens", ctypes.c_void_p)] + [(n, ctypes.c_int) for n in ("B", "Hkv", "D", "n_pages", "page",
                                                                         "max_pages")]


_lib = None


class GptAttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """Load libgpt_attn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m causal_attention_sdpa_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.gpt_attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.gpt_attn_fwd.restype = i
        L.gpt_attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, sz, vp]
        L.gpt_attn_bwd.restype = i
        L.gpt_attn_bwd_delta.argtypes = [vp, vp, vp, i, i, i, i, vp, sz, vp]
        L.gpt_attn_bwd_delta.restype = i
        L.gpt_attn_bwd_grads.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, sz, vp]
        L.gpt_attn_bwd_grads.restype = i
        L.gpt_attn_bwd_dq_convert.argtypes = [vp, i, i, i, i, f, vp, sz, vp]
        L.gpt_attn_bwd_dq_convert.restype = i
        L.gpt_attn_bwd_workspace_bytes.argtypes = [i, i, i, i]
        L.gpt_attn_bwd_workspace_bytes.restype = sz
        L.gpt_attn_check.argtypes = [vp]
        L.gpt_attn_check.restype = i
        L.gpt_attn_status_string.argtypes = [i]
        L.gpt_attn_status_string.restype = ctypes.c_char_p
        L.gpt_attn_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.gpt_attn_bwd_noalloc.restype = i
        L.gpt_attn_tmap_cache_stats.argtypes = [ctypes.POINTER(ctypes.c_longlong), ctypes.POINTER(ctypes.c_longlong),
                                                 ctypes.POINTER(ctypes.c_int)]
        L.gpt_attn_tmap_cache_stats.restype = None
        mp = ctypes.POINTER(GptAttnMask)
        lp = ctypes.POINTER(GptAttnLayout)
        L.gpt_attn_fwd_ex.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, mp, lp, vp]
        L.gpt_attn_fwd_ex.restype = i
        L.gpt_attn_bwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, mp, lp, vp, sz, vp]
        L.gpt_attn_bwd_ex.restype = i
        L.gpt_attn_fwd_sinks.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, mp, i, lp, vp]
        L.gpt_attn_fwd_sinks.restype = i
        L.gpt_attn_bwd_sinks.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, mp, i, lp, vp, sz, vp]
        L.gpt_attn_bwd_sinks.restype = i
        L.gpt_attn_bwd_sinks_workspace_bytes.argtypes = [i, i, i, i, i, i]
        L.gpt_attn_bwd_sinks_workspace_bytes.restype = sz
        L.gpt_attn_decode_workspace_bytes.argtypes = [i, i, i, i, i]
        L.gpt_attn_decode_workspace_bytes.restype = sz
        L.gpt_attn_decode.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, sz, vp]
        L.gpt_attn_decode.restype = i
        spp = ctypes.POINTER(GptAttnStrides)
        L.gpt_attn_qk_prologue_fwd.argtypes = [vp, vp, vp, vp, i, i, i, i, i, f, spp, vp]
        L.gpt_attn_qk_prologue_fwd.restype = i
        L.gpt_attn_qk_prologue_bwd.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, spp, vp]
        L.gpt_attn_qk_prologue_bwd.restype = i
        cp = ctypes.POINTER(GptAttnPagedCache)
        L.gpt_attn_paged_append.argtypes = [cp, vp, vp, i, vp, spp, vp]
        L.gpt_attn_paged_append.restype = i
        L.gpt_attn_paged_decode_workspace_bytes.argtypes = [i, i, i, i, i]
        L.gpt_attn_paged_decode_workspace_bytes.restype = sz
        L.gpt_attn_paged_decode.argtypes = [vp, cp, vp, vp, vp, vp, i, i, f, i, i, spp, vp, sz, vp]
        L.gpt_attn_paged_decode.restype = i
        L.gpt_attn_paged_accept.argtypes = [cp, vp, vp, i, vp]
        L.gpt_attn_paged_accept.restype = i
        L.gpt_attn_pages_workspace_bytes.argtypes = [i, i, i]
        L.gpt_attn_pages_workspace_bytes.restype = sz
        L.gpt_attn_pages_reserve.argtypes = [vp, vp, vp, i, i, i, i, vp, vp, vp, sz, vp]
        L.gpt_attn_pages_reserve.restype = i
        L.gpt_attn_pages_fork.argtypes = [vp, vp, vp, i, i, i, i, vp, vp, vp, vp, sz, vp]
        L.gpt_attn_pages_fork.restype = i
        L.gpt_attn_pages_free.argtypes = [vp, vp, vp, i, i, i, vp, vp]
        L.gpt_attn_pages_free.restype = i
        L.gpt_attn_pages_compact.argtypes = [vp, vp, i, i, i, vp, vp, vp, vp, vp, sz, vp]
        L.gpt_attn_pages_compact.restype = i
        L.gpt_attn_pages_copy.argtypes = [vp, vp, i, i, i, i, vp, i, vp, vp]
        L.gpt_attn_pages_copy.restype = i
        L.gpt_attn_debug_skip_load.argtypes = [i]
        L.gpt_attn_debug_skip_load.restype = i
        L.gpt_attn_debug_wait_timeout.argtypes = [i, vp]
        L.gpt_attn_debug_wait_timeout.restype = i
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().gpt_attn_status_string(int(status)).decode()


gpt_attn_status_string = status_string


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_HERE = contextlib.nullcontext()


def _memory_of(stream, dev):
    """Context in which memory for a call on `stream` is taken: on that stream, so that what the call
    writes comes after all that was done there with the memory before.  Work on the current stream
    may still use what the allocator would hand out there, and nothing orders it and the call."""
    if stream is None:
        return _HERE
    torch = _t()
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream_handle(stream)
        # 1 is another name of the legacy default stream, whose handle torch knows as 0
        stream = torch.cuda.ExternalStream(0 if handle == 1 else handle, device=dev)
    return torch.cuda.stream(stream)


def _hand_over(stream, *tensors):
    """Results of a call on another stream than the current one, whose memory came from there: not to be
    handed out again before what the current stream does with them has ended."""
    if stream is None:
        return
    here = _t().cuda.current_stream(tensors[0].device)
    for t in tensors:
        t.record_stream(here)


_INT_MAX = 2 ** 31 - 1


def _reach(x):
    """A window or a number of sinks as a C int: one past its range acts as its largest value does."""
    return min(max(int(x), -_INT_MAX), _INT_MAX)


def _fits(*sizes):
    """Whether sizes are at least 1 and a C int holds them; ctypes would wrap others without a word."""
    return min(sizes) >= 1 and max(sizes) <= _INT_MAX


def _ptr(t):
    # A plain int: the c_void_p argtypes convert it (and None to NULL) without a wrapper object.
    return t.data_ptr() if t is not None else None


def _check_bf16(name, t, shape):
    import torch
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a contiguous CUDA bf16 tensor of shape {tuple(shape)}")


def gpt_attn_fwd(q, k, v, scale=None, window=0, o=None, lse=None, stream=None):
    """Forward pass; returns (o, lse).  Asynchronous on `stream` (default: current)."""
    import torch
    B, H, T, D = q.shape
    for n, t in (("q", q), ("k", k), ("v", v)):
        _check_bf16(n, t, q.shape)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with _memory_of(stream, q.get_device()):
        if o is None:
            o = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    _check_bf16("o", o, q.shape)
    rc = lib().gpt_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, T, D, float(scale),
                            _reach(window), _stream_handle(stream))
    if rc != GPT_ATTN_OK:
        raise GptAttnError(rc, "gpt_attn_fwd")
    _hand_over(stream, o, lse)
    return o, lse


def gpt_attn_bwd_workspace_bytes(B, H, T, D) -> int:
    if not _fits(B, H, T, D):
        return 0
    return int(lib().gpt_attn_bwd_workspace_bytes(int(B), int(H), int(T), int(D)))


def gpt_attn_bwd(q, k, v, o, lse, dO, scale=None, window=0, dq=None, dk=None, dv=None, workspace=None,
                 stream=None):
    """Backward pass of sum(O * dO); returns (dq, dk, dv).  Asynchronous on `stream`."""
    import torch
    B, H, T, D = q.shape
    for n, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dO", dO)):
        _check_bf16(n, t, q.shape)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    need = gpt_attn_bwd_workspace_bytes(B, H, T, D)
    with _memory_of(stream, q.get_device()):
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(q) if dk is None else dk
        dv = torch.empty_like(q) if dv is None else dv
        if workspace is None:
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = lib().gpt_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk),
                            _ptr(dv), B, H, T, D, float(scale), _reach(window), _ptr(workspace), ws_bytes,
                            _stream_handle(stream))
    if rc != GPT_ATTN_OK:
        raise GptAttnError(rc, "gpt_attn_bwd")
    _hand_over(stream, dq, dk, dv)
    return dq, dk, dv


def gpt_attn_bwd_noalloc(q, k, v, o, lse, dO, scale=None, window=0, dq=None, dk=None, dv=None, stream=None):
    """gpt_attn_bwd with the library's built-in 32 MiB scratch instead of a workspace argument.

    For callers that must not allocate device memory when the backward pass runs.  Pass
    dq, dk and dv to keep this wrapper itself allocation-free.  Calls that overlap on the
    GPU share the scratch and race; the first call on a device should precede any capture.
    """
    import torch
    B, H, T, D = q.shape
    for n, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dO", dO)):
        _check_bf16(n, t, q.shape)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with _memory_of(stream, q.get_device()):
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(q) if dk is None else dk
        dv = torch.empty_like(q) if dv is None else dv
    rc = lib().gpt_attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk),
                                    _ptr(dv), B, H, T, D, float(scale), _reach(window), _stream_handle(stream))
    if rc != GPT_ATTN_OK:
        raise GptAttnError(rc, "gpt_attn_bwd_noalloc")
    _hand_over(stream, dq, dk, dv)
    return dq, dk, dv


def _mask(H, window=0, head_windows=None, doc_start=None):
    """A GptAttnMask (and the host array it points at, which must outlive the call)."""
    import torch
    hw = None
    if head_windows is not None:
        hw = (ctypes.c_int * H)(*[_reach(x) for x in head_windows])
        if len(head_windows) != H:
            raise ValueError(f"head_windows needs {H} entries")
    if doc_start is not None:
        if doc_start.dtype != torch.int32 or not doc_start.is_cuda or not doc_start.is_contiguous():
            raise ValueError("doc_start must be a contiguous CUDA int32 tensor [B, T]")
    m = GptAttnMask(_reach(window), ctypes.cast(hw, ctypes.POINTER(ctypes.c_int)) if hw is not None else None,
                    doc_start.data_ptr() if doc_start is not None else None)
    return m, hw


def _check_view(name, t, shape):
    """A bf16 CUDA tensor of the given [B, H, T, D] shape whose last dimension is contiguous."""
    import torch
    if t.dtype != torch.bfloat16 or not t.is_cuda or tuple(t.shape) != tuple(shape) or t.stride(3) != 1:
        raise ValueError(f"{name} must be a CUDA bf16 [B, H, T, D] view of shape {tuple(shape)} with stride 1 in D")


def _strides(t):
    return GptAttnStrides(*_steps(t))


def _steps(t):
    """Strides of the first three dimensions; one of size 1 is never stepped along, so its stride, which may be
    anything, is 0."""
    n, st = t.shape, t.stride()
    return st[0] if n[0] > 1 else 0, st[1] if n[1] > 1 else 0, st[2] if n[2] > 1 else 0


_STRIDES24 = ctypes.c_longlong * 24


def _layout(**tensors):
    """A GptAttnLayout of the tensors' strides (given in the struct's order q, k, v, o, dO, dq, dk,
    dv), or None when they are all contiguous [B, H, T, D] (the C default)."""
    ts = list(tensors.values())
    if all(t.is_contiguous() for t in ts):
        return None
    v = []
    for t in ts:
        v += _steps(t)
    return GptAttnLayout.from_buffer(_STRIDES24(*v))     # one flat copy; the struct keeps it alive


def _byref(x):
    return ctypes.byref(x) if x is not None else None


def gpt_attn_fwd_ex(q, k, v, scale=None, window=0, head_windows=None, doc_start=None, o=None, lse=None,
                    stream=None):
    """Forward pass with per-head windows and/or document starts, on any [B, H, T, D] views whose D
    dimension is contiguous (e.g. the q, k, v columns of a fused [B, T, 3, H, D] projection, and an
    o that is a view of a [B, T, H, D] buffer); returns (o, lse)."""
    import torch
    B, H, T, D = q.shape
    for n, t in (("q", q), ("k", k), ("v", v)):
        _check_view(n, t, q.shape)
    if doc_start is not None and tuple(doc_start.shape) != (B, T):
        raise ValueError(f"doc_start must have shape {(B, T)}")
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    with _memory_of(stream, q.get_device()):
        o = torch.empty((B, H, T, D), dtype=q.dtype, device=q.device) if o is None else o
        lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device) if lse is None else lse
    _check_view("o", o, q.shape)
    m, keep = _mask(H, window, head_windows, doc_start)
    lay = _layout(q=q, k=k, v=v, o=o, dO=o, dq=o, dk=o, dv=o)
    rc = lib().gpt_attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, T, D, float(scale),
                               ctypes.byref(m), _byref(lay), _stream_handle(stream))
    del keep
    if rc != GPT_ATTN_OK:
        raise GptAttnError(rc, "gpt_attn_fwd_ex")
    _hand_over(stream, o, lse)
    return o, lse


def gpt_attn_bwd_ex(q, k, v, o, lse, dO, scale=None, window=0, head_windows=None, doc_start=None, dq=None,
                    dk=None, dv=None, workspace=None, stream=None):
    """Backward pass under the same mask as gpt_attn_fwd_ex, on [B, H, T, D] views with contiguous D
    (dq, dk, dv may be views into one [B, T, 3, H, D] gradient buffer); returns (dq, dk, dv)."""
    import torch
    B, H, T, D = q.shape
    for n, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dO", dO)):
        _check_view(n, t, q.shape)
    if doc_start is not None and tuple(doc_start.shape) != (B, T):
        raise ValueError(f"doc_start must have shape {(B, T)}")
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    mk = lambda: torch.empty((B, H, T, D), dtype=q.dtype, device=q.device)
    with _memory_of(stream, q.get_device()):
        dq = mk() if dq is None else dq
        dk = mk() if dk is None else dk
        dv = mk() if dv is None else dv
        ws, nbytes = _ws(workspace, q)
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _check_view(n, t, q.shape)
    m, keep = _mask(H, window, head_windows, doc_start)
    lay = _layout(q=q, k=k, v=v, o=o, dO=dO, dq=dq, dk=dk, dv=dv)
    rc = lib().gpt_attn_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk),
                               _ptr(dv), B, H, T, D, float(scale), ctypes.byref(m), _byref(lay), _ptr(ws),
                               nbytes, _stream_handle(stream))
    del keep
    if rc != GPT_ATTN_OK:
        raise GptAttnError(rc, "gpt_attn_bwd_ex")
    _hand_over(stream, dq, dk, dv)
    return dq, dk, dv


# The calls from here on are often shorter on the GPU than their checks on the host: torch is looked up
# once, devices are compared by number, and the raw stream is asked for directly.
_torch = None


def _t():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _launch(what, dev, stream, *args):
    """Calls the entry point `what` with `args` and the stream, the tensors' device being current."""
    torch = _t()
    fn = getattr(_lib or lib(), what)
    if stream is not None:
        stream = _stream_handle(stream)
    if dev == torch._C._cuda_getDevice():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream)
    if rc != GPT_ATTN_OK:
        raise GptAttnError(rc, what)


def _check_tensor(name, t, dtype, shape, dev):
    """A contiguous tensor of the given type and shape on CUDA device number `dev`."""
    if t.dtype is not dtype or t.get_device() != dev or dev < 0 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {str(dtype)[6:]} tensor of shape {tuple(shape)} on CUDA device "
                         f"{dev}")


def _check_views(dev, shape, **views):
    """bf16 tensors of the given [b, h, t, d] shape on CUDA device `dev`, contiguous in their last dimension."""
    bf16 = _t().bfloat16
    for n, t in views.items():
        if t.dtype is not bf16 or t.get_device() != dev or dev < 0 or t.shape != shape or t.stride(3) != 1:
            raise ValueError(f"{n} must be a bf16 view of shape {tuple(shape)} with stride 1 in its last dimension on "
                             f"CUDA device {dev}")


def _check_workspace(t, dev):
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on CUDA device {dev}")


def _check_sinks_call(q, doc_start, head_windows, lse):
    """The arguments of a call with sinks; returns (B, H, T, D), the shape and the device number."""
    if q.dim() != 4:
        raise ValueError("q must be a CUDA bf16 [B, H, T, D] view")
    shape, dev = q.shape, q.get_device()
    B, H, T, D = shape
    if lse is not None:
        _check_tensor("lse", lse, _t().float32, (B, H, T), dev)
    if doc_start is not None:
        _check_tensor("doc_start", doc_start, _t().int32, (B, T), dev)
    if head_windows is not None and len(head_windows) != H:
        raise ValueError(f"head_windows needs {H} entries")
    return B, H, T, D, shape, dev


def _sinks_mask(H, window, head_windows, doc_start):
    if head_windows is not None:
        return _mask(H, window, head_windows, doc_start)
    return GptAttnMask(_reach(window), None, None if doc_start is None else doc_start.data_ptr()), None


def gpt_attn_fwd_sinks(q, k, v, window=0, sinks=0, scale=None, head_windows=None, doc_start=None, o=None, lse=None,
                       stream=None):
    """Sliding-window forward in which the first `sinks` tokens of each document (of the row without
    doc_start) stay visible: query i sees key j iff doc_start[i] <= j <= i and (i - j < window or
    j - doc_start[i] < sinks).  Views and the other arguments as for gpt_attn_fwd_ex; returns (o, lse)."""
    torch = _t()
    B, H, T, D, shape, dev = _check_sinks_call(q, doc_start, head_windows, lse)
    _check_views(dev, shape, q=q, k=k, v=v)
    if o is not None:
        _check_views(dev, shape, o=o)
    with _memory_of(stream, dev):
        if o is None:
            o = torch.empty_like(q) if q.is_contiguous() else torch.empty(shape, dtype=q.dtype, device=q.device)
        if lse is None:
            lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    m, keep = _sinks_mask(H, window, head_windows, doc_start)
    lay = None
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and o.is_contiguous()):
        lay = _layout(q=q, k=k, v=v, o=o, dO=o, dq=o, dk=o, dv=o)
    _launch("gpt_attn_fwd_sinks", dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B,
            H, T, D, D ** -0.5 if scale is None else float(scale), ctypes.byref(m), _reach(sinks), _byref(lay))
    _hand_over(stream, o, lse)
    return o, lse


def gpt_attn_bwd_sinks_workspace_bytes(B, H, T, D, window=0, sinks=0) -> int:
    """Bytes of workspace of gpt_attn_bwd_sinks (window: the largest of the call's windows)."""
    if not _fits(B, H, T, D):
        return 0
    return int(lib().gpt_attn_bwd_sinks_workspace_bytes(int(B), int(H), int(T), int(D), _reach(window),
                                                        _reach(sinks)))


def gpt_attn_bwd_sinks(q, k, v, o, lse, dO, window=0, sinks=0, scale=None, head_windows=None, doc_start=None,
                       dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Backward pass of gpt_attn_fwd_sinks under the same mask; returns (dq, dk, dv)."""
    torch = _t()
    B, H, T, D, shape, dev = _check_sinks_call(q, doc_start, head_windows, lse)
    _check_views(dev, shape, q=q, k=k, v=v, o=o, dO=dO)
    device = q.device
    if workspace is not None:
        _check_workspace(workspace, dev)
    with _memory_of(stream, dev):
        if dq is None and dk is None and dv is None:
            dq, dk, dv = torch.empty((3, B, H, T, D), dtype=q.dtype, device=device).unbind(0)     # one allocation
        else:
            dq, dk, dv = (torch.empty(shape, dtype=q.dtype, device=device) if t is None else t for t in (dq, dk, dv))
            _check_views(dev, shape, dq=dq, dk=dk, dv=dv)
        if workspace is None:
            top = max(head_windows) if head_windows is not None else window
            workspace = torch.empty(max(gpt_attn_bwd_sinks_workspace_bytes(B, H, T, D, top, sinks), 16),
                                    dtype=torch.uint8, device=device)
    m, keep = _sinks_mask(H, window, head_windows, doc_start)
    lay = _layout(q=q, k=k, v=v, o=o, dO=dO, dq=dq, dk=dk, dv=dv)
    _launch("gpt_attn_bwd_sinks", dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
            dO.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, T, D,
            D ** -0.5 if scale is None else float(scale), ctypes.byref(m), _reach(sinks), _byref(lay),
            workspace.data_ptr(), workspace.numel() * workspace.element_size())
    _hand_over(stream, dq, dk, dv)
    return dq, dk, dv


def _ws(workspace, q):
    import torch
    B, H, T, D = q.shape
    if workspace is None:
        workspace = torch.empty(max(gpt_attn_bwd_workspace_bytes(B, H, T, D), 16), dtype=torch.uint8,
                                device=q.device)
    return workspace, workspace.numel() * workspace.element_size()


def gpt_attn_bwd_delta(o, lse, dO, workspace, stream=None):
    """Stage 1 of the backward pass (Delta, scaled lse, zeroed dQ accumulator)."""
    B, H, T, D = o.shape
    with _memory_of(stream, o.get_device()):
        ws, nbytes = _ws(workspace, o)
    rc = lib().gpt_attn_bwd_delta(_ptr(o), _ptr(lse), _ptr(dO), B, H, T, D, _ptr(ws), nbytes,
                                  _stream_handle(stream))
    if rc != GPT_ATTN_OK:
        raise GptAttnError(rc, "gpt_attn_bwd_delta")
    _hand_over(stream, ws)
    return ws


def gpt_attn_bwd_grads(q, k, v, dO, dk, dv, workspace, scale=None, window=0, stream=None):
    """Stage 2 of the backward pass (dK, dV written; dQ accumulated in the workspace)."""
    B, H, T, D = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    ws, nbytes = _ws(workspace, q)
    rc = lib().gpt_attn_bwd_grads(_ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(dk), _ptr(dv), B, H, T, D,
                                  float(scale), _reach(window), _ptr(ws), nbytes, _stream_handle(stream))
    if rc != GPT_ATTN_OK:
        raise GptAttnError(rc, "gpt_attn_bwd_grads")


def gpt_attn_bwd_dq_convert(dq, workspace, scale=None, stream=None):
    """Stage 3 of the backward pass (bf16 dQ = scale * the fp32 accumulator)."""
    B, H, T, D = dq.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    ws, nbytes = _ws(workspace, dq)
    rc = lib().gpt_attn_bwd_dq_convert(_ptr(dq), B, H, T, D, float(scale), _ptr(ws), nbytes,
                                       _stream_handle(stream))
    if rc != GPT_ATTN_OK:
        raise GptAttnError(rc, "gpt_attn_bwd_dq_convert")


def gpt_attn_decode_workspace_bytes(B, H, T_max, D, window=0) -> int:
    if not _fits(B, H, T_max, D):
        return 0
    return int(lib().gpt_attn_decode_workspace_bytes(int(B), int(H), int(T_max), int(D), _reach(window)))


def gpt_attn_decode(q, k_cache, v_cache, seq_lens, scale=None, window=0, o=None, lse=None, workspace=None,
                    stream=None):
    """Decode: q bf16 [B, H, D] against caches bf16 [B, H, T_max, D]; seq_lens int32 [B] on the
    device.  Returns (o [B, H, D], lse [B, H])."""
    import torch
    B, H, T, D = k_cache.shape
    _check_bf16("k_cache", k_cache, (B, H, T, D))
    _check_bf16("v_cache", v_cache, (B, H, T, D))
    _check_bf16("q", q, (B, H, D))
    if seq_lens.dtype != torch.int32 or not seq_lens.is_cuda or tuple(seq_lens.shape) != (B,):
        raise ValueError("seq_lens must be a CUDA int32 tensor [B]")
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    need = gpt_attn_decode_workspace_bytes(B, H, T, D, window)
    with _memory_of(stream, q.get_device()):
        o = torch.empty_like(q) if o is None else o
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device) if lse is None else lse
        if workspace is None:
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    rc = lib().gpt_attn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens), _ptr(o), _ptr(lse), B, H,
                               T, D, float(scale), _reach(window), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if rc != GPT_ATTN_OK:
        raise GptAttnError(rc, "gpt_attn_decode")
    _hand_over(stream, o, lse)
    return o, lse


def _check_int32(name, t, shape, dev):
    _check_tensor(name, t, _t().int32, shape, dev)


def _check_pools(k_pages, v_pages):
    """Two pools [n_pages, Hkv, page, D]; returns their shape and device number."""
    shape, dev, bf16 = k_pages.shape, k_pages.get_device(), _t().bfloat16
    if len(shape) != 4 or dev < 0:
        raise ValueError("k_pages must be a contiguous CUDA bf16 tensor [n_pages, Hkv, page, D]")
    _check_tensor("k_pages", k_pages, bf16, shape, dev)
    _check_tensor("v_pages", v_pages, bf16, shape, dev)
    return shape, dev


def _paged_cache(k_pages, v_pages, table, lens):
    """A GptAttnPagedCache of the checked tensors, and the device number."""
    (P, Hkv, page, D), dev = _check_pools(k_pages, v_pages)
    if table.dim() != 2:
        raise ValueError("table must be a contiguous int32 tensor [B, max_pages]")
    B, M = table.shape
    _check_int32("table", table, (B, M), dev)
    _check_int32("lens", lens, (B,), dev)
    return GptAttnPagedCache(k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr(), lens.data_ptr(), B, Hkv, D, P,
                             page, M), dev


def _pair_strides(a, b):
    """Strides of two [b, h, n, d] tensors, or None when both are contiguous."""
    if a.is_contiguous() and b.is_contiguous():
        return None
    return (GptAttnStrides * 2)(GptAttnStrides(*_steps(a)), GptAttnStrides(*_steps(b)))


def gpt_attn_paged_append(k_pages, v_pages, table, lens, k_new, v_new, n_new=None, stream=None):
    """Writes the rows of N new tokens (k_new, v_new: bf16 [B, Hkv, N, D] views) of every sequence into
    its pages, token n at position lens[b] + n; n_new (int32 [B]): how many of them are used."""
    cache, dev = _paged_cache(k_pages, v_pages, table, lens)
    N = k_new.shape[2] if k_new.dim() == 4 else 0
    _check_views(dev, (cache.B, cache.Hkv, N, cache.D), k_new=k_new, v_new=v_new)
    if n_new is not None:
        _check_int32("n_new", n_new, (cache.B,), dev)
    _launch("gpt_attn_paged_append", dev, stream, ctypes.byref(cache), k_new.data_ptr(), v_new.data_ptr(), N,
            _ptr(n_new), _pair_strides(k_new, v_new))


def gpt_attn_paged_decode_workspace_bytes(B, H, Hkv, N, D) -> int:
    if not _fits(B, H, Hkv, N, D):
        return 0
    return int(lib().gpt_attn_paged_decode_workspace_bytes(int(B), int(H), int(Hkv), int(N), int(D)))


def gpt_attn_paged_decode(q, k_pages, v_pages, table, lens, parents=None, n_new=None, scale=None, window=0, sinks=0,
                          o=None, lse=None, workspace=None, stream=None):
    """Attention of N new tokens of every sequence (q: bf16 [B, H, N, D] view; their keys and values
    already appended) over the paged cache and, by the tree `parents` (int32 [B, N]; None: one after the
    other), over each other.  With a window each sees the tokens within it and the first `sinks` ones.
    Returns (o [B, H, N, D], lse [B, H, N])."""
    torch = _t()
    cache, dev = _paged_cache(k_pages, v_pages, table, lens)
    if q.dim() != 4:
        raise ValueError("q must be a CUDA bf16 [B, H, N, D] view")
    shape, device = q.shape, q.device
    _, H, N, D = shape
    B = cache.B
    _check_views(dev, (B, H, N, cache.D), q=q)
    if o is not None:
        _check_views(dev, shape, o=o)
    if lse is not None:
        _check_tensor("lse", lse, torch.float32, (B, H, N), dev)
    if parents is not None:
        _check_int32("parents", parents, (B, N), dev)
    if n_new is not None:
        _check_int32("n_new", n_new, (B,), dev)
    if workspace is not None:
        _check_workspace(workspace, dev)
    with _memory_of(stream, dev):
        if o is None:
            o = torch.empty_like(q) if q.is_contiguous() else torch.empty(shape, dtype=q.dtype, device=device)
        if lse is None:
            lse = torch.empty((B, H, N), dtype=torch.float32, device=device)
        if workspace is None:
            need = gpt_attn_paged_decode_workspace_bytes(B, H, cache.Hkv, N, D)
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    _launch("gpt_attn_paged_decode", dev, stream, q.data_ptr(), ctypes.byref(cache), _ptr(n_new), _ptr(parents),
            o.data_ptr(), lse.data_ptr(), H, N, D ** -0.5 if scale is None else float(scale), _reach(window),
            _reach(sinks), _pair_strides(q, o), workspace.data_ptr(), workspace.numel() * workspace.element_size())
    _hand_over(stream, o, lse)
    return o, lse


def gpt_attn_paged_accept(k_pages, v_pages, table, lens, accepted, n_accepted, stream=None):
    """Moves the rows of the accepted nodes up: node accepted[b, i] (int32 [B, N]) to position
    lens[b] + i for i < n_accepted[b] (int32 [B]).  lens itself is the caller's to change."""
    cache, dev = _paged_cache(k_pages, v_pages, table, lens)
    if accepted.dim() != 2:
        raise ValueError("accepted must be a contiguous int32 tensor [B, N]")
    N = accepted.shape[1]
    if N > _INT_MAX:
        raise ValueError("accepted must have fewer than 2^31 columns")
    _check_int32("accepted", accepted, (cache.B, N), dev)
    _check_int32("n_accepted", n_accepted, (cache.B,), dev)
    _launch("gpt_attn_paged_accept", dev, stream, ctypes.byref(cache), accepted.data_ptr(), n_accepted.data_ptr(), N)


def gpt_attn_pages_workspace_bytes(S, M, P) -> int:
    if not _fits(S, M, P):
        return 0
    return int(lib().gpt_attn_pages_workspace_bytes(int(S), int(M), int(P)))


def _check_state(table, refs, lens=None):
    """Table, lengths and holders of the pages; returns (S, M, P, device number)."""
    if table.dim() != 2 or refs.dim() != 1:
        raise ValueError("table must be an int32 tensor [S, M] and refs one [P]")
    S, M = table.shape
    P, dev = refs.shape[0], table.get_device()
    if max(S, M, P) > _INT_MAX:
        raise ValueError("table and refs must have fewer than 2^31 entries in each dimension")
    _check_int32("table", table, (S, M), dev)
    _check_int32("refs", refs, (P,), dev)
    if lens is not None:
        _check_int32("lens", lens, (S,), dev)
    return S, M, P, dev


def _page_tokens(page):
    if not -_INT_MAX <= page <= _INT_MAX:
        raise ValueError("page must be less than 2^31")
    return int(page)


def _pages_workspace(workspace, S, M, P, table):
    if workspace is None:
        return _t().empty(max(gpt_attn_pages_workspace_bytes(S, M, P), 16), dtype=_t().uint8, device=table.device)
    _check_workspace(workspace, table.get_device())
    return workspace


def _int32_out(name, t, shape, like):
    """An int32 result of the given shape: the caller's, checked, or a new one on the device of `like`."""
    if t is None:
        if like.shape == shape:
            return _t().empty_like(like)
        return _t().empty(shape, dtype=_t().int32, device=like.device)
    _check_int32(name, t, shape, like.get_device())
    return t


def gpt_attn_pages_reserve(table, lens, refs, page, tokens, status=None, workspace=None, stream=None):
    """Gives every slot pages for tokens[s] (int32 [S]) more tokens, the lowest free ones first; table
    and refs change in place.  Returns status int32 [S]: 0 nothing asked, 1 done, -1 refused (the table's
    row is too short, or has a page behind a -1), -2 not enough free pages."""
    S, M, P, dev = _check_state(table, refs, lens)
    _check_int32("tokens", tokens, (S,), dev)
    with _memory_of(stream, dev):
        status = _int32_out("status", status, (S,), tokens)
        ws = _pages_workspace(workspace, S, M, P, table)
    _launch("gpt_attn_pages_reserve", dev, stream, table.data_ptr(), lens.data_ptr(), refs.data_ptr(), S, M, P,
            _page_tokens(page), tokens.data_ptr(), status.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size())
    _hand_over(stream, status)
    return status


def gpt_attn_pages_fork(table, lens, refs, page, parents, status=None, pairs=None, workspace=None, stream=None):
    """Slot s becomes a copy of slot parents[s] (int32 [S], negative: nothing asked): full pages are
    shared, a partial last page gets a page of its own.  Table, lens and refs change in place.  Returns
    (status int32 [S], pairs int32 [S, 2]): status as for gpt_attn_pages_reserve, pairs the pages to copy
    with gpt_attn_pages_copy in every layer's pools."""
    S, M, P, dev = _check_state(table, refs, lens)
    _check_int32("parents", parents, (S,), dev)
    with _memory_of(stream, dev):
        status = _int32_out("status", status, (S,), parents)
        pairs = _int32_out("pairs", pairs, (S, 2), table)
        ws = _pages_workspace(workspace, S, M, P, table)
    _launch("gpt_attn_pages_fork", dev, stream, table.data_ptr(), lens.data_ptr(), refs.data_ptr(), S, M, P,
            _page_tokens(page), parents.data_ptr(), status.data_ptr(), pairs.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size())
    _hand_over(stream, status, pairs)
    return status, pairs


def gpt_attn_pages_free(table, lens, refs, drop, stream=None):
    """Slots with drop[s] > 0 (int32 [S]) give their pages back; table, lens and refs change in place."""
    S, M, P, dev = _check_state(table, refs, lens)
    _check_int32("drop", drop, (S,), dev)
    _launch("gpt_attn_pages_free", dev, stream, table.data_ptr(), lens.data_ptr(), refs.data_ptr(), S, M, P, drop.data_ptr())


def gpt_attn_pages_compact(table, refs, workspace=None, stream=None):
    """Packs the n pages in use into places 0 to n - 1.  Returns (new_table, new_refs, pairs int32
    [P // 2, 2], moves int32 [1]); gpt_attn_pages_copy(k, v, pairs, n_pairs=moves) moves the pages."""
    S, M, P, dev = _check_state(table, refs)
    n = P // 2
    with _memory_of(stream, dev):
        results = _t().empty(2 * n + S * M + P + 1, dtype=_t().int32, device=table.device)    # one allocation
        ws = _pages_workspace(workspace, S, M, P, table)
    pairs, new_table, new_refs, moves = results.split((2 * n, S * M, P, 1))
    pairs, new_table = pairs.view(n, 2), new_table.view(S, M)
    _launch("gpt_attn_pages_compact", dev, stream, table.data_ptr(), refs.data_ptr(), S, M, P, new_table.data_ptr(),
            new_refs.data_ptr(), pairs.data_ptr(), moves.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size())
    _hand_over(stream, results)
    return new_table, new_refs, pairs, moves


def gpt_attn_pages_copy(k_pages, v_pages, pairs, n_pairs=None, stream=None):
    """Copies page pairs[i, 0] onto page pairs[i, 1] in both pools, for the first n_pairs (int32 [1] on
    the device; None: all) rows of pairs (int32 [n, 2]); rows with a page outside the pools are skipped."""
    (P, Hkv, page, D), dev = _check_pools(k_pages, v_pages)
    if pairs.dim() != 2:
        raise ValueError("pairs must be a contiguous int32 tensor [n, 2]")
    n = pairs.shape[0]
    if n > _INT_MAX:
        raise ValueError("pairs must have fewer than 2^31 rows")
    _check_int32("pairs", pairs, (n, 2), dev)
    if n_pairs is not None:
        _check_int32("n_pairs", n_pairs, (1,), dev)
    _launch("gpt_attn_pages_copy", dev, stream, k_pages.data_ptr(), v_pages.data_ptr(), P, Hkv, page, D,
            pairs.data_ptr(), n, _ptr(n_pairs))


def gpt_attn_qk_prologue_fwd(q_raw, k_raw, qk_norm=True, rope_base=10000.0, q_out=None, k_out=None, stream=None):
    """QK-Norm + rotary prologue: returns (q, k) bf16 [B, H, T, D] (contiguous unless q_out/k_out are
    given); q_raw, k_raw may be strided views (e.g. of a fused [B, T, 3, H, D] projection)."""
    import torch
    B, H, T, D = q_raw.shape
    mk = lambda: torch.empty((B, H, T, D), dtype=torch.bfloat16, device=q_raw.device)
    with _memory_of(stream, q_raw.get_device()):
        q_out = mk() if q_out is None else q_out
        k_out = mk() if k_out is None else k_out
    ts = [q_raw, k_raw, q_out, k_out]
    for n, t in zip(("q_raw", "k_raw", "q_out", "k_out"), ts):
        _check_view(n, t, q_raw.shape)
    arr = (GptAttnStrides * 4)(*[_strides(t) for t in ts])
    rc = lib().gpt_attn_qk_prologue_fwd(*[_ptr(t) for t in ts], B, H, T, D, int(bool(qk_norm)), float(rope_base),
                                        arr, _stream_handle(stream))
    if rc != GPT_ATTN_OK:
        raise GptAttnError(rc, "gpt_attn_qk_prologue_fwd")
    _hand_over(stream, q_out, k_out)
    return q_out, k_out


def gpt_attn_qk_prologue_bwd(q_raw, k_raw, dq_out, dk_out, qk_norm=True, rope_base=10000.0, dq_raw=None,
                             dk_raw=None, stream=None):
    """Gradient of the prologue: returns (dq_raw, dk_raw)."""
    import torch
    B, H, T, D = q_raw.shape
    mk = lambda: torch.empty((B, H, T, D), dtype=torch.bfloat16, device=q_raw.device)
    with _memory_of(stream, q_raw.get_device()):
        dq_raw = mk() if dq_raw is None else dq_raw
        dk_raw = mk() if dk_raw is None else dk_raw
    ts = [q_raw, k_raw, dq_out, dk_out, dq_raw, dk_raw]
    for n, t in zip(("q_raw", "k_raw", "dq_out", "dk_out", "dq_raw", "dk_raw"), ts):
        _check_view(n, t, q_raw.shape)
    arr = (GptAttnStrides * 6)(*[_strides(t) for t in ts])
    rc = lib().gpt_attn_qk_prologue_bwd(*[_ptr(t) for t in ts], B, H, T, D, int(bool(qk_norm)), float(rope_base),
                                        arr, _stream_handle(stream))
    if rc != GPT_ATTN_OK:
        raise GptAttnError(rc, "gpt_attn_qk_prologue_bwd")
    _hand_over(stream, dq_raw, dk_raw)
    return dq_raw, dk_raw


def gpt_attn_check(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return int(lib().gpt_attn_check(_stream_handle(stream)))


def gpt_attn_tmap_cache_stats():
    """(hits, misses, entries) of the library's host-side tensor-map cache."""
    h, m, u = ctypes.c_longlong(0), ctypes.c_longlong(0), ctypes.c_int(0)
    lib().gpt_attn_tmap_cache_stats(ctypes.byref(h), ctypes.byref(m), ctypes.byref(u))
    return h.value, m.value, u.value


def gpt_attn_debug_wait_timeout(timeout_us: int, stream=None) -> int:
    return int(lib().gpt_attn_debug_wait_timeout(int(timeout_us), _stream_handle(stream)))
