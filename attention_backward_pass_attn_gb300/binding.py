"""ctypes binding of the C ABI in ``include/attn.h``.

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libattn_gb300.so``.  PyTorch supplies device memory (outputs and
the backward's workspace are allocated here with ``torch.empty`` unless the
caller passes them) and the current CUDA stream.  There is no fallback: if the
library is missing or a call fails, an exception is raised.
"""

from __future__ import annotations

import ctypes
import math
import operator
import os
import threading

import torch

from . import build as _build

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = 1
ATTN_ERR_UNSUPPORTED = 2
ATTN_ERR_CUDA = 3
ATTN_ERR_TIMEOUT = 4
ATTN_ERR_WORKSPACE = 5
ATTN_ERR_DEVICE = 6
ATTN_ERR_TOO_LARGE = 7

# How attn_bwd forms dQ (attn_dq_method_t in include/attn.h).
ATTN_DQ_AUTO = 0
ATTN_DQ_REDUCE = 1
ATTN_DQ_SEPARATE = 2

_lock = threading.Lock()
_lib = None


class AttnError(RuntimeError):
    """A non-zero status returned by the library."""

    def __init__(self, fn: str, status: int, text: str):
        super().__init__("%s failed: %s (status %d)" % (fn, text, status))
        self.status = status


def load_library(path: str | None = None):
    """Load ``libattn_gb300.so`` (built in-tree by ``__graft_entry__.build()``)."""
    global _lib
    if path is None and _lib is not None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or _build.LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                "CUDA library %s is not built; run __graft_entry__.build() (needs nvcc). "
                "There is no CPU fallback." % p)
        lib = ctypes.CDLL(p)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        sig = {
            "attn_fwd": (i, [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp]),
            "attn_fwd_ex": (i, [vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, f, vp]),
            "attn_fwd_fp8": (i, [vp, vp, vp, f, f, f, vp, vp, i, i, i, i, i, f, vp]),
            "attn_bwd_workspace_size": (sz, [i, i, i, i]),
            "attn_bwd": (i, [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, vp, sz, vp]),
            "attn_bwd_ex": (i, [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, f, vp,
                                sz, vp]),
            "attn_bwd_fp8": (i, [vp, vp, vp, vp, vp, vp, f, f, f, f, f, vp, vp, vp, vp, i, i, i,
                                 i, i, f, vp, sz, vp]),
            "attn_bwd_opts": (i, [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, f,
                                  i, vp, sz, vp]),
            "attn_bwd_main_dkdv": (i, [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, vp, sz, vp]),
            "attn_bwd_dq": (i, [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp, sz, vp]),
            "attn_bwd_preprocess": (i, [vp, vp, vp, i, i, i, i, vp, sz, vp]),
            "attn_bwd_main": (i, [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, vp, sz, vp]),
            "attn_bwd_dq_convert": (i, [vp, i, i, i, i, f, vp, sz, vp]),
            "attn_bwd_noalloc": (i, [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, vp]),
            "ssd_workspace_size": (sz, [i, i, i, i, i, i]),
            "ssd_fwd": (i, [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, sz, vp]),
            "ssd_bwd": (i, [vp] * 13 + [i, i, i, i, i, i, vp, sz, vp]),
            "rope_fwd": (i, [vp] * 5 + [i, i] + [vp] * 3 + [i] * 6 + [vp]),
            "rope_bwd": (i, [vp] * 5 + [i, i] + [vp] * 3 + [i] * 6 + [vp]),
            "kv_cache_write": (i, [vp] * 10 + [i] * 7 + [vp]),
            "kv_cache_read": (i, [vp] * 9 + [i] * 7 + [vp]),
            "attn_decode_workspace_size": (sz, [i]),
            "attn_decode": (i, [vp] * 9 + [i] * 8 + [f, vp, sz, vp]),
            "attn_last_device_error": (i, [vp]),
            "attn_device_error_word": (i, [vp, ctypes.POINTER(ctypes.c_int)]),
            "attn_watchdog_selftest": (i, [ctypes.c_uint64, vp]),
            "attn_status_string": (ctypes.c_char_p, [i]),
            "attn_version": (i, []),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        if path is None:
            _lib = lib
        return lib


def status_string(status: int) -> str:
    return load_library().attn_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != ATTN_OK:
        raise AttnError(fn, status, status_string(status))


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _shape4(t: torch.Tensor, name: str):
    if t.dim() != 4:
        raise ValueError("%s must be [B, H, N, d], got %s" % (name, tuple(t.shape)))
    return tuple(t.shape)


def _check_tensor(t: torch.Tensor, name: str, shape, dtype=torch.bfloat16):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device.type != "cuda":
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _doc_ptr(doc, B: int, N: int):
    """Device pointer of a document map (int32 CUDA tensor [B, N], contiguous), or None."""
    if doc is None:
        return None
    _check_tensor(doc, "doc", (B, N), torch.int32)
    return doc.data_ptr()


def _default_scale(d: int, scale):
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


def attn_bwd_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(load_library().attn_bwd_workspace_size(B, H, N, d))


def alloc_workspace(B: int, H: int, N: int, d: int, device) -> torch.Tensor:
    """A uint8 device buffer of the size attn_bwd needs (torch allocations are
    256-byte aligned)."""
    n = max(attn_bwd_workspace_size(B, H, N, d), 256)
    return torch.empty(n, dtype=torch.uint8, device=device)


def attn_fwd(q, k, v, causal: bool, scale=None, out=None, lse=None, stream=None, window=0,
             doc=None):
    """O = softmax(scale q k^T [+ causal mask]) v and the row log-sum-exp L.

    q, k, v: bf16 CUDA tensors [B, H, N, d] (d = 64 or 128), contiguous.
    window > 0 (causal only): query i sees keys i - window < j <= i.
    doc (causal only): int32 CUDA tensor [B, N], the first position of each
    position's document; query i sees keys doc[b, i] <= j <= i.
    Returns (O bf16 [B, H, N, d], L fp32 [B, H, N]).
    """
    B, H, N, d = _shape4(q, "q")
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check_tensor(t, n, (B, H, N, d))
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    _check_tensor(out, "out", (B, H, N, d))
    _check_tensor(lse, "lse", (B, H, N), torch.float32)
    st = load_library().attn_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                    lse.data_ptr(), B, H, N, d, int(bool(causal)), int(window),
                                    _doc_ptr(doc, B, N), _default_scale(d, scale),
                                    _stream(stream))
    _check("attn_fwd_ex", st)
    return out, lse


def _check_fp8(t: torch.Tensor, name: str, shape):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.element_size() != 1 or t.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise ValueError("%s must hold e4m3 bytes (float8_e4m3fn or uint8), got %s"
                         % (name, t.dtype))
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError("%s must be contiguous with shape %s" % (name, tuple(shape)))


def attn_fwd_fp8(q8, k8, v8, descales, causal: bool, scale=None, out=None, lse=None,
                 stream=None):
    """O (bf16) and L (fp32) of exact attention over e4m3 inputs.

    q8, k8, v8: e4m3 bytes [B, H, N, 128] (float8_e4m3fn or uint8 views);
    descales: (q_descale, k_descale, v_descale), the factors that turn the
    stored values into the values they stand for.
    """
    B, H, N, d = _shape4(q8, "q8")
    for t, n in ((q8, "q8"), (k8, "k8"), (v8, "v8")):
        _check_fp8(t, n, (B, H, N, d))
    out = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q8.device) if out is None \
        else out
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q8.device) if lse is None else lse
    _check_tensor(out, "out", (B, H, N, d))
    _check_tensor(lse, "lse", (B, H, N), torch.float32)
    qd, kd, vd = (float(x) for x in descales)
    st = load_library().attn_fwd_fp8(q8.data_ptr(), k8.data_ptr(), v8.data_ptr(), qd, kd, vd,
                                     out.data_ptr(), lse.data_ptr(), B, H, N, d,
                                     int(bool(causal)), _default_scale(d, scale),
                                     _stream(stream))
    _check("attn_fwd_fp8", st)
    return out, lse


def attn_bwd_fp8(q8, k8, v8, o, do8, lse, descales, ds_scale: float, causal: bool, scale=None,
                 ds_amax=None, workspace=None, stream=None):
    """dQ, dK, dV (bf16) of exact attention with e4m3 operands.

    q8, k8, v8, do8: e4m3 bytes [B, H, N, 128]; descales: (q, k, v, dO)
    factors; o (bf16) and lse: the forward's outputs; ds_scale: the factor
    dS is multiplied by before its rounding to e4m3 (keep ds_scale x
    max|dS| <= 448).  ds_amax: a 1-element float32 CUDA tensor that receives
    the largest |dS| of the call (or None).  Returns (dQ, dK, dV).
    """
    B, H, N, d = _shape4(q8, "q8")
    for t, n in ((q8, "q8"), (k8, "k8"), (v8, "v8"), (do8, "do8")):
        _check_fp8(t, n, (B, H, N, d))
    _check_tensor(o, "o", (B, H, N, d))
    _check_tensor(lse, "lse", (B, H, N), torch.float32)
    if ds_amax is not None:
        _check_tensor(ds_amax, "ds_amax", (1,), torch.float32)
    dq, dk, dv = (torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q8.device)
                  for _ in range(3))
    if workspace is None:
        workspace = alloc_workspace(B, H, N, d, q8.device)
    qd, kd, vd, dod = (float(x) for x in descales)
    st = load_library().attn_bwd_fp8(q8.data_ptr(), k8.data_ptr(), v8.data_ptr(), o.data_ptr(),
                                     do8.data_ptr(), lse.data_ptr(), qd, kd, vd, dod,
                                     float(ds_scale), dq.data_ptr(), dk.data_ptr(),
                                     dv.data_ptr(),
                                     None if ds_amax is None else ds_amax.data_ptr(), B, H, N,
                                     d, int(bool(causal)), _default_scale(d, scale),
                                     workspace.data_ptr(),
                                     workspace.numel() * workspace.element_size(),
                                     _stream(stream))
    _check("attn_bwd_fp8", st)
    return dq, dk, dv


def attn_bwd(q, k, v, o, do, lse, causal: bool, scale=None, dq=None, dk=None, dv=None,
             workspace=None, stream=None, window=0, doc=None, dq_method=ATTN_DQ_AUTO):
    """dQ, dK, dV of exact attention (the fused backward).

    o, lse: the forward's outputs; do: the upstream gradient of o.
    dq_method: ATTN_DQ_AUTO, ATTN_DQ_REDUCE (the main kernel reduces dQ
    partials into an fp32 accumulator) or ATTN_DQ_SEPARATE (a separate
    query-stationary dQ pass).
    Returns (dQ, dK, dV), bf16 [B, H, N, d].
    """
    B, H, N, d = _shape4(q, "q")
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (do, "do")):
        _check_tensor(t, n, (B, H, N, d))
    _check_tensor(lse, "lse", (B, H, N), torch.float32)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    for t, n in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        _check_tensor(t, n, (B, H, N, d))
    if workspace is None:
        workspace = alloc_workspace(B, H, N, d, q.device)
    st = load_library().attn_bwd_opts(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                      do.data_ptr(), lse.data_ptr(), dq.data_ptr(),
                                      dk.data_ptr(), dv.data_ptr(), B, H, N, d,
                                      int(bool(causal)), int(window), _doc_ptr(doc, B, N),
                                      _default_scale(d, scale), int(dq_method),
                                      workspace.data_ptr(),
                                      workspace.numel() * workspace.element_size(),
                                      _stream(stream))
    _check("attn_bwd_opts", st)
    return dq, dk, dv


def attn_bwd_preprocess(o, do, lse, workspace, stream=None):
    B, H, N, d = _shape4(o, "o")
    st = load_library().attn_bwd_preprocess(o.data_ptr(), do.data_ptr(), lse.data_ptr(), B, H, N,
                                            d, workspace.data_ptr(),
                                            workspace.numel() * workspace.element_size(),
                                            _stream(stream))
    _check("attn_bwd_preprocess", st)


def attn_bwd_main(q, k, v, do, dk, dv, causal: bool, workspace, scale=None, stream=None):
    B, H, N, d = _shape4(q, "q")
    st = load_library().attn_bwd_main(q.data_ptr(), k.data_ptr(), v.data_ptr(), do.data_ptr(),
                                      dk.data_ptr(), dv.data_ptr(), B, H, N, d,
                                      int(bool(causal)), _default_scale(d, scale),
                                      workspace.data_ptr(),
                                      workspace.numel() * workspace.element_size(),
                                      _stream(stream))
    _check("attn_bwd_main", st)


def attn_bwd_main_dkdv(q, k, v, do, dk, dv, causal: bool, workspace, scale=None, stream=None):
    B, H, N, d = _shape4(q, "q")
    st = load_library().attn_bwd_main_dkdv(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                           do.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N,
                                           d, int(bool(causal)), _default_scale(d, scale),
                                           workspace.data_ptr(),
                                           workspace.numel() * workspace.element_size(),
                                           _stream(stream))
    _check("attn_bwd_main_dkdv", st)


def attn_bwd_dq(q, k, v, do, dq, causal: bool, workspace, scale=None, stream=None):
    B, H, N, d = _shape4(q, "q")
    st = load_library().attn_bwd_dq(q.data_ptr(), k.data_ptr(), v.data_ptr(), do.data_ptr(),
                                    dq.data_ptr(), B, H, N, d, int(bool(causal)),
                                    _default_scale(d, scale), workspace.data_ptr(),
                                    workspace.numel() * workspace.element_size(),
                                    _stream(stream))
    _check("attn_bwd_dq", st)


def attn_bwd_dq_convert(dq, workspace, scale=None, stream=None):
    B, H, N, d = _shape4(dq, "dq")
    st = load_library().attn_bwd_dq_convert(dq.data_ptr(), B, H, N, d, _default_scale(d, scale),
                                            workspace.data_ptr(),
                                            workspace.numel() * workspace.element_size(),
                                            _stream(stream))
    _check("attn_bwd_dq_convert", st)


def attn_last_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error status."""
    return int(load_library().attn_last_device_error(_stream(stream)))


def attn_device_error_word(stream=None):
    w = ctypes.c_int(0)
    st = load_library().attn_device_error_word(_stream(stream), ctypes.byref(w))
    return int(st), int(w.value)


def attn_watchdog_selftest(limit_ns: int, stream=None) -> int:
    return int(load_library().attn_watchdog_selftest(int(limit_ns), _stream(stream)))


# ------------------------------------------------------------------ Mamba-2 layer
def _ssd_dims(x, B):
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [Bt, T, H, P] and B [Bt, T, G, N]")
    Bt, T, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    return Bt, T, H, G, N, P


def ssd_workspace(Bt, T, H, G, N, P, device) -> torch.Tensor:
    n = max(int(load_library().ssd_workspace_size(Bt, T, H, G, N, P)), 256)
    return torch.empty(n, dtype=torch.uint8, device=device)


def _ssd_check_inputs(x, dt, A, B, C, D, dims):
    Bt, T, H, G, N, P = dims
    _check_tensor(x, "x", (Bt, T, H, P))
    _check_tensor(B, "B", (Bt, T, G, N))
    _check_tensor(C, "C", (Bt, T, G, N))
    _check_tensor(dt, "dt", (Bt, T, H), torch.float32)
    _check_tensor(A, "A", (H,), torch.float32)
    _check_tensor(D, "D", (H,), torch.float32)


def ssd_fwd(x, dt, A, B, C, D, y=None, workspace=None, stream=None):
    """y [Bt, T, H, P] fp32 of the Mamba-2 state-space layer."""
    dims = _ssd_dims(x, B)
    _ssd_check_inputs(x, dt, A, B, C, D, dims)
    y = torch.empty(x.shape, dtype=torch.float32, device=x.device) if y is None else y
    _check_tensor(y, "y", x.shape, torch.float32)
    ws = ssd_workspace(*dims, x.device) if workspace is None else workspace
    st = load_library().ssd_fwd(x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(),
                                C.data_ptr(), D.data_ptr(), y.data_ptr(), *dims, ws.data_ptr(),
                                ws.numel() * ws.element_size(), _stream(stream))
    _check("ssd_fwd", st)
    return y


def ssd_bwd(x, dt, A, B, C, D, dy, workspace=None, out=None, stream=None):
    """Gradients of <dy, y>: dict with dx, ddt, dA, dB, dC, dD (fp32)."""
    dims = _ssd_dims(x, B)
    _ssd_check_inputs(x, dt, A, B, C, D, dims)
    _check_tensor(dy, "dy", x.shape)
    f32 = dict(dtype=torch.float32, device=x.device)
    if out is None:
        out = {"dx": torch.empty(x.shape, **f32), "ddt": torch.empty(dt.shape, **f32),
               "dA": torch.empty(A.shape, **f32), "dB": torch.empty(B.shape, **f32),
               "dC": torch.empty(C.shape, **f32), "dD": torch.empty(D.shape, **f32)}
    ws = ssd_workspace(*dims, x.device) if workspace is None else workspace
    st = load_library().ssd_bwd(x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(),
                                C.data_ptr(), D.data_ptr(), dy.data_ptr(), out["dx"].data_ptr(),
                                out["ddt"].data_ptr(), out["dA"].data_ptr(),
                                out["dB"].data_ptr(), out["dC"].data_ptr(),
                                out["dD"].data_ptr(), *dims, ws.data_ptr(),
                                ws.numel() * ws.element_size(), _stream(stream))
    _check("ssd_bwd", st)
    return out


# ------------------------------------------------------------------ the answering path
# Rotary positions, the paged key/value cache, attention of one new token.
# Tensors must live on the current CUDA device, whose current stream the calls
# run on unless ``stream`` names another; what a call allocates belongs to the
# stream it runs on.
# The checks come first as one cheap test; only what fails it is looked at for
# the reason, so that a call of a few microseconds on the GPU is not drowned by
# its checks.
_INT_MAX = 2 ** 31 - 1  # ctypes would drop the bits above
_E4M3_DTYPES = (torch.float8_e4m3fn, torch.uint8)
_DEVICES = [torch.device("cuda", i) for i in range(64)]  # cheaper to pass than an index
# PyTorch's own shortcuts where it has them; a build without CUDA does not, and
# the host-side checks work there too.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing",
                     torch.cuda.is_current_stream_capturing)


def _device_index(t: torch.Tensor, name: str) -> int:
    """The index of the current CUDA device, which t must be on."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    dev = t.get_device()
    if dev < 0:
        raise ValueError("%s must be a CUDA tensor" % name)
    if dev != _current_device():
        raise ValueError("%s must be on the current CUDA device" % name)
    return dev


def _stream_on(stream, dev: int) -> int:
    """The CUDA stream handle of ``stream``, or of device dev's current one."""
    if stream is None:
        return _current_stream(dev)
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != dev:
        raise ValueError("stream must be on CUDA device %d, like the first tensor" % dev)
    return _stream(stream)


def _empty(shape, dtype, dev: int, stream) -> torch.Tensor:
    """Uninitialised memory of the stream the call runs on: on another than
    the current one, the allocator must not hand it to the current one when it
    is freed."""
    if stream is None or _stream_on(stream, dev) == _current_stream(dev):
        return torch.empty(shape, dtype=dtype, device=_DEVICES[dev])
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


# ctypes arrays of strides and section counts by their values: making one
# costs more than the rest of a call's checks.
_arrays = {}


def _array(ctype, values: tuple):
    got = _arrays.get((ctype, values))
    if got is None:
        if len(_arrays) >= 4096:
            _arrays.clear()
        got = _arrays[(ctype, values)] = (ctype * len(values))(*values)
    return got


def _check_like(t: torch.Tensor, name: str, shape, dtype, dev: int):
    """A contiguous tensor of this shape and type on CUDA device ``dev``."""
    if type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape \
            and t.get_device() == dev and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.get_device() != dev:
        raise ValueError("%s must be on CUDA device %d, like the first tensor" % (name, dev))
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _check_rows(t: torch.Tensor, name: str, shape, dev: int):
    """A bf16 [B, H, N, d] tensor whose head dimension is contiguous, with any
    16-byte strides; returns its three element strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype is not torch.bfloat16:
        raise ValueError("%s must be torch.bfloat16, got %s" % (name, t.dtype))
    if t.get_device() != dev:
        raise ValueError("%s must be on CUDA device %d, like the first tensor" % (name, dev))
    sb, sh, sn, sd = t.stride()
    if sd != 1 and shape[3] > 1:
        raise ValueError("%s must be contiguous in its head dimension" % name)
    if (sb | sh | sn) & 7:
        for n, s in zip(shape, (sb, sh, sn)):
            if n > 1 and s % 8:
                raise ValueError("%s must have strides that are multiples of 8" % name)
    return sb, sh, sn


def _check_cache(k_cache, v_cache, k_descale, v_descale, page_table, dev):
    """(pages, Hkv, page_size, d, B, max_pages) of a cache and its page table."""
    shape = k_cache.shape
    if len(shape) != 4:
        raise ValueError("k_cache must be [pages, Hkv, page_size, d], got %s" % (tuple(shape),))
    dtype = k_cache.dtype
    if k_descale is None or v_descale is None:
        if k_descale is not v_descale:
            raise ValueError("k_descale and v_descale come together")
        if dtype is not torch.bfloat16:
            raise ValueError("k_cache must be torch.bfloat16 without descale factors, got %s"
                             % dtype)
    else:
        if dtype not in _E4M3_DTYPES:
            raise ValueError("k_cache must hold e4m3 bytes (float8_e4m3fn or uint8) with descale "
                             "factors, got %s" % dtype)
        _check_like(k_descale, "k_descale", shape[:3], torch.float32, dev)
        _check_like(v_descale, "v_descale", shape[:3], torch.float32, dev)
    _check_like(k_cache, "k_cache", shape, dtype, dev)
    _check_like(v_cache, "v_cache", shape, dtype, dev)
    table = page_table.shape
    if len(table) != 2:
        raise ValueError("page_table must be [B, max_pages], got %s" % (tuple(table),))
    _check_like(page_table, "page_table", table, torch.int32, dev)
    return (*shape, *table)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _rope(fn, q, k, pos, inv_freq, sections, interleaved, out, stream):
    dev = _device_index(q, "q")
    shape = q.shape if q.dim() == 4 else _shape4(q, "q")
    B, H, N, d = shape
    strides = _check_rows(q, "q", shape, dev)
    if k is None:
        Hk, strides = 0, strides + (0, 0, 0)
    else:
        Hk = (k.shape if k.dim() == 4 else _shape4(k, "k"))[1]
        strides += _check_rows(k, "k", (B, Hk, N, d), dev)
    pshape = pos.shape
    if len(pshape) != 3 or (pshape[1] != B and pshape[1] != 1) or pshape[2] != N:
        raise ValueError("pos must be [axes, B or 1, N], got %s" % (tuple(pshape),))
    axes = pshape[0]
    _check_like(pos, "pos", pshape, torch.int32, dev)
    _check_like(inv_freq, "inv_freq", (d // 2,), torch.float32, dev)
    sections = (d // 2,) if sections is None else tuple(sections)
    if not 1 <= axes <= 4 or len(sections) != axes or sum(sections) != d // 2 \
            or min(sections) < 0:
        raise ValueError("sections must be one count for each of pos's 1 to 4 axes that sum to "
                         "d/2 = %d, got %s for %d" % (d // 2, sections, axes))
    oq, ok = (None, None) if out is None else out
    if oq is None:
        oq = _empty(shape, torch.bfloat16, dev, stream)
    else:
        _check_like(oq, "out[0]", shape, torch.bfloat16, dev)
    if k is None:
        ok, kp, okp = None, None, None
    else:
        if ok is None:
            ok = _empty((B, Hk, N, d), torch.bfloat16, dev, stream)
        else:
            _check_like(ok, "out[1]", (B, Hk, N, d), torch.bfloat16, dev)
        kp, okp = k.data_ptr(), ok.data_ptr()
    st = fn(load_library())(q.data_ptr(), kp, pos.data_ptr(), inv_freq.data_ptr(),
                            _array(ctypes.c_int, sections), axes, 1 if interleaved else 0,
                            _array(ctypes.c_int64, strides), oq.data_ptr(), okp, B, H, Hk, N, d,
                            pshape[1], _stream_on(stream, dev))
    if st:
        _check("rope", st)
    return oq, ok


_ROPE_FWD = operator.attrgetter("rope_fwd")
_ROPE_BWD = operator.attrgetter("rope_bwd")


def rope_fwd(q, k, pos, inv_freq, sections=None, interleaved=False, out=None, stream=None):
    """q and k turned by their positions: (q', k'), bf16, contiguous.

    q [B, H, N, d] and k [B, Hk, N, d] (or None): bf16 CUDA tensors, d = 64 or
    128, contiguous in d; other strides are free as long as they are multiples
    of 8 (so q may be ``qkv[:, :, :H].transpose(1, 2)`` of a fused projection).
    pos: int32 [axes, B or 1, N].  inv_freq: fp32 [d/2], radians per position.
    sections: how many pairs turn by each axis (sum d/2; default: one axis).
    interleaved: pairs are (2i, 2i+1) instead of (i, i + d/2).
    out: (q', k') to write into, contiguous; may be the inputs themselves when
    those are contiguous.
    """
    return _rope(_ROPE_FWD, q, k, pos, inv_freq, sections, interleaved, out, stream)


def rope_bwd(dq, dk, pos, inv_freq, sections=None, interleaved=False, out=None, stream=None):
    """The gradients of rope_fwd's q and k from those of its results (the turn
    by the negative angles); arguments as for rope_fwd."""
    return _rope(_ROPE_BWD, dq, dk, pos, inv_freq, sections, interleaved, out, stream)


def alloc_kv_cache(num_pages: int, Hkv: int, page_size: int, d: int, device,
                   dtype=torch.bfloat16):
    """(k_cache, v_cache, k_descale, v_descale), zeroed: a bf16 cache (factors
    None), or an e4m3 one (dtype torch.float8_e4m3fn) with its fp32 factors."""
    if dtype not in (torch.bfloat16, torch.float8_e4m3fn):
        raise ValueError("dtype must be torch.bfloat16 or torch.float8_e4m3fn, got %s" % dtype)
    shape = (num_pages, Hkv, page_size, d)
    fp8 = dtype == torch.float8_e4m3fn
    caches = [torch.zeros(shape, dtype=torch.uint8 if fp8 else dtype, device=device)
              for _ in range(2)]
    if not fp8:
        return caches[0], caches[1], None, None
    factors = [torch.ones(shape[:3], dtype=torch.float32, device=device) for _ in range(2)]
    return caches[0].view(dtype), caches[1].view(dtype), factors[0], factors[1]


def _check_span(start, count, B, dev):
    _check_like(start, "start", (B,), torch.int32, dev)
    if count is not None:
        _check_like(count, "count", (B,), torch.int32, dev)


def kv_cache_write(k, v, k_cache, v_cache, page_table, start, count=None, k_descale=None,
                   v_descale=None, stream=None):
    """Append k, v to a paged cache, in place.

    k, v: bf16 [B, Hkv, T, d], strides as free as rope_fwd's.  Token t <
    count[b] (default: all T) becomes position start[b] + t of sequence b.
    k_cache, v_cache: [pages, Hkv, page_size, d], bf16, or e4m3 with fp32
    factors k_descale, v_descale [pages, Hkv, page_size], which the call
    chooses for every row it writes.  page_table: int32 [B, max_pages];
    start, count: int32 [B].
    """
    dev = _device_index(k_cache, "k_cache")
    P, Hkv, ps, d, B, mp = _check_cache(k_cache, v_cache, k_descale, v_descale, page_table, dev)
    T = (k.shape if k.dim() == 4 else _shape4(k, "k"))[2]
    shape = (B, Hkv, T, d)
    strides = _check_rows(k, "k", shape, dev) + _check_rows(v, "v", shape, dev)
    _check_span(start, count, B, dev)
    if B * Hkv * T > _INT_MAX:  # expanded rows take no memory
        _check("kv_cache_write", ATTN_ERR_UNSUPPORTED)
    st = load_library().kv_cache_write(k.data_ptr(), v.data_ptr(),
                                       _array(ctypes.c_int64, strides),
                                       k_cache.data_ptr(), v_cache.data_ptr(), _ptr(k_descale),
                                       _ptr(v_descale), page_table.data_ptr(), start.data_ptr(),
                                       _ptr(count), B, Hkv, T, d, ps, P, mp,
                                       _stream_on(stream, dev))
    if st:
        _check("kv_cache_write", st)


def kv_cache_read(k_cache, v_cache, page_table, start, T: int, count=None, k_descale=None,
                  v_descale=None, out=None, stream=None):
    """(k, v), bf16 [B, Hkv, T, d]: positions start[b] .. start[b] + count[b] - 1
    (default count: T) of each sequence, times their factors; zeros after them.
    Arguments as for kv_cache_write; out: (k, v) to write into."""
    dev = _device_index(k_cache, "k_cache")
    P, Hkv, ps, d, B, mp = _check_cache(k_cache, v_cache, k_descale, v_descale, page_table, dev)
    _check_span(start, count, B, dev)
    shape = (B, Hkv, int(T), d)
    if out is None:
        k = _empty(shape, torch.bfloat16, dev, stream)
        v = _empty(shape, torch.bfloat16, dev, stream)
    else:
        k, v = out
        _check_like(k, "out[0]", shape, torch.bfloat16, dev)
        _check_like(v, "out[1]", shape, torch.bfloat16, dev)
    st = load_library().kv_cache_read(k_cache.data_ptr(), v_cache.data_ptr(), _ptr(k_descale),
                                      _ptr(v_descale), page_table.data_ptr(), start.data_ptr(),
                                      _ptr(count), k.data_ptr(), v.data_ptr(), B, Hkv, int(T), d,
                                      ps, P, mp, _stream_on(stream, dev))
    if st:
        _check("kv_cache_read", st)
    return k, v


def alloc_decode_workspace(d: int, device) -> torch.Tensor:
    """The uint8 device buffer attn_decode needs for head dim d, whatever the
    batch; calls that may overlap on the GPU need one each."""
    n = max(int(load_library().attn_decode_workspace_size(d)), 256)
    return torch.empty(n, dtype=torch.uint8, device=device)


# attn_decode's own workspaces, one for every stream it was called on without
# one: calls on a stream follow one another.  Only for streams that live as long
# as the process, the default one and those of PyTorch's pool, whose handle is
# theirs alone.  Any other owner may destroy its stream, and the handle then be
# another stream's while work of the first still runs; such a call allocates,
# as every call does for its results.  A call that is being captured gets
# memory of its graph, which may replay on any stream.
_decode_workspaces = {}
_PER_THREAD_STREAM = 2  # cudaStreamPerThread: one handle, a stream in every thread


def _decode_workspace(dev: int, stream):
    handle = _stream_on(stream, dev)
    if handle == _PER_THREAD_STREAM:
        # kept or freed and handed out again, it would reach another thread's stream
        raise ValueError("workspace must be given on the per-thread default stream")
    if stream is not None or _capturing():
        n = int(load_library().attn_decode_workspace_size(128))
        return _empty((n,), torch.uint8, dev, stream), handle
    ws = _decode_workspaces.get((dev, handle))
    if ws is None:
        if handle and torch.cuda.current_stream(dev).stream_id == handle:  # not PyTorch's own
            n = int(load_library().attn_decode_workspace_size(128))
            return _empty((n,), torch.uint8, dev, None), handle
        ws = _decode_workspaces[(dev, handle)] = alloc_decode_workspace(128, dev)
    return ws, handle


def attn_decode(q, k_cache, v_cache, page_table, seq_lens, scale=None, k_descale=None,
                v_descale=None, window=0, out=None, lse=None, workspace=None, stream=None):
    """O and the log-sum-exp L of one new token per sequence over a paged cache.

    q: bf16 [B, Hq, 1, d], contiguous, Hq a multiple of the cache's Hkv;
    cache arguments as for kv_cache_write; seq_lens: int32 [B], the sequences'
    lengths with the new token (whose k and v are in the cache already).
    window > 0: only the last ``window`` positions are seen.
    Returns (O bf16 [B, Hq, 1, d], L fp32 [B, Hq, 1]); a sequence of length 0
    has O = 0 and L = -inf.  workspace: from alloc_decode_workspace; without
    one, the call uses one that is kept for its stream (7.5 MB; allocated anew
    on a stream that is not PyTorch's, or in a graph), and is refused on the
    per-thread default stream.
    """
    dev = _device_index(q, "q")
    P, Hkv, ps, d, B, mp = _check_cache(k_cache, v_cache, k_descale, v_descale, page_table, dev)
    Hq = (q.shape if q.dim() == 4 else _shape4(q, "q"))[1]
    shape = (B, Hq, 1, d)
    _check_like(q, "q", shape, torch.bfloat16, dev)
    if Hkv < 1 or Hq % Hkv:
        raise ValueError("q's %d heads must be a multiple of the cache's %d" % (Hq, Hkv))
    _check_like(seq_lens, "seq_lens", (B,), torch.int32, dev)
    if out is None:
        out = torch.empty_like(q) if stream is None else _empty(shape, torch.bfloat16, dev, stream)
    else:
        _check_like(out, "out", shape, torch.bfloat16, dev)
    if lse is None:
        lse = _empty((B, Hq, 1), torch.float32, dev, stream)
    else:
        _check_like(lse, "lse", (B, Hq, 1), torch.float32, dev)
    if workspace is None:
        workspace, handle = _decode_workspace(dev, stream)
    else:
        if not isinstance(workspace, torch.Tensor):
            raise TypeError("workspace must be a torch.Tensor")
        if workspace.get_device() != dev:
            raise ValueError("workspace must be on CUDA device %d, like the first tensor" % dev)
        if not workspace.is_contiguous():  # its bytes would not be its memory
            raise ValueError("workspace must be contiguous")
        handle = _stream_on(stream, dev)
    if k_descale is None:
        kd = vd = None
    else:
        kd, vd = k_descale.data_ptr(), v_descale.data_ptr()
    window = max(-1, min(int(window), _INT_MAX))  # what no length reaches hides nothing
    st = load_library().attn_decode(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), kd, vd,
                                    page_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(),
                                    lse.data_ptr(), B, Hq, Hkv, d, ps, P, mp, window,
                                    _default_scale(d, scale), workspace.data_ptr(),
                                    workspace.nbytes, handle)
    if st:
        _check("attn_decode", st)
    return out, lse
