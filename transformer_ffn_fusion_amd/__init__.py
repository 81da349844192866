"""Fused two-layer FFN (and its grouped MoE form) on AMD Instinct MI355X.

Thin Python binding over ``libffn.so`` (C ABI in ``include/ffn.h``).  The
functions here only marshal torch tensors into pointers, sizes and the
current HIP stream; every step of the computation runs in the library's HIP
kernels.  There is no CPU or PyTorch fallback: if the library is missing, or a
call fails, an exception is raised.

Names mirror the C entry points: ``ffn_forward``, ``ffn_forward_ex``,
``ffn_workspace_size``, ``moe_route``, ``moe_ffn_forward``,
``moe_workspace_size``, ``ffn_last_error``.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "F32", "BF16", "ACT_NONE", "ACT_RELU", "ACT_GELU_TANH",
    "VARIANT_AUTO", "VARIANT_FUSED", "VARIANT_SKINNY", "VARIANT_F32", "VARIANT_DECODE",
    "FFNError", "lib", "lib_path", "ffn_workspace_size", "ffn_forward", "ffn_forward_ex",
    "ffn_forward_family",
    "ffn_forward_noalloc", "NOALLOC_SCRATCH_BYTES",
    "ffn_swiglu_workspace_size", "ffn_swiglu_forward", "ffn_swiglu_backward_workspace_size",
    "ffn_swiglu_backward", "ffn_layernorm_forward", "ffn_layernorm_backward_workspace_size",
    "ffn_layernorm_backward", "ffn_rmsnorm_forward", "ffn_rmsnorm_q8_forward",
    "ffn_rmsnorm_backward_workspace_size", "ffn_rmsnorm_backward",
    "ffn_orthogonalize_workspace_size", "ffn_orthogonalize",
    "moe_workspace_size", "moe_route", "moe_ffn_forward", "ffn_last_error", "workspace",
    "moe_dispatch_workspace_size", "moe_dispatch", "moe_dispatch_backward", "moe_combine",
    "moe_combine_backward", "moe_route_backward", "Q4_INT", "Q4_E2M1", "ffn_q4_bytes", "ffn_q4_empty",
    "ffn_q4_quantize", "ffn_q4_pack", "ffn_q4_matvec", "ffn_q4_swiglu", "moe_q4_matvec", "moe_q4_swiglu",
]

F32, BF16, E4M3 = 0, 1, 2
Q4_INT, Q4_E2M1 = 0, 1
Q4_CODES = {"int4": Q4_INT, "e2m1": Q4_E2M1}
ACT_NONE, ACT_RELU, ACT_GELU_TANH = 0, 1, 2
VARIANT_AUTO, VARIANT_FUSED, VARIANT_SKINNY, VARIANT_F32, VARIANT_DECODE = 0, 1, 2, 3, 4
ACTS = {"none": ACT_NONE, "relu": ACT_RELU, "gelu_tanh": ACT_GELU_TANH}
NOALLOC_SCRATCH_BYTES = 16 << 20   # FFN_NOALLOC_SCRATCH_BYTES in include/ffn.h

_PKG = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_PKG, "libffn.so")
_lib = None


class FFNError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libffn error {code}: {msg}")
        self.code = code


def lib():
    """The loaded libffn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise FFNError(-100, f"{lib_path} is missing; run `python -m transformer_ffn_fusion_amd.build`")
        L = ctypes.CDLL(lib_path)
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        L.ffn_workspace_size.argtypes = [i64, i64, i64, i64, i32]
        L.ffn_workspace_size.restype = sz
        L.ffn_workspace_size_ex.argtypes = [i64, i64, i64, i64, i32, i32]
        L.ffn_workspace_size_ex.restype = sz
        L.ffn_forward_family.argtypes = [i64, i64, i64, i64, i32, i32]
        L.ffn_forward_family.restype = i32
        L.ffn_forward.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i32, i32, i32, vp, sz, vp]
        L.ffn_forward.restype = i32
        L.ffn_forward_ex.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i32, i32, i32, i32,
                                     vp, sz, vp]
        L.ffn_forward_ex.restype = i32
        L.ffn_forward_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i32, i32,
                                          i32, i32, vp]
        L.ffn_forward_noalloc.restype = i32
        L.moe_workspace_size.argtypes = [i64, i64, i32, i64, i64, i64, i32]
        L.moe_workspace_size.restype = sz
        L.moe_route.argtypes = [vp, i64, i64, i32, vp, vp, vp, vp, vp, sz, vp]
        L.moe_route.restype = i32
        L.moe_ffn_forward.argtypes = [vp, vp, i64, i64, i32, vp, vp, vp, vp, vp, i64, i64, i64, i32,
                                      i32, i32, vp, vp, vp, vp, vp, sz, vp]
        L.moe_ffn_forward.restype = i32
        evp = ctypes.POINTER(ctypes.c_void_p)
        L.ffn_forward_traced.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i32, i32, i32,
                                         i32, vp, sz, vp, evp, i32]
        L.ffn_forward_traced.restype = i32
        L.moe_ffn_forward_traced.argtypes = [vp, vp, i64, i64, i32, vp, vp, vp, vp, vp, i64, i64,
                                             i64, i32, i32, i32, vp, sz, vp, evp, i32]
        L.moe_ffn_forward_traced.restype = i32
        L.ffn_swiglu_workspace_size.argtypes = [i64, i64, i64, i64, i32, i32]
        L.ffn_swiglu_workspace_size.restype = sz
        L.ffn_swiglu_forward.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i32, i32, vp, sz, vp]
        L.ffn_swiglu_forward.restype = i32
        L.ffn_swiglu_forward_traced.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i32, i32, vp,
                                                sz, vp, ctypes.POINTER(vp), i32]
        L.ffn_swiglu_forward_traced.restype = i32
        L.moe_router.argtypes = [vp, vp, vp, i64, i64, i64, i32, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_router.restype = i32
        L.moe_ffn_forward_router.argtypes = [vp, vp, vp, i64, i64, i32, vp, vp, vp, vp, vp, i64, i64,
                                             i64, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_ffn_forward_router.restype = i32
        L.ffn_backward_workspace_size.argtypes = [i64, i64, i64, i64, i32]
        L.ffn_backward_workspace_size.restype = sz
        L.ffn_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i32,
                                   i32, vp, sz, vp]
        L.ffn_backward.restype = i32
        L.ffn_backward_traced.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64,
                                          i32, i32, vp, sz, vp, ctypes.POINTER(vp), i32]
        L.ffn_backward_traced.restype = i32
        L.ffn_swiglu_backward_workspace_size.argtypes = [i64, i64, i64, i64, i32]
        L.ffn_swiglu_backward_workspace_size.restype = sz
        L.ffn_swiglu_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64,
                                          i32, i32, vp, sz, vp]
        L.ffn_swiglu_backward.restype = i32
        L.ffn_layernorm_forward.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i32, ctypes.c_float, vp]
        L.ffn_layernorm_forward.restype = i32
        L.ffn_layernorm_backward_workspace_size.argtypes = [i64, i64, i32]
        L.ffn_layernorm_backward_workspace_size.restype = sz
        L.ffn_layernorm_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i32, vp, sz, vp]
        L.ffn_layernorm_backward.restype = i32
        L.ffn_rmsnorm_forward.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i32, ctypes.c_float, vp]
        L.ffn_rmsnorm_forward.restype = i32
        L.ffn_rmsnorm_q8_forward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, ctypes.c_float, vp]
        L.ffn_rmsnorm_q8_forward.restype = i32
        L.ffn_rmsnorm_backward_workspace_size.argtypes = [i64, i64, i32]
        L.ffn_rmsnorm_backward_workspace_size.restype = sz
        L.ffn_rmsnorm_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i32, vp, sz, vp]
        L.ffn_rmsnorm_backward.restype = i32
        L.moe_dispatch_workspace_size.argtypes = [i64, i64, i32]
        L.moe_dispatch_workspace_size.restype = sz
        L.moe_dispatch.argtypes = [vp, vp, vp, i64, i64, i64, i32, i32, i64, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_dispatch.restype = i32
        L.moe_dispatch_backward.argtypes = [vp, vp, vp, i64, i64, i32, i64, i32, vp]
        L.moe_dispatch_backward.restype = i32
        L.moe_combine.argtypes = [vp, vp, vp, vp, vp, i64, i64, i32, i64, i32, vp]
        L.moe_combine.restype = i32
        L.moe_combine_backward.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i32, i64, i32, vp]
        L.moe_combine_backward.restype = i32
        L.moe_route_backward.argtypes = [vp, vp, vp, vp, i64, i64, i32, vp]
        L.moe_route_backward.restype = i32
        L.ffn_q4_bytes.argtypes = [i64, i64]
        L.ffn_q4_bytes.restype = sz
        L.ffn_q4_matvec.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, i32, vp]
        L.ffn_q4_matvec.restype = i32
        L.ffn_q4_swiglu.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, vp]
        L.ffn_q4_swiglu.restype = i32
        L.moe_q4_matvec.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i32, i32, i32, vp]
        L.moe_q4_matvec.restype = i32
        L.moe_q4_swiglu.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i32, i32, vp]
        L.moe_q4_swiglu.restype = i32
        L.ffn_q4_quantize.argtypes = [vp, vp, vp, vp, i64, i64, i32, i32, i32, vp]
        L.ffn_q4_quantize.restype = i32
        L.ffn_q4_pack.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, vp]
        L.ffn_q4_pack.restype = i32
        L.ffn_orthogonalize_workspace_size.argtypes = [i64, i64, i64, i32]
        L.ffn_orthogonalize_workspace_size.restype = sz
        L.ffn_orthogonalize.argtypes = [vp, vp, i64, i64, i64, i32, i32, vp, sz, vp]
        L.ffn_orthogonalize.restype = i32
        L.ffn_last_error.argtypes = []
        L.ffn_last_error.restype = ctypes.c_char_p
        L.ffn_version.restype = i32
        L.ffn_selftest_layout.restype = i32
        L.ffn_selftest_decode_expiry.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i32,
                                                 i32, vp, sz, vp]
        L.ffn_selftest_decode_expiry.restype = i32
        L.ffn_ceiling_sink_bytes.argtypes = []
        L.ffn_ceiling_sink_bytes.restype = sz
        L.ffn_ceiling_mfma.argtypes = [vp, sz, i32, ctypes.POINTER(ctypes.c_double), vp]
        L.ffn_ceiling_mfma.restype = i32
        L.ffn_ceiling_read.argtypes = [vp, sz, vp, sz, vp]
        L.ffn_ceiling_read.restype = i32
        _lib = L
    return _lib


def ffn_last_error() -> str:
    return lib().ffn_last_error().decode()


def _check(rc: int):
    if rc != 0:
        raise FFNError(rc, ffn_last_error())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream
    import torch
    # the current stream's handle, without building a Stream object per call
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _act(a):
    return ACTS[a] if isinstance(a, str) else int(a)


# ---------------------------------------------------------------- argument checks
#
# The library receives raw pointers and sizes only, so a tensor of the wrong
# shape, dtype or layout would make its kernels read or write out of bounds.
# Every wrapper checks its tensors here before anything reaches the library.

def _dims(t, name, ndim):
    if t is None:
        raise ValueError(f"{name} must not be None")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions (got shape {tuple(t.shape)})")
    return tuple(t.shape)


def _arg(t, name, shape, dtype, optional=False):
    """One tensor argument: shape, dtype and row-major contiguity."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} must not be None")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")


def _ws_arg(ws):
    import torch
    if ws is None:
        return
    if ws.dtype != torch.uint8 or ws.dim() != 1 or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous 1-D uint8 tensor")


def _on_device(*ts):
    """Every given tensor on the current GPU (the library launches there)."""
    import torch
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"every tensor must be on the GPU (got one on {t.device})")
        i = t.get_device()
        if dev is None:
            dev = i
        elif i != dev:
            raise ValueError(f"tensors on different devices (cuda:{dev} and cuda:{i})")
    if dev is not None and dev != torch.cuda.current_device():
        raise ValueError(f"tensors are on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")


def _torch_dtype(code):
    import torch
    return torch.bfloat16 if code == BF16 else torch.float32


def _tensors(need, may=()):
    """Checks (tensor, name, shape, dtype) as ``_arg`` and ``_on_device`` do, in one pass for calls of a few
    microseconds; ``may``: those that may be None.  Returns the device's index."""
    import torch
    good = torch.cuda.is_initialized()
    dev = torch._C._cuda_getDevice() if good else -1
    for t, name, shape, dtype in need:
        if t is None or t.shape != shape or t.dtype is not dtype or not t.is_contiguous() or t.get_device() != dev:
            good = False
    for t, name, shape, dtype in may:
        if t is not None and (t.shape != shape or t.dtype is not dtype or not t.is_contiguous()
                              or t.get_device() != dev):
            good = False
    if not good:      # which one, and why
        for spec in need:
            _arg(*spec)
        for spec in may:
            _arg(*spec, optional=True)
        _on_device(*(s[0] for s in (*need, *may)))
    return dev


def _stream_of(stream, dev):
    """The call's stream: the given one, or the current one of the device that its tensors are on."""
    if stream is not None:
        return stream
    import torch
    return torch._C._cuda_getCurrentRawStream(dev)


def ffn_workspace_size(M, N, O, P, dtype=BF16, variant=VARIANT_AUTO) -> int:
    return lib().ffn_workspace_size_ex(M, N, O, P, dtype, variant)


def moe_workspace_size(M, E, k, N, O, P, dtype=BF16) -> int:
    return lib().moe_workspace_size(M, E, k, N, O, P, dtype)


def ffn_forward_family(M, N, O, P, dtype=BF16, variant=VARIANT_AUTO) -> int:
    """The kernel family (VARIANT_FUSED, _SKINNY, _F32 or _DECODE) that ``ffn_forward_ex``
    runs for this shape on the current device."""
    rc = lib().ffn_forward_family(M, N, O, P, dtype, variant)
    if rc < 0:
        raise FFNError(rc, ffn_last_error())
    return rc


def workspace(nbytes: int, device="cuda"):
    """A zero-filled device workspace of ``nbytes`` (torch allocations are 256-byte aligned)."""
    import torch
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _own_workspace(nbytes, device, stream):
    """The workspace of a call that brings none, allocated and filled on the stream that the call
    runs on: on another one the fill could come after the kernels' first writes, and the memory
    could be given to other work before the last ones."""
    import torch
    if stream is not None:
        stream = getattr(stream, "value", stream) or 0   # (a ctypes handle; NULL's value is None)
    if stream is None or stream == _stream(None):
        return workspace(nbytes, device)
    on = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(on):
        return workspace(nbytes, device)


def _dense_args(X, W1, b1, W2, b2, Y, ws=None):
    """Checks the dense call's tensors; returns M, N, O, P and the dtype code."""
    M, N = _dims(X, "X", 2)
    O = _dims(W1, "W1", 2)[1]
    P = _dims(W2, "W2", 2)[1]
    dt = _dtype_code(X)
    tdt = _torch_dtype(dt)
    _arg(X, "X", (M, N), tdt)
    _arg(W1, "W1", (N, O), tdt)
    _arg(b1, "b1", (O,), tdt, optional=True)
    _arg(W2, "W2", (O, P), tdt)
    _arg(b2, "b2", (P,), tdt, optional=True)
    _arg(Y, "Y", (M, P), tdt)
    _ws_arg(ws)
    _on_device(X, W1, b1, W2, b2, Y, ws)
    return M, N, O, P, dt


def ffn_forward_noalloc(X, W1, b1, W2, b2, Y, act1="gelu_tanh", act2="none",
                        variant=VARIANT_AUTO, stream=None):
    """As ``ffn_forward_ex`` with the library's static device scratch as the workspace:
    nothing is allocated (the shape's workspace must fit FFN_NOALLOC_SCRATCH_BYTES)."""
    M, N, O, P, dt = _dense_args(X, W1, b1, W2, b2, Y)
    _check(lib().ffn_forward_noalloc(_ptr(X), _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2), _ptr(Y),
                                     M, N, O, P, dt, _act(act1), _act(act2), int(variant),
                                     _stream(stream)))
    return Y


def ffn_forward_ex(X, W1, b1, W2, b2, Y, act1="gelu_tanh", act2="none", variant=VARIANT_AUTO,
                   ws=None, stream=None):
    """``Y = act2(act1(X W1 + b1) W2 + b2)`` on the GPU; ``Y`` is written in place.

    ``ws`` is a zero-initialised uint8 device tensor of at least
    ``ffn_workspace_size(...)`` bytes (allocated here when None)."""
    M, N, O, P, dt = _dense_args(X, W1, b1, W2, b2, Y, ws)
    if ws is None:
        ws = _own_workspace(ffn_workspace_size(M, N, O, P, dt, variant), X.device, stream)
    _check(lib().ffn_forward_ex(_ptr(X), _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2), _ptr(Y),
                                M, N, O, P, dt, _act(act1), _act(act2), int(variant),
                                _ptr(ws), ws.numel(), _stream(stream)))
    return Y


def ffn_forward(X, W1, b1, W2, b2, Y, act1="gelu_tanh", act2="none", ws=None, stream=None):
    return ffn_forward_ex(X, W1, b1, W2, b2, Y, act1, act2, VARIANT_AUTO, ws, stream)


def ffn_backward_workspace_size(M, N, O, P, dtype=BF16) -> int:
    return lib().ffn_backward_workspace_size(M, N, O, P, dtype)


def ffn_backward(X, W1, b1, W2, dY, dX, dW1, db1, dW2, db2, act1="gelu_tanh", ws=None, stream=None):
    """Gradients of the FFN (act2 none) for the output gradient ``dY``; writes dX (bf16),
    dW1, db1, dW2, db2 (fp32; db1/db2 may be None) in place."""
    import torch
    M, N = _dims(X, "X", 2)
    O = _dims(W1, "W1", 2)[1]
    P = _dims(W2, "W2", 2)[1]
    dt = _dtype_code(X)
    bf, f32 = torch.bfloat16, torch.float32
    _arg(X, "X", (M, N), bf)
    _arg(W1, "W1", (N, O), bf)
    _arg(b1, "b1", (O,), bf, optional=True)
    _arg(W2, "W2", (O, P), bf)
    _arg(dY, "dY", (M, P), bf)
    _arg(dX, "dX", (M, N), bf)
    _arg(dW1, "dW1", (N, O), f32)
    _arg(db1, "db1", (O,), f32, optional=True)
    _arg(dW2, "dW2", (O, P), f32)
    _arg(db2, "db2", (P,), f32, optional=True)
    _ws_arg(ws)
    _on_device(X, W1, b1, W2, dY, dX, dW1, db1, dW2, db2, ws)
    if ws is None:
        ws = _own_workspace(ffn_backward_workspace_size(M, N, O, P, dt), X.device, stream)
    _check(lib().ffn_backward(_ptr(X), _ptr(W1), _ptr(b1), _ptr(W2), _ptr(dY), _ptr(dX), _ptr(dW1),
                              _ptr(db1), _ptr(dW2), _ptr(db2), M, N, O, P, dt, _act(act1),
                              _ptr(ws), ws.numel(), _stream(stream)))


def ffn_swiglu_workspace_size(M, N, O, P, dtype=BF16, variant=VARIANT_AUTO) -> int:
    return lib().ffn_swiglu_workspace_size(M, N, O, P, dtype, variant)


def ffn_swiglu_forward(X, Wg, Wu, Wd, Y, variant=VARIANT_AUTO, ws=None, stream=None):
    """``Y = (silu(X Wg) * (X Wu)) Wd`` on the GPU; ``Y`` is written in place."""
    M, N = _dims(X, "X", 2)
    O = _dims(Wg, "Wg", 2)[1]
    P = _dims(Wd, "Wd", 2)[1]
    dt = _dtype_code(X)
    tdt = _torch_dtype(dt)
    _arg(X, "X", (M, N), tdt)
    _arg(Wg, "Wg", (N, O), tdt)
    _arg(Wu, "Wu", (N, O), tdt)
    _arg(Wd, "Wd", (O, P), tdt)
    _arg(Y, "Y", (M, P), tdt)
    _ws_arg(ws)
    _on_device(X, Wg, Wu, Wd, Y, ws)
    if ws is None:
        ws = _own_workspace(ffn_swiglu_workspace_size(M, N, O, P, dt, variant), X.device, stream)
    _check(lib().ffn_swiglu_forward(_ptr(X), _ptr(Wg), _ptr(Wu), _ptr(Wd), _ptr(Y), M, N, O, P,
                                    dt, int(variant), _ptr(ws), ws.numel(), _stream(stream)))
    return Y


def ffn_swiglu_backward_workspace_size(M, N, O, P, dtype=BF16) -> int:
    return lib().ffn_swiglu_backward_workspace_size(M, N, O, P, dtype)


def ffn_swiglu_backward(X, Wg, Wu, Wd, dY, dX, dWg, dWu, dWd, ws=None, stream=None):
    """Gradients of ``ffn_swiglu_forward`` for the output gradient ``dY``; writes dX (bf16) and
    dWg, dWu, dWd (all bf16 or all fp32) in place.  Every input is bf16."""
    import torch
    M, N = _dims(X, "X", 2)
    O = _dims(Wg, "Wg", 2)[1]
    P = _dims(Wd, "Wd", 2)[1]
    bf = torch.bfloat16
    _arg(X, "X", (M, N), bf)
    _arg(Wg, "Wg", (N, O), bf)
    _arg(Wu, "Wu", (N, O), bf)
    _arg(Wd, "Wd", (O, P), bf)
    _arg(dY, "dY", (M, P), bf)
    _arg(dX, "dX", (M, N), bf)
    _dims(dWg, "dWg", 2)
    gdt = _dtype_code(dWg)
    _arg(dWg, "dWg", (N, O), dWg.dtype)
    _arg(dWu, "dWu", (N, O), dWg.dtype)
    _arg(dWd, "dWd", (O, P), dWg.dtype)
    _ws_arg(ws)
    _on_device(X, Wg, Wu, Wd, dY, dX, dWg, dWu, dWd, ws)
    if ws is None:
        ws = _own_workspace(ffn_swiglu_backward_workspace_size(M, N, O, P), X.device, stream)
    _check(lib().ffn_swiglu_backward(_ptr(X), _ptr(Wg), _ptr(Wu), _ptr(Wd), _ptr(dY), _ptr(dX),
                                     _ptr(dWg), _ptr(dWu), _ptr(dWd), M, N, O, P, BF16, gdt,
                                     _ptr(ws), ws.numel(), _stream(stream)))


def ffn_layernorm_forward(X, gamma, beta, Y, mean=None, rstd=None, eps=1e-5, stream=None):
    """``Y = (X - mean) rstd gamma + beta`` over the last dimension of X (M x N, bf16 or fp32);
    ``Y`` and, when given, ``mean`` and ``rstd`` (M, fp32) are written in place."""
    import torch
    M, N = _dims(X, "X", 2)
    dt = _dtype_code(X)
    _arg(X, "X", (M, N), X.dtype)
    _arg(gamma, "gamma", (N,), X.dtype)
    _arg(beta, "beta", (N,), X.dtype)
    _arg(Y, "Y", (M, N), X.dtype)
    _arg(mean, "mean", (M,), torch.float32, optional=True)
    _arg(rstd, "rstd", (M,), torch.float32, optional=True)
    _on_device(X, gamma, beta, Y, mean, rstd)
    _check(lib().ffn_layernorm_forward(_ptr(X), _ptr(gamma), _ptr(beta), _ptr(Y), _ptr(mean),
                                       _ptr(rstd), M, N, dt, float(eps), _stream(stream)))
    return Y


def ffn_layernorm_backward_workspace_size(M, N, dtype=BF16) -> int:
    return lib().ffn_layernorm_backward_workspace_size(M, N, dtype)


def ffn_layernorm_backward(X, dY, gamma, mean, rstd, dX, dgamma, dbeta, ws=None, stream=None):
    """Gradients of ``ffn_layernorm_forward``: dX in X's type, dgamma and dbeta (N, fp32), written
    in place.  ``mean`` and ``rstd`` are what the forward wrote."""
    import torch
    M, N = _dims(X, "X", 2)
    dt = _dtype_code(X)
    f32 = torch.float32
    _arg(X, "X", (M, N), X.dtype)
    _arg(dY, "dY", (M, N), X.dtype)
    _arg(gamma, "gamma", (N,), X.dtype)
    _arg(mean, "mean", (M,), f32)
    _arg(rstd, "rstd", (M,), f32)
    _arg(dX, "dX", (M, N), X.dtype)
    _arg(dgamma, "dgamma", (N,), f32)
    _arg(dbeta, "dbeta", (N,), f32)
    _ws_arg(ws)
    _on_device(X, dY, gamma, mean, rstd, dX, dgamma, dbeta, ws)
    if ws is None:
        ws = _own_workspace(ffn_layernorm_backward_workspace_size(M, N, dt), X.device, stream)
    _check(lib().ffn_layernorm_backward(_ptr(X), _ptr(dY), _ptr(gamma), _ptr(mean), _ptr(rstd),
                                        _ptr(dX), _ptr(dgamma), _ptr(dbeta), M, N, dt, _ptr(ws),
                                        ws.numel(), _stream(stream)))


def _rmsnorm_args(X, gamma, R, S, rstd, *more):
    import torch
    M, N = _dims(X, "X", 2)
    dt = _dtype_code(X)
    if (R is None) != (S is None):
        raise ValueError("S is written with R alone: give both or neither")
    full, d = (M, N), X.dtype
    dev = _tensors(((X, "X", full, d), (gamma, "gamma", (N,), d), *more),
                   ((R, "R", full, d), (S, "S", full, d), (rstd, "rstd", (M,), torch.float32)))
    return M, N, dt, dev


def ffn_rmsnorm_forward(X, gamma, Y, R=None, S=None, rstd=None, eps=1e-5, stream=None):
    """``S = X + R`` (where a residual ``R`` is given) and ``Y = S rstd gamma`` over the last dimension
    (M x N, bf16 or fp32); ``S``, ``Y`` and, when given, ``rstd`` (M, fp32) are written in place."""
    M, N, dt, dev = _rmsnorm_args(X, gamma, R, S, rstd, (Y, "Y", X.shape, X.dtype))
    _check(lib().ffn_rmsnorm_forward(X.data_ptr(), _ptr(R), gamma.data_ptr(), _ptr(S), Y.data_ptr(), _ptr(rstd), M, N,
                                     dt, float(eps), _stream_of(stream, dev)))
    return Y


def ffn_rmsnorm_q8_forward(X, gamma, Q, scale, R=None, S=None, rstd=None, group=128, eps=1e-5, stream=None):
    """As ``ffn_rmsnorm_forward`` with the output as e4m3 codes ``Q`` (M x N, float8_e4m3fn) and fp32
    ``scale``: M x ceil(N / 128) for groups of 128 columns, M x 1 for whole rows (``group=0``)."""
    import torch
    if group not in (0, 128):
        raise ValueError(f"group must be 128, or 0 for whole rows (got {group})")
    M, N = _dims(X, "X", 2)
    M, N, dt, dev = _rmsnorm_args(X, gamma, R, S, rstd, (Q, "Q", X.shape, torch.float8_e4m3fn),
                                  (scale, "scale", (M, -(-N // group) if group else 1), torch.float32))
    _check(lib().ffn_rmsnorm_q8_forward(X.data_ptr(), _ptr(R), gamma.data_ptr(), _ptr(S), Q.data_ptr(),
                                        scale.data_ptr(), _ptr(rstd), M, N, dt, group, float(eps),
                                        _stream_of(stream, dev)))
    return Q


def ffn_rmsnorm_backward_workspace_size(M, N, dtype=BF16) -> int:
    return lib().ffn_rmsnorm_backward_workspace_size(M, N, dtype)


def ffn_rmsnorm_backward(S, dY, gamma, rstd, dX, dgamma, dS=None, ws=None, stream=None):
    """Gradients of ``ffn_rmsnorm_forward``: dX (of X and of R alike) in S's type, dgamma (N, fp32),
    written in place.  ``S`` is the normed sum (X without a residual), ``rstd`` what the forward wrote,
    ``dS`` the gradient that reaches S by the residual path."""
    import torch
    M, N = _dims(S, "S", 2)
    dt = _dtype_code(S)
    f32, full, d = torch.float32, (M, N), S.dtype
    _ws_arg(ws)
    dev = _tensors(((S, "S", full, d), (dY, "dY", full, d), (gamma, "gamma", (N,), d), (rstd, "rstd", (M,), f32),
                    (dX, "dX", full, d), (dgamma, "dgamma", (N,), f32)),
                   ((dS, "dS", full, d), (ws, "ws", () if ws is None else ws.shape, torch.uint8)))
    if ws is None:
        ws = _own_workspace(ffn_rmsnorm_backward_workspace_size(M, N, dt), S.device, stream)
    _check(lib().ffn_rmsnorm_backward(S.data_ptr(), dY.data_ptr(), _ptr(dS), gamma.data_ptr(), rstd.data_ptr(),
                                      dX.data_ptr(), dgamma.data_ptr(), M, N, dt, ws.data_ptr(), ws.numel(),
                                      _stream_of(stream, dev)))


def ffn_orthogonalize_workspace_size(B, R, C, dtype=BF16) -> int:
    return lib().ffn_orthogonalize_workspace_size(B, R, C, dtype)


def ffn_orthogonalize(G, U, steps=5, ws=None, stream=None):
    """Newton-Schulz orthogonalisation of a gradient ``G`` (R x C, or a stack B x R x C; bf16 or
    fp32) in ``steps`` (1 to 8) steps; ``U`` (the same shape, bf16) is written in place."""
    import torch
    if G is None:
        raise ValueError("G must not be None")
    if G.dim() not in (2, 3):
        raise ValueError(f"G must have 2 or 3 dimensions (got shape {tuple(G.shape)})")
    B, R, C = (1, *G.shape) if G.dim() == 2 else G.shape
    dt = _dtype_code(G)
    _arg(G, "G", G.shape, G.dtype)
    _arg(U, "U", G.shape, torch.bfloat16)
    _ws_arg(ws)
    _on_device(G, U, ws)
    if ws is None:
        ws = _own_workspace(ffn_orthogonalize_workspace_size(B, R, C, dt), G.device, stream)
    _check(lib().ffn_orthogonalize(_ptr(G), _ptr(U), B, R, C, dt, int(steps), _ptr(ws), ws.numel(),
                                   _stream(stream)))
    return U


def _route_outputs(M, E, k, topk_ids, topk_w, expert_offsets, sorted_entries):
    import torch
    _arg(topk_ids, "topk_ids", (M, k), torch.int32, optional=True)
    _arg(topk_w, "topk_w", (M, k), torch.float32, optional=True)
    _arg(expert_offsets, "expert_offsets", (E + 1,), torch.int32, optional=True)
    _arg(sorted_entries, "sorted_entries", (M * k,), torch.int32, optional=True)


def _experts(X, W1, b1, W2, b2, Y):
    """Shapes of the grouped form's tensors: returns M, N, E, O, P."""
    M, N = _dims(X, "X", 2)
    E, _, O = _dims(W1, "W1", 3)
    P = _dims(W2, "W2", 3)[2]
    bf = _torch_dtype(BF16)
    if X.dtype != bf:
        raise TypeError(f"X has dtype {X.dtype}; the grouped form takes bfloat16")
    _arg(X, "X", (M, N), bf)
    _arg(W1, "W1", (E, N, O), bf)
    _arg(b1, "b1", (E, O), bf, optional=True)
    _arg(W2, "W2", (E, O, P), bf)
    _arg(b2, "b2", (E, P), bf, optional=True)
    _arg(Y, "Y", (M, P), bf)
    return M, N, E, O, P


def moe_route(logits, k, topk_ids=None, topk_w=None, expert_offsets=None, sorted_entries=None,
              ws=None, stream=None):
    """Top-k routing on the GPU; fills whichever output tensors are given."""
    import torch
    M, E = _dims(logits, "logits", 2)
    _arg(logits, "logits", (M, E), torch.float32)
    _route_outputs(M, E, k, topk_ids, topk_w, expert_offsets, sorted_entries)
    _ws_arg(ws)
    _on_device(logits, topk_ids, topk_w, expert_offsets, sorted_entries, ws)
    if ws is None:
        ws = _own_workspace(moe_workspace_size(M, E, k, 8, 8, 8), logits.device, stream)
    _check(lib().moe_route(_ptr(logits), M, E, k, _ptr(topk_ids), _ptr(topk_w),
                           _ptr(expert_offsets), _ptr(sorted_entries), _ptr(ws), ws.numel(),
                           _stream(stream)))


def moe_ffn_forward(X, logits, k, W1, b1, W2, b2, Y, act1="gelu_tanh", act2="none",
                    topk_ids=None, topk_w=None, expert_offsets=None, sorted_entries=None,
                    ws=None, stream=None):
    """Grouped FFN over the top-k experts of each token; ``Y`` written in place."""
    import torch
    M, N, E, O, P = _experts(X, W1, b1, W2, b2, Y)
    _arg(logits, "logits", (M, E), torch.float32)
    _route_outputs(M, E, k, topk_ids, topk_w, expert_offsets, sorted_entries)
    _ws_arg(ws)
    _on_device(X, logits, W1, b1, W2, b2, Y, topk_ids, topk_w, expert_offsets, sorted_entries, ws)
    dt = BF16
    if ws is None:
        ws = _own_workspace(moe_workspace_size(M, E, k, N, O, P, dt), X.device, stream)
    _check(lib().moe_ffn_forward(_ptr(X), _ptr(logits), M, E, k, _ptr(W1), _ptr(b1), _ptr(W2),
                                 _ptr(b2), _ptr(Y), N, O, P, dt, _act(act1), _act(act2),
                                 _ptr(topk_ids), _ptr(topk_w), _ptr(expert_offsets),
                                 _ptr(sorted_entries), _ptr(ws), ws.numel(), _stream(stream)))
    return Y


def moe_router(X, Wr, br, k, logits_out=None, topk_ids=None, topk_w=None, expert_offsets=None,
               sorted_entries=None, ws=None, stream=None):
    """Router logits X Wr + br and top-k routing on the GPU; fills the given outputs."""
    import torch
    M, N = _dims(X, "X", 2)
    E = _dims(Wr, "Wr", 2)[1]
    _arg(X, "X", (M, N), torch.bfloat16)
    _arg(Wr, "Wr", (N, E), torch.bfloat16)
    _arg(br, "br", (E,), torch.float32, optional=True)
    _arg(logits_out, "logits_out", (M, E), torch.float32, optional=True)
    _route_outputs(M, E, k, topk_ids, topk_w, expert_offsets, sorted_entries)
    _ws_arg(ws)
    _on_device(X, Wr, br, logits_out, topk_ids, topk_w, expert_offsets, sorted_entries, ws)
    if ws is None:
        ws = _own_workspace(moe_workspace_size(M, E, k, N, 8, 8), X.device, stream)
    _check(lib().moe_router(_ptr(X), _ptr(Wr), _ptr(br), M, N, E, k, _ptr(logits_out),
                            _ptr(topk_ids), _ptr(topk_w), _ptr(expert_offsets),
                            _ptr(sorted_entries), _ptr(ws), ws.numel(), _stream(stream)))


def moe_ffn_forward_router(X, Wr, br, k, W1, b1, W2, b2, Y, act1="gelu_tanh", act2="none",
                           logits_out=None, topk_ids=None, topk_w=None, expert_offsets=None,
                           sorted_entries=None, ws=None, stream=None):
    """The MoE layer with the router on the GPU; ``Y`` written in place."""
    import torch
    M, N, E, O, P = _experts(X, W1, b1, W2, b2, Y)
    _arg(Wr, "Wr", (N, E), torch.bfloat16)
    _arg(br, "br", (E,), torch.float32, optional=True)
    _arg(logits_out, "logits_out", (M, E), torch.float32, optional=True)
    _route_outputs(M, E, k, topk_ids, topk_w, expert_offsets, sorted_entries)
    _ws_arg(ws)
    _on_device(X, Wr, br, W1, b1, W2, b2, Y, logits_out, topk_ids, topk_w, expert_offsets,
               sorted_entries, ws)
    dt = BF16
    if ws is None:
        ws = _own_workspace(moe_workspace_size(M, E, k, N, O, P, dt), X.device, stream)
    _check(lib().moe_ffn_forward_router(_ptr(X), _ptr(Wr), _ptr(br), M, E, k, _ptr(W1), _ptr(b1),
                                        _ptr(W2), _ptr(b2), _ptr(Y), N, O, P, dt, _act(act1),
                                        _act(act2), _ptr(logits_out), _ptr(topk_ids), _ptr(topk_w),
                                        _ptr(expert_offsets), _ptr(sorted_entries), _ptr(ws),
                                        ws.numel(), _stream(stream)))
    return Y


# ---------------------------------------------------------------- rows by expert and back

def moe_dispatch_workspace_size(M, E, k) -> int:
    return lib().moe_dispatch_workspace_size(M, E, k)


def moe_dispatch(X, topk_ids, Xs, expert_offsets, sorted_entries, positions, scale=None, scale_sorted=None,
                 ws=None, stream=None):
    """Tokens sorted by expert: entry ``t * k + s`` of ``topk_ids`` (M x k, int32; ids outside [0, E) are
    dropped) goes to row ``positions[t, s]`` (-1: dropped) of ``Xs`` (M*k x N), whose rows of expert e are
    ``expert_offsets[e]`` to ``expert_offsets[e + 1]`` (E + 1, int32) and come from ``sorted_entries``
    (M*k, int32).  X is bf16, fp32 or float8_e4m3fn; ``scale`` (M x G, fp32) travels with the rows.  Rows
    behind the last kept entry are left as they were."""
    import torch
    M, N = _dims(X, "X", 2)
    k = _dims(topk_ids, "topk_ids", 2)[1]
    E = _dims(expert_offsets, "expert_offsets", 1)[0] - 1
    i32 = torch.int32
    dt = E4M3 if X.dtype == torch.float8_e4m3fn else _dtype_code(X)
    if (scale is None) != (scale_sorted is None):
        raise ValueError("give scale and scale_sorted together or neither")
    G = 0
    if scale is not None:
        G = _dims(scale, "scale", 2)[1]
        if G < 1:
            raise ValueError("scale must have columns")
    _ws_arg(ws)
    dev = _tensors(((X, "X", (M, N), X.dtype), (topk_ids, "topk_ids", (M, k), i32), (Xs, "Xs", (M * k, N), X.dtype),
                    (expert_offsets, "expert_offsets", (E + 1,), i32),
                    (sorted_entries, "sorted_entries", (M * k,), i32), (positions, "positions", (M, k), i32)),
                   ((scale, "scale", (M, G), torch.float32), (scale_sorted, "scale_sorted", (M * k, G), torch.float32),
                    (ws, "ws", () if ws is None else ws.shape, torch.uint8)))
    if ws is None:
        ws = _own_workspace(moe_dispatch_workspace_size(M, E, k), X.device, stream)
    _check(lib().moe_dispatch(X.data_ptr(), topk_ids.data_ptr(), _ptr(scale), M, N, E, k, dt, G, Xs.data_ptr(),
                              _ptr(scale_sorted), expert_offsets.data_ptr(), sorted_entries.data_ptr(),
                              positions.data_ptr(), ws.data_ptr(), ws.numel(), _stream_of(stream, dev)))
    return Xs


def moe_dispatch_backward(dXs, positions, dX, stream=None):
    """``dX[t] = sum_s dXs[positions[t, s]]``, the gradient of ``moe_dispatch``; written in place."""
    import torch
    M, N = _dims(dX, "dX", 2)
    k = _dims(positions, "positions", 2)[1]
    dt = _dtype_code(dX)
    rows = _dims(dXs, "dXs", 2)[0]
    dev = _tensors(((dXs, "dXs", (rows, N), dX.dtype), (positions, "positions", (M, k), torch.int32),
                    (dX, "dX", (M, N), dX.dtype)))
    _check(lib().moe_dispatch_backward(dXs.data_ptr(), positions.data_ptr(), dX.data_ptr(), M, N, k, rows, dt,
                                       _stream_of(stream, dev)))
    return dX


def moe_combine(Ys, positions, Y, topk_w=None, R=None, stream=None):
    """``Y[t] = R[t] + sum_s topk_w[t, s] Ys[positions[t, s]]`` (weights of 1 and no residual where they are
    None; dropped entries add nothing); ``Y`` is written in place."""
    import torch
    M, N = _dims(Y, "Y", 2)
    k = _dims(positions, "positions", 2)[1]
    dt = _dtype_code(Y)
    rows = _dims(Ys, "Ys", 2)[0]
    dev = _tensors(((Ys, "Ys", (rows, N), Y.dtype), (positions, "positions", (M, k), torch.int32),
                    (Y, "Y", (M, N), Y.dtype)),
                   ((topk_w, "topk_w", (M, k), torch.float32), (R, "R", (M, N), Y.dtype)))
    _check(lib().moe_combine(Ys.data_ptr(), positions.data_ptr(), _ptr(topk_w), _ptr(R), Y.data_ptr(), M, N, k, rows,
                             dt, _stream_of(stream, dev)))
    return Y


def moe_combine_backward(dY, Ys, positions, topk_w, dYs, dw, stream=None):
    """Gradients of ``moe_combine``: ``dYs[positions[t, s]] = topk_w[t, s] dY[t]`` and
    ``dw[t, s] = <Ys[positions[t, s]], dY[t]>`` (fp32; ``dw`` and ``Ys`` may both be None), written in place."""
    import torch
    M, N = _dims(dY, "dY", 2)
    k = _dims(positions, "positions", 2)[1]
    dt = _dtype_code(dY)
    rows = _dims(dYs, "dYs", 2)[0]
    if (Ys is None) != (dw is None):
        raise ValueError("dw takes Ys: give both or neither")
    f32 = torch.float32
    dev = _tensors(((dY, "dY", (M, N), dY.dtype), (positions, "positions", (M, k), torch.int32),
                    (dYs, "dYs", (rows, N), dY.dtype)),
                   ((Ys, "Ys", (rows, N), dY.dtype), (topk_w, "topk_w", (M, k), f32), (dw, "dw", (M, k), f32)))
    _check(lib().moe_combine_backward(dY.data_ptr(), _ptr(Ys), positions.data_ptr(), _ptr(topk_w), dYs.data_ptr(),
                                      _ptr(dw), M, N, k, rows, dt, _stream_of(stream, dev)))


def moe_route_backward(topk_ids, topk_w, dw, dlogits, stream=None):
    """The gradient of the gate's softmax over the chosen logits: ``dlogits`` (M x E, fp32), written in place.
    ``topk_ids`` are the router's own, also where a copy with dropped entries at -1 went into ``moe_dispatch``:
    a dropped choice still stands in the softmax, and its logit has a gradient."""
    import torch
    M, E = _dims(dlogits, "dlogits", 2)
    k = _dims(topk_ids, "topk_ids", 2)[1]
    f32 = torch.float32
    dev = _tensors(((topk_ids, "topk_ids", (M, k), torch.int32), (topk_w, "topk_w", (M, k), f32),
                    (dw, "dw", (M, k), f32), (dlogits, "dlogits", (M, E), f32)))
    _check(lib().moe_route_backward(topk_ids.data_ptr(), topk_w.data_ptr(), dw.data_ptr(), dlogits.data_ptr(), M, E,
                                    k, _stream_of(stream, dev)))
    return dlogits


# ---------------------------------------------------------------- 4-bit weights

def ffn_q4_bytes(K, C) -> int:
    return lib().ffn_q4_bytes(K, C)


def ffn_q4_empty(K, C, group=128, zero=False, experts=None, device="cuda"):
    """Buffers ``(Wq, scale, zero or None)`` of the packed layout of a K x C matrix, or of ``experts`` of them."""
    import torch
    if group not in (32, 64, 128):
        raise ValueError(f"group must be 32, 64 or 128 (got {group})")
    lead = () if experts is None else (experts,)
    ct, kt = -(-C // 16), -(-K // 128)
    scale = torch.zeros(*lead, ct, kt, 16, 128 // group, dtype=torch.bfloat16, device=device)
    return (torch.zeros(*lead, ct, kt, 1024, dtype=torch.uint8, device=device), scale,
            torch.zeros_like(scale) if zero else None)


def _q4_code(code):
    if isinstance(code, str) and code not in Q4_CODES:
        raise ValueError(f"code must be one of {sorted(Q4_CODES)} (got {code!r})")
    return Q4_CODES[code] if isinstance(code, str) else int(code)


def _q4_weight(Wq, scale, zero, lead, K, C, names=("Wq", "scale", "zero")):
    """The group size of one packed weight, and what ``_tensors`` checks of it: (needed, optional)."""
    import torch
    ct, kt = -(-C // 16), -(-K // 128)
    per = _dims(scale, names[1], 4 + len(lead))[-1]
    if per not in (1, 2, 4):
        raise ValueError(f"{names[1]} must have 1, 2 or 4 groups per 128 rows (got {per})")
    groups = (*lead, ct, kt, 16, per)
    return 128 // per, ((Wq, names[0], (*lead, ct, kt, 1024), torch.uint8),
                        (scale, names[1], groups, torch.bfloat16)), (zero, names[2], groups, torch.bfloat16)


def ffn_q4_quantize(W, Wq, scale, zero=None, code="int4", stream=None):
    """4-bit codes, scales and, when given, zero points of ``W`` (K x C, bf16 or fp32) in the packed layout
    (``ffn_q4_empty`` makes the buffers; the group size is the scales'), written in place."""
    K, C = _dims(W, "W", 2)
    dt = _dtype_code(W)
    group, packed, z = _q4_weight(Wq, scale, zero, (), K, C)
    dev = _tensors(((W, "W", (K, C), W.dtype), *packed), (z,))
    _check(lib().ffn_q4_quantize(W.data_ptr(), Wq.data_ptr(), scale.data_ptr(), _ptr(zero), K, C, dt, _q4_code(code),
                                 group, _stream_of(stream, dev)))
    return Wq


def ffn_q4_pack(codes, scale_in, Wq, scale, zero_in=None, zero=None, code="int4", stream=None):
    """Another quantiser's codes (K x C, uint8), scales and zero points (groups x C, bf16) into the packed
    layout, written in place."""
    import torch
    K, C = _dims(codes, "codes", 2)
    group, packed, z = _q4_weight(Wq, scale, zero, (), K, C)
    if (zero_in is None) != (zero is None):
        raise ValueError("give zero_in and zero together or neither")
    rows = (-(-K // group), C)
    dev = _tensors(((codes, "codes", (K, C), torch.uint8), (scale_in, "scale_in", rows, torch.bfloat16), *packed),
                   ((zero_in, "zero_in", rows, torch.bfloat16), z))
    _check(lib().ffn_q4_pack(codes.data_ptr(), scale_in.data_ptr(), _ptr(zero_in), Wq.data_ptr(), scale.data_ptr(),
                             _ptr(zero), K, C, _q4_code(code), group, _stream_of(stream, dev)))
    return Wq


def ffn_q4_matvec(X, Wq, scale, Y, zero=None, bias=None, act="none", code="int4", stream=None):
    """``Y = act(X W + bias)`` for up to 16 rows of X (bf16) and a K x C matrix of packed 4-bit weights;
    ``Y`` (bf16) is written in place."""
    import torch
    M, K = _dims(X, "X", 2)
    C = _dims(Y, "Y", 2)[1]
    bf = torch.bfloat16
    group, packed, z = _q4_weight(Wq, scale, zero, (), K, C)
    dev = _tensors(((X, "X", (M, K), bf), (Y, "Y", (M, C), bf), *packed), (z, (bias, "bias", (C,), bf)))
    _check(lib().ffn_q4_matvec(X.data_ptr(), Wq.data_ptr(), scale.data_ptr(), _ptr(zero), _ptr(bias), Y.data_ptr(), M,
                               K, C, _q4_code(code), group, _act(act), _stream_of(stream, dev)))
    return Y


def _q4_pair(Wg, scale_g, zero_g, Wu, scale_u, zero_u, lead, K, C):
    if (zero_g is None) != (zero_u is None):
        raise ValueError("give both zero points or neither")
    group, g, zg = _q4_weight(Wg, scale_g, zero_g, lead, K, C, ("Wg", "scale_g", "zero_g"))
    group_u, u, zu = _q4_weight(Wu, scale_u, zero_u, lead, K, C, ("Wu", "scale_u", "zero_u"))
    if group_u != group:
        raise ValueError("both matrices must have the same group size")
    return group, (*g, *u), (zg, zu)


def ffn_q4_swiglu(X, Wg, scale_g, Wu, scale_u, H, zero_g=None, zero_u=None, code="int4", stream=None):
    """``H = silu(X Wg) * (X Wu)`` for up to 16 rows of X (bf16) and two K x C matrices of packed 4-bit
    weights; ``H`` (bf16) is written in place."""
    import torch
    M, K = _dims(X, "X", 2)
    C = _dims(H, "H", 2)[1]
    bf = torch.bfloat16
    group, packed, z = _q4_pair(Wg, scale_g, zero_g, Wu, scale_u, zero_u, (), K, C)
    dev = _tensors(((X, "X", (M, K), bf), (H, "H", (M, C), bf), *packed), z)
    _check(lib().ffn_q4_swiglu(X.data_ptr(), Wg.data_ptr(), scale_g.data_ptr(), _ptr(zero_g), Wu.data_ptr(),
                               scale_u.data_ptr(), _ptr(zero_u), H.data_ptr(), M, K, C, _q4_code(code), group,
                               _stream_of(stream, dev)))
    return H


def moe_q4_matvec(X, expert_offsets, Wq, scale, Y, zero=None, bias=None, act="none", code="int4", stream=None):
    """``ffn_q4_matvec`` over the experts' row lists: rows ``expert_offsets[e]`` to ``expert_offsets[e + 1]``
    of X go through matrix e (Wq, scale, zero, bias: one per expert in front); other rows of ``Y`` are
    left as they were."""
    import torch
    rows, K = _dims(X, "X", 2)
    C = _dims(Y, "Y", 2)[1]
    E = _dims(expert_offsets, "expert_offsets", 1)[0] - 1
    bf = torch.bfloat16
    group, packed, z = _q4_weight(Wq, scale, zero, (E,), K, C)
    dev = _tensors(((X, "X", (rows, K), bf), (Y, "Y", (rows, C), bf),
                    (expert_offsets, "expert_offsets", (E + 1,), torch.int32), *packed),
                   (z, (bias, "bias", (E, C), bf)))
    _check(lib().moe_q4_matvec(X.data_ptr(), expert_offsets.data_ptr(), Wq.data_ptr(), scale.data_ptr(), _ptr(zero),
                               _ptr(bias), Y.data_ptr(), rows, E, K, C, _q4_code(code), group, _act(act),
                               _stream_of(stream, dev)))
    return Y


def moe_q4_swiglu(X, expert_offsets, Wg, scale_g, Wu, scale_u, H, zero_g=None, zero_u=None, code="int4",
                  stream=None):
    """``ffn_q4_swiglu`` over the experts' row lists, as ``moe_q4_matvec`` is ``ffn_q4_matvec`` over them."""
    import torch
    rows, K = _dims(X, "X", 2)
    C = _dims(H, "H", 2)[1]
    E = _dims(expert_offsets, "expert_offsets", 1)[0] - 1
    bf = torch.bfloat16
    group, packed, z = _q4_pair(Wg, scale_g, zero_g, Wu, scale_u, zero_u, (E,), K, C)
    dev = _tensors(((X, "X", (rows, K), bf), (H, "H", (rows, C), bf),
                    (expert_offsets, "expert_offsets", (E + 1,), torch.int32), *packed), z)
    _check(lib().moe_q4_swiglu(X.data_ptr(), expert_offsets.data_ptr(), Wg.data_ptr(), scale_g.data_ptr(),
                               _ptr(zero_g), Wu.data_ptr(), scale_u.data_ptr(), _ptr(zero_u), H.data_ptr(), rows, E,
                               K, C, _q4_code(code), group, _stream_of(stream, dev)))
    return H


# ---------------------------------------------------------------- measurement support

def ceiling_mfma(sink, iters, stream=None) -> float:
    """Enqueue the bf16 MFMA loop kernel; returns the FLOP count of the launch."""
    _on_device(sink)
    f = ctypes.c_double()
    _check(lib().ffn_ceiling_mfma(_ptr(sink), sink.numel() * sink.element_size(), iters,
                                  ctypes.byref(f), _stream(stream)))
    return f.value


def ceiling_read(src, sink, stream=None) -> int:
    """Enqueue one streaming read of ``src`` (a device tensor); returns the bytes read."""
    if not src.is_contiguous():
        raise ValueError("src must be contiguous")
    _on_device(src, sink)
    nbytes = src.numel() * src.element_size()
    _check(lib().ffn_ceiling_read(_ptr(src), nbytes, _ptr(sink), sink.numel() * sink.element_size(),
                                  _stream(stream)))
    return nbytes
