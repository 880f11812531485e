"""Thin ctypes binding of ``liblinattn.so`` (argument marshalling only).

Function names match the C ABI in ``include/linattn.h``.  Tensors are torch
CUDA tensors; the binding checks shapes and dtypes, allocates outputs that
were not supplied, passes raw device pointers and the current CUDA stream,
and raises :class:`LinAttnError` on a non-OK status.  Every step of the
computation runs in the library's kernels.  Importing this module fails if
the library has not been built (``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblinattn.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() before use")

lib = ctypes.CDLL(LIB_PATH)

LA_F32, LA_BF16 = 0, 1
STATUS_NAMES = {0: "LA_OK", 1: "LA_ERR_INVALID_VALUE", 2: "LA_ERR_UNSUPPORTED", 3: "LA_ERR_MISALIGNED",
                4: "LA_ERR_OUT_OF_MEMORY", 5: "LA_ERR_LAUNCH", 6: "LA_ERR_TIMEOUT", 7: "LA_ERR_NO_DEVICE",
                8: "LA_ERR_TOO_LARGE"}

_vp, _fp, _i, _f = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
_SEQ_ARGS = [_vp, _vp, _vp, _fp, _fp, _fp, _i, _i, _i, _i, _i, _f, _i, _vp]
for _name in ("la_global", "la_causal", "la_causal_with_state", "la_causal_noalloc", "la_causal_features",
              "la_global_features"):
    getattr(lib, _name).argtypes = _SEQ_ARGS
    getattr(lib, _name).restype = _i
for _name in ("la_retention", "la_retention_with_state"):
    getattr(lib, _name).argtypes = [_vp, _vp, _vp, _fp, _fp, ctypes.POINTER(_f), _i, _i, _i, _i, _i, _i, _vp]
    getattr(lib, _name).restype = _i
lib.la_decode_step.argtypes = [_vp, _vp, _vp, _fp, _fp, _fp, _i, _i, _i, _i, _f, _i, _vp]
lib.la_retention_decode_step.argtypes = [_vp, _vp, _vp, _fp, _fp, ctypes.POINTER(_f), _i, _i, _i, _i, _i, _vp]
lib.la_retention_decode_step.restype = _i
lib.la_causal_backward.argtypes = [_vp] * 13 + [_i, _i, _i, _i, _i, _f, _i, _vp]
lib.la_causal_backward.restype = _i
lib.la_favor_features.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp]
lib.la_favor_features.restype = _i
_sz = ctypes.c_size_t
for _name in ("la_gated", "la_gated_with_state"):
    getattr(lib, _name).argtypes = [_vp] * 7 + [_i] * 6 + [_vp, _sz, _vp]
    getattr(lib, _name).restype = _i
lib.la_gated_workspace.argtypes = [_i] * 7
lib.la_gated_workspace.restype = _sz
lib.la_gated_backward.argtypes = [_vp] * 13 + [_i] * 6 + [_vp, _sz, _vp]
lib.la_gated_backward.restype = _i
lib.la_gated_decode_step.argtypes = [_vp] * 7 + [_i] * 6 + [_vp]
lib.la_gated_decode_step.restype = _i
lib.la_group_norm.argtypes = [_vp] * 5 + [_i] * 4 + [_f, _i, _vp]
lib.la_group_norm.restype = _i
lib.la_group_norm_workspace.argtypes = [_i] * 4
lib.la_group_norm_workspace.restype = _sz
lib.la_group_norm_backward.argtypes = [_vp] * 9 + [_i] * 4 + [_f, _i, _vp, _sz, _vp]
lib.la_group_norm_backward.restype = _i
lib.la_decode_step.restype = _i
lib.la_status_string.argtypes = [_i]
lib.la_status_string.restype = ctypes.c_char_p
lib.la_version.argtypes = []
lib.la_version.restype = _i
lib.la_device_status.argtypes = [_vp]
lib.la_device_status.restype = _i
lib.la_last_error_detail.argtypes = []
lib.la_last_error_detail.restype = ctypes.c_char_p
lib.la_kernel_launches.argtypes = []
lib.la_kernel_launches.restype = ctypes.c_ulonglong
lib.la_diag_force_segments.argtypes = [_i]
lib.la_diag_force_segments.restype = _i
lib.la_test_inject_missing_load.argtypes = [_i, ctypes.c_uint]
lib.la_test_inject_missing_load.restype = _i
lib.la_profile_enable.argtypes = [_i]
lib.la_profile_enable.restype = _i
lib.la_profile_read.argtypes = [_i, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_longlong)]
lib.la_profile_read.restype = _i

# la_kernel ids of the device-time diagnostics
KERNELS = {"causal_main": 0, "causal_state": 1, "exact_head": 2, "causal_simt": 3, "global_state": 4,
           "global_read": 5, "decode": 6, "retention_main": 7, "retention_state": 8, "retention_decode": 9,
           "backward": 10, "favor": 11, "global_fused": 12, "gated": 13, "gated_state": 14, "gated_backward": 15,
           "gated_decode": 16, "group_norm": 17, "group_norm_backward": 18}


class LinAttnError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        detail = f"; {lib.la_last_error_detail().decode()}" if code in (4, 5, 7) else ""
        super().__init__(f"{fn}: {STATUS_NAMES.get(code, code)} ({status_string(code)}{detail})")


def status_string(code: int) -> str:
    return lib.la_status_string(code).decode()


def version() -> int:
    return lib.la_version()


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return LA_F32
    if t.dtype == torch.bfloat16:
        return LA_BF16
    raise TypeError(f"q, k, v must be float32 or bfloat16, got {t.dtype}")


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_in(q, k, v, nd):
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda or not t.is_contiguous() or t.dim() != nd:
            raise ValueError(f"{name} must be a contiguous {nd}-d CUDA tensor")
    if q.dtype != k.dtype or q.dtype != v.dtype:
        raise TypeError("q, k, v must share one dtype")
    if q.shape != k.shape or q.shape[:-1] != v.shape[:-1]:
        raise ValueError("q, k must have equal shapes and v the same leading dims")


def _state(S, z, lead, dk, dv, dev):
    if S is None:
        S = torch.empty(*lead, dk, dv, dtype=torch.float32, device=dev)
    if z is None:
        z = torch.empty(*lead, dk, dtype=torch.float32, device=dev)
    if S.dtype != torch.float32 or z.dtype != torch.float32 or not S.is_contiguous() or not z.is_contiguous():
        raise ValueError("S and z must be contiguous float32 tensors")
    if tuple(S.shape) != (*lead, dk, dv) or tuple(z.shape) != (*lead, dk):
        raise ValueError(f"S must be {(*lead, dk, dv)} and z {(*lead, dk)}")
    return S, z


def _seq_call(fn, q, k, v, out, S, z, eps, stream, need_state_in=False):
    _check_in(q, k, v, 4)
    B, H, N, dk = q.shape
    dv = v.shape[-1]
    if need_state_in and (S is None or z is None):
        raise ValueError(f"{fn} needs the initial state S, z")
    S, z = _state(S, z, (B, H), dk, dv, q.device)
    if out is None:
        out = torch.empty(B, H, N, dv, dtype=torch.float32, device=q.device)
    if out.dtype != torch.float32 or not out.is_contiguous() or tuple(out.shape) != (B, H, N, dv):
        raise ValueError("out must be a contiguous float32 [B, H, N, d_v] tensor")
    rc = getattr(lib, fn)(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(S), _ptr(z), B, H, N, dk, dv, float(eps),
                          _dt(q), _stream(stream))
    if rc != 0:
        raise LinAttnError(fn, rc)
    return out, S, z


def la_global(q, k, v, out=None, S=None, z=None, eps: float = 1e-6, stream=None):
    """Global read; returns (out, S, z).  S, z are overwritten with the whole-sequence state."""
    return _seq_call("la_global", q, k, v, out, S, z, eps, stream)


def la_causal(q, k, v, out=None, S=None, z=None, eps: float = 1e-6, stream=None):
    """Causal prefill from the zero state; returns (out, S, z) with the final state."""
    return _seq_call("la_causal", q, k, v, out, S, z, eps, stream)


def la_causal_noalloc(q, k, v, out=None, S=None, z=None, eps: float = 1e-6, stream=None):
    """la_causal without device allocation inside the library (fixed scratch; see linattn.h).

    Pass preallocated out, S, z to keep the whole call allocation-free: the
    binding only allocates the outputs that were not supplied.
    """
    return _seq_call("la_causal_noalloc", q, k, v, out, S, z, eps, stream)


def la_causal_features(phi_q, phi_k, v, out=None, S=None, z=None, eps: float = 1e-6, stream=None):
    """Causal prefill on given (non-negative) features; returns (out, S, z)."""
    return _seq_call("la_causal_features", phi_q, phi_k, v, out, S, z, eps, stream)


def la_global_features(phi_q, phi_k, v, out=None, S=None, z=None, eps: float = 1e-6, stream=None):
    """Global read on given (non-negative) features; returns (out, S, z)."""
    return _seq_call("la_global_features", phi_q, phi_k, v, out, S, z, eps, stream)


def la_favor_features(x, W, out=None, stream=None):
    """Positive random features of x [B, H, N, d] for projections W [m, d]: [B, H, N, m], x's dtype."""
    if not x.is_cuda or not x.is_contiguous() or x.dim() != 4:
        raise ValueError("x must be a contiguous 4-d CUDA tensor")
    if not W.is_cuda or not W.is_contiguous() or W.dim() != 2 or W.shape[1] != x.shape[-1] or W.dtype != x.dtype:
        raise ValueError("W must be a contiguous [m, d] CUDA tensor of x's dtype")
    B, H, N, d = x.shape
    m = W.shape[0]
    if out is None:
        out = torch.empty(B, H, N, m, dtype=x.dtype, device=x.device)
    if out.dtype != x.dtype or not out.is_contiguous() or tuple(out.shape) != (B, H, N, m):
        raise ValueError("out must be a contiguous [B, H, N, m] tensor of x's dtype")
    rc = lib.la_favor_features(_ptr(x), _ptr(W), _ptr(out), B, H, N, d, m, _dt(x), _stream(stream))
    if rc != 0:
        raise LinAttnError("la_favor_features", rc)
    return out


def la_causal_with_state(q, k, v, S, z, out=None, eps: float = 1e-6, stream=None):
    """Causal prefill continuing from (S, z), which are updated in place; returns (out, S, z)."""
    return _seq_call("la_causal_with_state", q, k, v, out, S, z, eps, stream, need_state_in=True)


def _retention_call(fn, q, k, v, gamma, out, S, stream, need_state_in=False):
    _check_in(q, k, v, 4)
    B, H, N, dk = q.shape
    dv = v.shape[-1]
    g = [float(x) for x in gamma]
    if len(g) != H:
        raise ValueError(f"gamma must hold one decay per head ({H}), got {len(g)}")
    if need_state_in and S is None:
        raise ValueError(f"{fn} needs the initial state S")
    if S is None:
        S = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    if S.dtype != torch.float32 or not S.is_contiguous() or tuple(S.shape) != (B, H, dk, dv):
        raise ValueError(f"S must be a contiguous float32 {(B, H, dk, dv)} tensor")
    if out is None:
        out = torch.empty(B, H, N, dv, dtype=torch.float32, device=q.device)
    if out.dtype != torch.float32 or not out.is_contiguous() or tuple(out.shape) != (B, H, N, dv):
        raise ValueError("out must be a contiguous float32 [B, H, N, d_v] tensor")
    garr = (_f * max(H, 1))(*g)
    rc = getattr(lib, fn)(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(S), garr, B, H, N, dk, dv, _dt(q),
                          _stream(stream))
    if rc != 0:
        raise LinAttnError(fn, rc)
    return out, S


def la_retention(q, k, v, gamma, out=None, S=None, stream=None):
    """Retention from the zero state (decay gamma[h] per head, no denominator); returns (out, S)."""
    return _retention_call("la_retention", q, k, v, gamma, out, S, stream)


def la_retention_with_state(q, k, v, S, gamma, out=None, stream=None):
    """Retention continuing from S, which is updated in place; returns (out, S)."""
    return _retention_call("la_retention_with_state", q, k, v, gamma, out, S, stream, need_state_in=True)


def la_decode_step(q, k, v, S, z, out=None, eps: float = 1e-6, stream=None):
    """One decode step; q, k [B, H, d_k], v [B, H, d_v]; S, z updated in place; returns out."""
    _check_in(q, k, v, 3)
    B, H, dk = q.shape
    dv = v.shape[-1]
    S, z = _state(S, z, (B, H), dk, dv, q.device)
    if out is None:
        out = torch.empty(B, H, dv, dtype=torch.float32, device=q.device)
    rc = lib.la_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(S), _ptr(z), B, H, dk, dv, float(eps),
                            _dt(q), _stream(stream))
    if rc != 0:
        raise LinAttnError("la_decode_step", rc)
    return out


def la_retention_decode_step(q, k, v, S, gamma, out=None, stream=None):
    """One retention step; q, k [B, H, d_k], v [B, H, d_v]; S updated in place; returns out."""
    _check_in(q, k, v, 3)
    B, H, dk = q.shape
    dv = v.shape[-1]
    g = [float(x) for x in gamma]
    if len(g) != H:
        raise ValueError(f"gamma must hold one decay per head ({H}), got {len(g)}")
    if S is None or S.dtype != torch.float32 or not S.is_contiguous() or tuple(S.shape) != (B, H, dk, dv):
        raise ValueError(f"S must be a contiguous float32 {(B, H, dk, dv)} tensor")
    if out is None:
        out = torch.empty(B, H, dv, dtype=torch.float32, device=q.device)
    rc = lib.la_retention_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(S), (_f * max(H, 1))(*g), B, H,
                                      dk, dv, _dt(q), _stream(stream))
    if rc != 0:
        raise LinAttnError("la_retention_decode_step", rc)
    return out


def la_causal_backward(q, k, v, dout, S0=None, z0=None, dS=None, dz=None, need_state_grad: bool = False,
                       eps: float = 1e-6, stream=None):
    """Gradients of la_causal (la_causal_with_state when S0, z0 are given) for the
    upstream gradient ``dout`` of its output and, optionally, ``dS``, ``dz`` of its
    final state.  Returns (dq, dk, dv), plus (dS0, dz0) when ``need_state_grad``."""
    _check_in(q, k, v, 4)
    B, H, N, dk = q.shape
    dv = v.shape[-1]

    def f32(t, shape, name):
        if t is None:
            return None
        if not t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != shape:
            raise ValueError(f"{name} must be a contiguous float32 CUDA tensor of shape {shape}")
        return t

    dout = f32(dout, (B, H, N, dv), "dout")
    S0, dS = f32(S0, (B, H, dk, dv), "S0"), f32(dS, (B, H, dk, dv), "dS")
    z0, dz = f32(z0, (B, H, dk), "z0"), f32(dz, (B, H, dk), "dz")
    new = lambda *shape: torch.empty(*shape, dtype=torch.float32, device=q.device)
    dq, dkk, dvv = new(B, H, N, dk), new(B, H, N, dk), new(B, H, N, dv)
    dS0, dz0 = (new(B, H, dk, dv), new(B, H, dk)) if need_state_grad else (None, None)
    rc = lib.la_causal_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(S0), _ptr(z0), _ptr(dS), _ptr(dz),
                                _ptr(dq), _ptr(dkk), _ptr(dvv), _ptr(dS0), _ptr(dz0), B, H, N, dk, dv, float(eps),
                                _dt(q), _stream(stream))
    if rc != 0:
        raise LinAttnError("la_causal_backward", rc)
    return (dq, dkk, dvv, dS0, dz0) if need_state_grad else (dq, dkk, dvv)


# The current device and a device's current stream without the public calls' wrappers (host time counts in small
# calls); where torch does not have these, the public calls.
_device_index = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_stream_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(device, stream):
    """(stream handle, context to leave) of a call on `device`: the given stream, or that device's current one.

    Outputs and workspaces are allocated between this and :func:`_off`, so that they belong to that stream.
    Entering a context is needed only for another stream or device than the current ones.
    """
    if stream is None:
        if device.index == _device_index():
            return _stream_handle(device.index), None
        stream = torch.cuda.current_stream(device)
    elif not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {device}")
    ctx = torch.cuda.stream(stream)
    ctx.__enter__()  # makes the stream's device current too
    return stream.cuda_stream, ctx


def _off(ctx):
    if ctx is not None:
        ctx.__exit__(None, None, None)


def _need(name, t, shape, dtype, device):
    """t itself, after checking that it is a contiguous tensor of that shape, dtype and (CUDA) device."""
    if isinstance(t, torch.Tensor) and t.get_device() == device.index and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _opt(name, t, shape, dtype, device):
    return None if t is None else _need(name, t, shape, dtype, device)


def _out(name, t, shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device) if t is None else _need(name, t, shape, dtype, device)


def _first(name, t, nd):
    """The device of a call, from its first tensor."""
    if not isinstance(t, torch.Tensor) or t.dim() != nd:
        raise ValueError(f"{name} must be a {nd}-d tensor")
    if not t.is_cuda:
        _dt(t)
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return t.device


def _gated_inputs(q, k, v, g, nd):
    """(device, lead, d_k, d_v, dtype code) of gated inputs whose leading dims are [B, H, N] (nd = 4) or [B, H] (nd = 3)."""
    dev = _first("q", q, nd)
    _first("v", v, nd)
    dt, dtype, shape = _dt(q), q.dtype, q.shape
    lead, dk, dv = shape[:-1], shape[-1], v.shape[-1]
    _need("q", q, shape, dtype, dev)
    _need("k", k, shape, dtype, dev)
    _need("v", v, (*lead, dv), dtype, dev)
    _need("g", g, lead, torch.float32, dev)
    return dev, lead, dk, dv, dt


@functools.lru_cache(maxsize=1024)
def _gated_workspace(device, B, H, N, dk, dv, dt, backward):
    with torch.cuda.device(device):
        return lib.la_gated_workspace(B, H, N, dk, dv, dt, backward)


def _workspace(need, device):
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


def _gated_call(fn, q, k, v, g, lengths, out, S, stream):
    dev, (B, H, N), dk, dv, dt = _gated_inputs(q, k, v, g, 4)
    _opt("lengths", lengths, (B,), torch.int32, dev)
    s, ctx = _on(dev, stream)
    try:
        if out is None and lengths is not None:  # the call does not write padding rows, the next layer may read them
            out = torch.zeros((B, H, N, dv), dtype=q.dtype, device=dev)
        out = _out("out", out, (B, H, N, dv), q.dtype, dev)
        S = _out("S", S, (B, H, dk, dv), torch.float32, dev)
        need = _gated_workspace(dev.index, B, H, N, dk, dv, dt, 0)
        ws = _workspace(need, dev)
        rc = getattr(lib, fn)(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(lengths), _ptr(out), _ptr(S), B, H, N, dk, dv, dt,
                              _ptr(ws), need, s)
    finally:
        _off(ctx)
    if rc != 0:
        raise LinAttnError(fn, rc)
    return out, S


def la_gated(q, k, v, g, lengths=None, out=None, S=None, stream=None):
    """Gated linear attention S_t = e^{g_t} S_{t-1} + k_t v_t^T, out_t = q_t^T S_t from the zero state.

    q, k [B, H, N, d_k], v [B, H, N, d_v] (float32 or bfloat16); g [B, H, N] float32 log decays (<= 0; -inf resets).
    lengths [B] int32: tokens past a row's length take no part and their rows of a given ``out`` are not written (give
    it finite rows there if la_group_norm and its gradient read them); without ``out`` they are zero.
    Returns (out in q's dtype, final state S float32).
    """
    return _gated_call("la_gated", q, k, v, g, lengths, out, S, stream)


def la_gated_with_state(q, k, v, g, S, lengths=None, out=None, stream=None):
    """Gated linear attention continuing from S, which is updated in place; returns (out, S)."""
    if S is None:
        raise ValueError("la_gated_with_state needs the initial state S")
    return _gated_call("la_gated_with_state", q, k, v, g, lengths, out, S, stream)


def la_gated_backward(q, k, v, g, dout, S0=None, dS=None, lengths=None, need_state_grad: bool = False, stream=None):
    """Gradients of la_gated (la_gated_with_state when S0 is given) for the upstream gradient ``dout`` of its output
    (q's dtype) and, optionally, ``dS`` of its final state.  Returns (dq, dk, dv, dg), plus dS0 when
    ``need_state_grad``; dq, dk, dv in q's dtype, dg and dS0 float32."""
    dev, (B, H, N), dk, dv, dt = _gated_inputs(q, k, v, g, 4)
    _need("dout", dout, (B, H, N, dv), q.dtype, dev)
    _opt("lengths", lengths, (B,), torch.int32, dev)
    _opt("S0", S0, (B, H, dk, dv), torch.float32, dev)
    _opt("dS", dS, (B, H, dk, dv), torch.float32, dev)
    s, ctx = _on(dev, stream)
    try:
        dq, dkk, dvv, dg = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(g)
        dS0 = torch.empty(B, H, dk, dv, dtype=torch.float32, device=dev) if need_state_grad else None
        need = _gated_workspace(dev.index, B, H, N, dk, dv, dt, 1)
        ws = _workspace(need, dev)
        rc = lib.la_gated_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(lengths), _ptr(dout), _ptr(S0), _ptr(dS),
                                   _ptr(dq), _ptr(dkk), _ptr(dvv), _ptr(dg), _ptr(dS0), B, H, N, dk, dv, dt, _ptr(ws),
                                   need, s)
    finally:
        _off(ctx)
    if rc != 0:
        raise LinAttnError("la_gated_backward", rc)
    return (dq, dkk, dvv, dg, dS0) if need_state_grad else (dq, dkk, dvv, dg)


def la_gated_decode_step(q, k, v, g, S, slots=None, out=None, stream=None):
    """One gated step; q, k [B, H, d_k], v [B, H, d_v], g [B, H]; returns out [B, H, d_v] in q's dtype.

    S [n_slots, H, d_k, d_v] is a pool of states: row b works in place on S[slots[b]] (slots [B] int32; without it,
    row b on S[b]).  g = -inf starts a state anew, whatever its slot held.  A negative slot marks an unused row (out
    zero).  A slot out of range or repeated in the batch is skipped too, and the next device_status() is 1.
    """
    dev, (B, H), dk, dv, dt = _gated_inputs(q, k, v, g, 3)
    if not isinstance(S, torch.Tensor) or S.dim() != 4:
        raise ValueError("S must be a [n_slots, H, d_k, d_v] tensor")
    n_slots = S.shape[0]
    _need("S", S, (n_slots, H, dk, dv), torch.float32, dev)
    _opt("slots", slots, (B,), torch.int32, dev)
    if slots is None and n_slots < B:
        raise ValueError(f"S holds {n_slots} states for {B} rows")
    s, ctx = _on(dev, stream)
    try:
        out = _out("out", out, (B, H, dv), q.dtype, dev)
        rc = lib.la_gated_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(S), _ptr(slots), _ptr(out), B, H, n_slots,
                                      dk, dv, dt, s)
    finally:
        _off(ctx)
    if rc != 0:
        raise LinAttnError("la_gated_decode_step", rc)
    return out


def _norm_inputs(x, gate, weight, bias):
    dev = _first("x", x, 4)
    B, H, N, d = x.shape
    dt = _dt(x)
    _need("x", x, x.shape, x.dtype, dev)
    _opt("gate", gate, (B, N, H * d), x.dtype, dev)
    _opt("weight", weight, (H * d,), torch.float32, dev)
    _opt("bias", bias, (H * d,), torch.float32, dev)
    return dev, B, H, N, d, dt


def la_group_norm(x, gate=None, weight=None, bias=None, eps: float = 1e-5, out=None, stream=None):
    """Group norm of each head's channels times silu(gate): x [B, H, N, d] -> [B, N, H*d], x's dtype.

    gate [B, N, H*d] (x's dtype); weight, bias [H*d] float32; each may be None.
    """
    dev, B, H, N, d, dt = _norm_inputs(x, gate, weight, bias)
    s, ctx = _on(dev, stream)
    try:
        out = _out("out", out, (B, N, H * d), x.dtype, dev)
        rc = lib.la_group_norm(_ptr(x), _ptr(gate), _ptr(weight), _ptr(bias), _ptr(out), B, H, N, d, float(eps), dt, s)
    finally:
        _off(ctx)
    if rc != 0:
        raise LinAttnError("la_group_norm", rc)
    return out


@functools.lru_cache(maxsize=1024)
def _norm_workspace(device, B, H, N, d):
    with torch.cuda.device(device):
        return lib.la_group_norm_workspace(B, H, N, d)


def la_group_norm_backward(x, dy, gate=None, weight=None, bias=None, eps: float = 1e-5, stream=None):
    """Gradients of la_group_norm for dy [B, N, H*d]: (dx, dgate, dweight, dbias), None for an argument not given.

    Every row adds to dweight and dbias: padding rows need finite x and gate, and zeros in dy.
    """
    dev, B, H, N, d, dt = _norm_inputs(x, gate, weight, bias)
    _need("dy", dy, (B, N, H * d), x.dtype, dev)
    s, ctx = _on(dev, stream)
    try:
        dx = torch.empty_like(x)
        dgate, dw, db = (None if t is None else torch.empty_like(t) for t in (gate, weight, bias))
        need = 0 if dw is None and db is None else _norm_workspace(dev.index, B, H, N, d)
        ws = _workspace(need, dev)
        rc = lib.la_group_norm_backward(_ptr(x), _ptr(dy), _ptr(gate), _ptr(weight), _ptr(bias), _ptr(dx), _ptr(dgate),
                                        _ptr(dw), _ptr(db), B, H, N, d, float(eps), dt, _ptr(ws), need, s)
    finally:
        _off(ctx)
    if rc != 0:
        raise LinAttnError("la_group_norm_backward", rc)
    return dx, dgate, dw, db


def device_status(stream=None) -> int:
    """Synchronize the stream and return (and clear) the device status: 0 = OK, 6 = a bounded wait timed out."""
    return int(lib.la_device_status(_stream(stream)))


def diag_force_segments(segments: int) -> None:
    """Diagnostics: segments per head of the tensor-core causal passes (0: the planner's choice)."""
    rc = lib.la_diag_force_segments(int(segments))
    if rc != 0:
        raise LinAttnError("la_diag_force_segments", rc)


def test_inject_missing_load(chunk: int, wait_us: int) -> None:
    """Testing only: the next tensor-core causal launch leaves out one key load of its
    first CTA and gives every wait ``wait_us`` microseconds (see linattn.h)."""
    rc = lib.la_test_inject_missing_load(int(chunk), int(wait_us))
    if rc != 0:
        raise LinAttnError("la_test_inject_missing_load", rc)


def profile_enable(on: bool = True) -> None:
    """Start (clearing the totals) or stop per-launch device timing."""
    lib.la_profile_enable(1 if on else 0)


def profile_read(kernel: str):
    """(total milliseconds, timed launches) of one kernel since profile_enable(True)."""
    ms, n = ctypes.c_double(), ctypes.c_longlong()
    rc = lib.la_profile_read(KERNELS[kernel], ctypes.byref(ms), ctypes.byref(n))
    if rc != 0:
        raise LinAttnError("la_profile_read", rc)
    return ms.value, n.value


def kernel_launches() -> int:
    """Kernels the library has enqueued in this process so far."""
    return int(lib.la_kernel_launches())
