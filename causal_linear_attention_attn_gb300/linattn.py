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
_l = ctypes.c_long
_CONV_ARGS = [_vp, _l, _vp, _vp, _vp]
for _name in ("la_short_conv", "la_short_conv_with_state"):
    getattr(lib, _name).argtypes = _CONV_ARGS + [_vp, _vp] + [_i] * 6 + [_vp]
    getattr(lib, _name).restype = _i
lib.la_short_conv_workspace.argtypes = [_i] * 4
lib.la_short_conv_workspace.restype = _sz
lib.la_short_conv_backward.argtypes = _CONV_ARGS + [_vp] * 7 + [_i] * 6 + [_vp, _sz, _vp]
lib.la_short_conv_backward.restype = _i
lib.la_short_conv_step.argtypes = [_vp, _l] + [_vp] * 5 + [_i] * 6 + [_vp]
lib.la_short_conv_step.restype = _i
_SCAN_ARGS = [_vp, _l, _vp, _l, _vp, _vp, _l, _vp, _l, _vp, _vp, _l, _vp]
for _name in ("la_selective_scan", "la_selective_scan_with_state"):
    getattr(lib, _name).argtypes = _SCAN_ARGS + [_vp] * 3 + [_i] * 6 + [_vp, _sz, _vp]
    getattr(lib, _name).restype = _i
lib.la_selective_scan_workspace.argtypes = [_i] * 6
lib.la_selective_scan_workspace.restype = _sz
lib.la_selective_scan_backward.argtypes = _SCAN_ARGS + [_vp] * 13 + [_i] * 6 + [_vp, _sz, _vp]
lib.la_selective_scan_backward.restype = _i
lib.la_selective_scan_step.argtypes = _SCAN_ARGS + [_vp] * 3 + [_i] * 6 + [_vp]
lib.la_selective_scan_step.restype = _i
lib.la_beam_select.argtypes = [_vp, _l] + [_vp] * 5 + [_i] * 6 + [_vp, _sz, _vp]
lib.la_beam_select.restype = _i
lib.la_beam_select_workspace.argtypes = [_i] * 5
lib.la_beam_select_workspace.restype = _sz
lib.la_beam_reorder.argtypes = [ctypes.POINTER(_vp), ctypes.POINTER(_sz), _i, _vp, _vp, _vp, _i, _i, _i, _vp]
lib.la_beam_reorder.restype = _i
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
           "gated_decode": 16, "group_norm": 17, "group_norm_backward": 18, "short_conv": 19, "short_conv_backward": 20,
           "short_conv_step": 21, "selective_scan": 22, "selective_state": 23, "selective_backward": 24,
           "selective_step": 25, "beam_select": 26, "beam_reorder": 27}


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


def _rows(name, t, shape, dtype, device):
    """The distance of t's rows in elements, after checking its shape, dtype and device: rows of consecutive values at
    one distance throughout (a contiguous tensor, or a part of the last dimension of one)."""
    if isinstance(t, torch.Tensor) and t.get_device() == device.index and t.dtype is dtype and t.shape == shape:
        strides = t.stride()
        if strides[-1] == 1:  # (dimensions of one row have no distance)
            rows = shape[-2]
            if len(shape) == 2:
                return strides[0] if rows > 1 else shape[1]
            if rows == 1:
                return strides[0] if shape[0] > 1 else shape[2]
            if shape[0] == 1 or strides[0] == rows * strides[1]:
                return strides[1]
        if t.numel() == 0:
            return shape[-1]
        raise ValueError(f"{name} must be contiguous, or one part of the last dimension of a contiguous tensor")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _first_rows(name, t, nd):
    """The device of a call, from its first tensor, which may be a part of a wider one."""
    if not isinstance(t, torch.Tensor) or t.dim() != nd:
        raise ValueError(f"{name} must be a {nd}-d tensor")
    _dt(t)
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _conv_inputs(x, weight, bias, nd):
    dev = _first_rows("x", x, nd)
    D = x.shape[-1]
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a [D, K] tensor")
    K = weight.shape[1]
    ldx = _rows("x", x, x.shape, x.dtype, dev)
    _need("weight", weight, (D, K), torch.float32, dev)
    _opt("bias", bias, (D,), torch.float32, dev)
    return dev, D, K, ldx, _dt(x)


def _zero_padding(t, lengths, shape, dtype, device):
    """An output to allocate, zero where the call does not write padding rows that the next layer may read."""
    return torch.zeros(shape, dtype=dtype, device=device) if t is None and lengths is not None else t


def _short_conv_call(fn, x, weight, S, bias, silu, lengths, out, stream):
    dev, D, K, ldx, dt = _conv_inputs(x, weight, bias, 3)
    B, N, _ = x.shape
    _opt("lengths", lengths, (B,), torch.int32, dev)
    s, ctx = _on(dev, stream)
    try:
        out = _out("out", _zero_padding(out, lengths, (B, N, D), x.dtype, dev), (B, N, D), x.dtype, dev)
        S = _out("S", S, (B, max(K - 1, 0), D), x.dtype, dev)
        rc = getattr(lib, fn)(_ptr(x), ldx, _ptr(weight), _ptr(bias), _ptr(lengths), _ptr(out), _ptr(S), B, N, D, K,
                              int(silu), dt, s)
    finally:
        _off(ctx)
    if rc != 0:
        raise LinAttnError(fn, rc)
    return out, S


def la_short_conv(x, weight, bias=None, silu: bool = True, lengths=None, out=None, S=None, stream=None):
    """Causal convolution along the tokens with a window of K = 2, 3 or 4 weights per channel, and SiLU.

    x [B, N, D] (float32 or bfloat16, D a multiple of 8; a part of the last dimension of a wider tensor will do); weight
    [D, K] (the last one is the current token's), bias [D], float32.  lengths [B] int32: tokens past a row's length take
    no part and their rows of a given ``out`` (not over an input) are not written; without ``out`` they are zero.
    Returns (out [B, N, D], S [B, K-1, D] the last inputs), both in x's dtype.
    """
    return _short_conv_call("la_short_conv", x, weight, S, bias, silu, lengths, out, stream)


def la_short_conv_with_state(x, weight, S, bias=None, silu: bool = True, lengths=None, out=None, stream=None):
    """Short convolution continuing from the inputs in S, which is updated in place; returns (out, S)."""
    if S is None:
        raise ValueError("la_short_conv_with_state needs the inputs S before the first")
    return _short_conv_call("la_short_conv_with_state", x, weight, S, bias, silu, lengths, out, stream)


@functools.lru_cache(maxsize=1024)
def _conv_workspace(device, B, N, D, K):
    with torch.cuda.device(device):
        return lib.la_short_conv_workspace(B, N, D, K)


def la_short_conv_backward(x, weight, dout, bias=None, silu: bool = True, S0=None, dS=None, lengths=None,
                           need_state_grad: bool = False, stream=None):
    """Gradients of la_short_conv (la_short_conv_with_state when S0 is given) for ``dout`` [B, N, D] (x's dtype) and,
    optionally, ``dS`` of the inputs it carries on.  Returns (dx, dweight, dbias), plus dS0 when ``need_state_grad``; dx
    and dS0 in x's dtype, dweight and dbias float32, dbias None without bias."""
    dev, D, K, ldx, dt = _conv_inputs(x, weight, bias, 3)
    B, N, _ = x.shape
    _need("dout", dout, (B, N, D), x.dtype, dev)
    _opt("lengths", lengths, (B,), torch.int32, dev)
    _opt("S0", S0, (B, max(K - 1, 0), D), x.dtype, dev)
    _opt("dS", dS, (B, max(K - 1, 0), D), x.dtype, dev)
    s, ctx = _on(dev, stream)
    try:
        dx, dw = torch.empty(B, N, D, dtype=x.dtype, device=dev), torch.empty_like(weight)
        db = None if bias is None else torch.empty_like(bias)
        dS0 = torch.empty(B, max(K - 1, 0), D, dtype=x.dtype, device=dev) if need_state_grad else None
        need = _conv_workspace(dev.index, B, N, D, K)
        ws = _workspace(need, dev)
        rc = lib.la_short_conv_backward(_ptr(x), ldx, _ptr(weight), _ptr(bias), _ptr(lengths), _ptr(dout), _ptr(S0),
                                        _ptr(dS), _ptr(dx), _ptr(dw), _ptr(db), _ptr(dS0), B, N, D, K, int(silu), dt,
                                        _ptr(ws), need, s)
    finally:
        _off(ctx)
    if rc != 0:
        raise LinAttnError("la_short_conv_backward", rc)
    return (dx, dw, db, dS0) if need_state_grad else (dx, dw, db)


def _pool(S, B, slots, row, dtype, device):
    if not isinstance(S, torch.Tensor) or S.dim() != 1 + len(row):
        raise ValueError(f"S must be a [n_slots, {', '.join(map(str, row))}] tensor")
    _need("S", S, (S.shape[0], *row), dtype, device)
    _opt("slots", slots, (B,), torch.int32, device)
    if slots is None and S.shape[0] < B:
        raise ValueError(f"S holds {S.shape[0]} states for {B} rows")
    return S.shape[0]


def la_short_conv_step(x, weight, S, bias=None, silu: bool = True, slots=None, out=None, stream=None):
    """One token of the short convolution; x [B, D]; returns out [B, D] in x's dtype.

    S [n_slots, K-1, D] (x's dtype) is a pool of windows: row b works in place on S[slots[b]].  slots as in
    la_gated_decode_step, unused, bad and repeated ones too.
    """
    dev, D, K, ldx, dt = _conv_inputs(x, weight, bias, 2)
    B = x.shape[0]
    n_slots = _pool(S, B, slots, (max(K - 1, 0), D), x.dtype, dev)
    s, ctx = _on(dev, stream)
    try:
        out = _out("out", out, (B, D), x.dtype, dev)
        rc = lib.la_short_conv_step(_ptr(x), ldx, _ptr(weight), _ptr(bias), _ptr(S), _ptr(slots), _ptr(out), B, n_slots, D,
                                    K, int(silu), dt, s)
    finally:
        _off(ctx)
    if rc != 0:
        raise LinAttnError("la_short_conv_step", rc)
    return out


def _scan_inputs(x, dt, A, Bm, Cm, D, z, dt_bias, nd):
    """(device, lead, channels, d_state, dtype code, the arguments that every selective call begins with)."""
    dev = _first_rows("x", x, nd)
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a [D, d_state] tensor")
    shape, dtype = x.shape, x.dtype
    lead, C, ds = shape[:-1], shape[-1], A.shape[1]
    ldx, ldt = _rows("x", x, shape, dtype, dev), _rows("dt", dt, shape, dtype, dev)
    ldb, ldc = _rows("Bm", Bm, (*lead, ds), dtype, dev), _rows("Cm", Cm, (*lead, ds), dtype, dev)
    ldz = 0 if z is None else _rows("z", z, shape, dtype, dev)
    _need("A", A, (C, ds), torch.float32, dev)
    _opt("D", D, (C,), torch.float32, dev)
    _opt("dt_bias", dt_bias, (C,), torch.float32, dev)
    args = (_ptr(x), ldx, _ptr(dt), ldt, _ptr(A), _ptr(Bm), ldb, _ptr(Cm), ldc, _ptr(D), _ptr(z), ldz, _ptr(dt_bias))
    return dev, lead, C, ds, _dt(x), args


@functools.lru_cache(maxsize=1024)
def _scan_workspace(device, B, N, D, ds, dt, backward):
    with torch.cuda.device(device):
        return lib.la_selective_scan_workspace(B, N, D, ds, dt, backward)


def _scan_call(fn, x, dt, A, Bm, Cm, S, D, z, dt_bias, softplus, lengths, out, stream):
    dev, (B, N), C, ds, code, args = _scan_inputs(x, dt, A, Bm, Cm, D, z, dt_bias, 3)
    _opt("lengths", lengths, (B,), torch.int32, dev)
    s, ctx = _on(dev, stream)
    try:
        out = _out("out", _zero_padding(out, lengths, (B, N, C), x.dtype, dev), (B, N, C), x.dtype, dev)
        S = _out("S", S, (B, C, ds), torch.float32, dev)
        need = _scan_workspace(dev.index, B, N, C, ds, code, 0)
        ws = _workspace(need, dev)
        rc = getattr(lib, fn)(*args, _ptr(lengths), _ptr(out), _ptr(S), B, N, C, ds, int(softplus), code, _ptr(ws), need, s)
    finally:
        _off(ctx)
    if rc != 0:
        raise LinAttnError(fn, rc)
    return out, S


def la_selective_scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, softplus: bool = True, lengths=None, out=None,
                      S=None, stream=None):
    """Selective state space scan from the zero state: with delta = softplus(dt + dt_bias), per channel

        h_t = e^{delta A} h_{t-1} + (delta x_t) Bm_t,   out_t = (Cm_t . h_t + D x_t) silu(z_t).

    x, dt, z [B, N, D], Bm, Cm [B, N, d_state] (float32 or bfloat16; parts of the last dimension of wider tensors will
    do); A [D, d_state], D and dt_bias [D] float32.  D a multiple of 8, d_state 8, 16, 32 or 64.  lengths and padding rows
    as in la_short_conv.  Returns (out in x's dtype, final state S [B, D, d_state] float32).
    """
    return _scan_call("la_selective_scan", x, dt, A, Bm, Cm, S, D, z, dt_bias, softplus, lengths, out, stream)


def la_selective_scan_with_state(x, dt, A, Bm, Cm, S, D=None, z=None, dt_bias=None, softplus: bool = True, lengths=None,
                                 out=None, stream=None):
    """Selective scan continuing from S, which is updated in place; returns (out, S)."""
    if S is None:
        raise ValueError("la_selective_scan_with_state needs the initial state S")
    return _scan_call("la_selective_scan_with_state", x, dt, A, Bm, Cm, S, D, z, dt_bias, softplus, lengths, out, stream)


def la_selective_scan_backward(x, dt, A, Bm, Cm, dout, D=None, z=None, dt_bias=None, softplus: bool = True, S0=None,
                               dS=None, lengths=None, need_state_grad: bool = False, stream=None):
    """Gradients of la_selective_scan (la_selective_scan_with_state when S0 is given) for the upstream gradient ``dout``
    of its output (x's dtype) and, optionally, ``dS`` of its final state.  Returns (dx, ddt, dA, dBm, dCm, dD, dz,
    ddt_bias), plus dS0 when ``need_state_grad``; None for an argument not given.  Gradients of x, dt, Bm, Cm, z have x's
    dtype, the others are float32."""
    dev, (B, N), C, ds, code, args = _scan_inputs(x, dt, A, Bm, Cm, D, z, dt_bias, 3)
    _need("dout", dout, (B, N, C), x.dtype, dev)
    _opt("lengths", lengths, (B,), torch.int32, dev)
    _opt("S0", S0, (B, C, ds), torch.float32, dev)
    _opt("dS", dS, (B, C, ds), torch.float32, dev)
    s, ctx = _on(dev, stream)
    try:
        wide = lambda t: None if t is None else torch.empty(B, N, t.shape[-1], dtype=x.dtype, device=dev)  # noqa: E731
        dx, ddt, dB, dC, dz = wide(x), wide(dt), wide(Bm), wide(Cm), wide(z)
        dA, dD, dbias = torch.empty_like(A), *(None if t is None else torch.empty_like(t) for t in (D, dt_bias))
        dS0 = torch.empty(B, C, ds, dtype=torch.float32, device=dev) if need_state_grad else None
        need = _scan_workspace(dev.index, B, N, C, ds, code, 1)
        ws = _workspace(need, dev)
        rc = lib.la_selective_scan_backward(*args, _ptr(lengths), _ptr(dout), _ptr(S0), _ptr(dS), _ptr(dx), _ptr(ddt),
                                            _ptr(dA), _ptr(dB), _ptr(dC), _ptr(dD), _ptr(dz), _ptr(dbias), _ptr(dS0), B, N,
                                            C, ds, int(softplus), code, _ptr(ws), need, s)
    finally:
        _off(ctx)
    if rc != 0:
        raise LinAttnError("la_selective_scan_backward", rc)
    r = (dx, ddt, dA, dB, dC, dD, dz, dbias)
    return (*r, dS0) if need_state_grad else r


def la_selective_scan_step(x, dt, A, Bm, Cm, S, D=None, z=None, dt_bias=None, softplus: bool = True, slots=None, out=None,
                           stream=None):
    """One token of the selective scan; x, dt, z [B, D], Bm, Cm [B, d_state]; returns out [B, D] in x's dtype.

    S [n_slots, D, d_state] float32 is a pool of states: row b works in place on S[slots[b]].  slots as in
    la_gated_decode_step, unused, bad and repeated ones too.
    """
    dev, (B,), C, ds, code, args = _scan_inputs(x, dt, A, Bm, Cm, D, z, dt_bias, 2)
    n_slots = _pool(S, B, slots, (C, ds), torch.float32, dev)
    s, ctx = _on(dev, stream)
    try:
        out = _out("out", out, (B, C), x.dtype, dev)
        rc = lib.la_selective_scan_step(*args, _ptr(S), _ptr(slots), _ptr(out), B, n_slots, C, ds, int(softplus), code, s)
    finally:
        _off(ctx)
    if rc != 0:
        raise LinAttnError("la_selective_scan_step", rc)
    return out


@functools.lru_cache(maxsize=1024)
def _beam_workspace(device, G, W, k, V, dt):
    with torch.cuda.device(device):
        return lib.la_beam_select_workspace(G, W, k, V, dt)


def la_beam_select(logits, scores, k=None, finished=None, eos: int = 0, stream=None):
    """The k (default W) best continuations of each group's W beams by score + log_softmax(logits), best first.

    logits [G, W, V] (float32 or bfloat16; a part of the last dimension of a wider tensor will do), scores [G, W] float32
    accumulated log probabilities (-inf: an unused beam).  Ties go to the lowest beam and token.  Within a beam the logits
    decide; between beams scores are compared in 64 bits, with a float32 sum of exponentials for each beam: continuations
    of different beams within about 1e-6 may change places.
    finished [G, W] bool: such a beam has one continuation, token ``eos``, and keeps its score.  Logits of -inf or NaN are
    chosen only where nothing else is left.  W and k up to 64.  Returns (scores float32, parents int32, tokens int32),
    each [G, k].
    """
    dev = _first_rows("logits", logits, 3)
    G, W, V = logits.shape
    k = W if k is None else int(k)
    ld, dt = _rows("logits", logits, logits.shape, logits.dtype, dev), _dt(logits)
    _need("scores", scores, (G, W), torch.float32, dev)
    _opt("finished", finished, (G, W), torch.bool, dev)
    s, ctx = _on(dev, stream)
    try:
        best = torch.empty((G, max(k, 0)), dtype=torch.float32, device=dev)
        parents, tokens = (torch.empty((G, max(k, 0)), dtype=torch.int32, device=dev) for _ in range(2))
        need = _beam_workspace(dev.index, G, W, k, V, dt)
        ws = _workspace(need, dev)
        rc = lib.la_beam_select(_ptr(logits), ld, _ptr(scores), _ptr(finished), _ptr(best), _ptr(parents), _ptr(tokens), G,
                                W, k, V, int(eos), dt, _ptr(ws), need, s)
    finally:
        _off(ctx)
    if rc != 0:
        raise LinAttnError("la_beam_select", rc)
    return best, parents, tokens


def la_beam_reorder(pools, slots, parents, stream=None):
    """Pools of states follow the beams that la_beam_select chose; returns the new slots [G, W].

    pools: contiguous tensors [n_slots, ...] of any dtype (rows of a multiple of 16 bytes), changed in place; slots [G, W]
    int32: each beam's row in every pool; parents [G, W] int32.  A beam's first child keeps its slot, the others get the
    slots of the group's childless beams (lowest first) with a copy of their parent's rows; a negative parent gets one
    without a copy.  A parent or slot out of range, and a slot that two beams have, are not copied to, and the next
    device_status() is 1.
    """
    if isinstance(pools, torch.Tensor):
        pools = [pools]
    if not isinstance(slots, torch.Tensor) or slots.dim() != 2 or not slots.is_cuda:
        raise ValueError("slots must be a contiguous 2-d CUDA tensor")
    dev, (G, W) = slots.device, slots.shape
    _need("slots", slots, (G, W), torch.int32, dev)
    _need("parents", parents, (G, W), torch.int32, dev)
    n = len(pools)
    at, rows, n_slots = (_vp * max(n, 1))(), (_sz * max(n, 1))(), None
    for i, p in enumerate(pools):
        if not isinstance(p, torch.Tensor) or p.dim() < 1 or p.get_device() != dev.index or not p.is_contiguous():
            raise ValueError(f"pools[{i}] must be a contiguous [n_slots, ...] tensor on {dev}")
        if n_slots not in (None, p.shape[0]):
            raise ValueError(f"pools[{i}] has {p.shape[0]} slots, pools[0] has {n_slots}")
        n_slots = p.shape[0]
        at[i], rows[i] = p.data_ptr() or None, p.nbytes // n_slots if n_slots else 0
    s, ctx = _on(dev, stream)
    try:
        new = torch.empty_like(slots)
        rc = lib.la_beam_reorder(at, rows, n, _ptr(slots), _ptr(parents), _ptr(new), G, W, n_slots or 0, s)
    finally:
        _off(ctx)
    if rc != 0:
        raise LinAttnError("la_beam_reorder", rc)
    return new


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
