"""ctypes binding of the state-space block's operators (``la_linear``,
``la_causal_conv``, ``la_causal_conv_step``, ``la_selective_scan``,
``la_selective_step`` in include/linattn.h).

Argument marshalling only, as in ``_binding``.  Unlike the attention entry
points these take strided views: the last axis is contiguous, the others may
have any stride that is a multiple of 16 bytes, so the parts of a projection's
output are passed as slices.  With an explicit ``stream`` the outputs are
allocated for that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import struct

import torch

from ._binding import _DT, _check, load

_ACT = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "softplus": 4}


class LaRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int), ("B", ctypes.c_int64),
                ("n", ctypes.c_int64), ("d", ctypes.c_int64), ("stride_b", ctypes.c_int64),
                ("stride_n", ctypes.c_int64)]


_vp, _i, _R = ctypes.c_void_p, ctypes.c_int, ctypes.c_char_p
# la_rows arguments are passed as the bytes of the structure: packing them
# costs a third of building a ctypes structure, and a decoding step makes six
ARGTYPES = {
    "la_linear": [_R, _R, _vp, _i, _R, _R, _vp],
    "la_causal_conv": [_R, _vp, _i, _vp, _i, _vp, _vp, _R, _vp, _vp],
    "la_causal_conv_step": [_vp, _R, _vp, _i, _vp, _i, _R, _vp],
    "la_selective_scan": [_R, _R, _vp, _i, _R, _R, _vp, _R, _vp, _i, _vp, _vp, _R, _vp, _vp],
    "la_selective_step": [_vp, _R, _R, _vp, _i, _R, _R, _vp, _R, _vp, _i, _R, _vp],
}
_fns = {}


def _fn(name):
    f = _fns.get(name)
    if f is None:
        f = getattr(load(), name)
        f.argtypes, f.restype = ARGTYPES[name], ctypes.c_int
        _fns[name] = f
    return f


_pack = struct.Struct("Pi4xqqqqq").pack


def _complain(name, t, dtype):
    """The reason why a tensor was not taken."""
    if not isinstance(t, torch.Tensor):
        return TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        return ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if t.dtype is not dtype:
        return ValueError(f"{name} must be {dtype}")
    return ValueError(f"{name}'s last axis must be contiguous")


def _view3(name, t, dtype):
    """The la_rows of a [B, n, d] tensor whose last axis is contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 axes, not {t.dim()}")
    B, n, d = t.shape
    sb, sn, one = t.stride()
    if t.dtype is not dtype or not t.is_cuda or (one != 1 and d != 1):
        raise _complain(name, t, dtype)
    return _pack(t.data_ptr(), _DT[dtype], B, n, d, sb, sn)


def _view2(name, t, dtype):
    """The la_rows [B, 1, d] of a [B, d] tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 axes, not {t.dim()}")
    B, d = t.shape
    sb, one = t.stride()
    if t.dtype is not dtype or not t.is_cuda or (one != 1 and d != 1):
        raise _complain(name, t, dtype)
    return _pack(t.data_ptr(), _DT[dtype], B, 1, d, sb, 0)


def _matrix(name, t, dtype):
    """The la_rows [1, rows, d] of a tensor whose leading axes flatten
    without a copy."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() < 2:
        raise ValueError(f"{name} must have at least two axes")
    if t.dim() > 2:
        try:
            t = t.view(-1, t.shape[-1]) if t.numel() else t.new_empty(0, t.shape[-1])
        except RuntimeError:
            raise ValueError(f"{name}'s leading axes must flatten without a copy") from None
    rows, d = t.shape
    sn, one = t.stride()
    if t.dtype is not dtype or not t.is_cuda or (one != 1 and d != 1):
        raise _complain(name, t, dtype)
    return _pack(t.data_ptr(), _DT[dtype], 1, rows, d, 0, sn)


def _dense(name, t, dtype, shape):
    """Pointer of a dense tensor of the given type and shape; None for None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype or not t.is_cuda:
        raise _complain(name, t, dtype)
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _dtype_of(x):
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dtype not in _DT:
        raise ValueError(f"x: unsupported dtype {x.dtype}")
    return x.dtype


def _act(activation):
    try:
        return _ACT[activation]
    except (KeyError, TypeError):
        raise ValueError(f"activation must be one of {sorted(_ACT)}") from None


def _stream(stream, x):
    """The handle of ``stream``, or of the current stream of x's device (whose
    raw getter is asked first: it costs a thirtieth of building a Stream)."""
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(x.device.index)
        return torch.cuda.current_stream(x.device).cuda_stream
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _alloc_on(stream):
    """Allocations inside belong to ``stream``, so that they are not handed out
    again while work queued there still uses them."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def _new(stream, shape, like, dtype):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with _alloc_on(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def linear(x, weight, bias=None, activation="none", residual=None, out=None, stream=None):
    """la_linear: act(x·weightᵀ + bias) + residual.  x [..., K], weight [N, K],
    bias [N], residual [..., N], all bf16 or all fp32; activation "none",
    "relu", "silu", "gelu" or "softplus".  K and N are multiples of 8 (bf16)
    or 4 (fp32).  ``out`` may be ``residual``.  Returns out [..., N]."""
    dt = _dtype_of(x)
    act = _act(activation)
    xd = _matrix("x", x, dt)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be an [N, K] tensor")
    wd = _matrix("weight", weight, dt)
    N = weight.shape[0]
    shape = x.shape[:-1] + (N,)
    bp = _dense("bias", bias, dt, (N,))
    rd = None
    if residual is not None:
        rd = _matrix("residual", residual, dt)
        if residual.shape != shape:
            raise ValueError(f"residual must have the shape {tuple(shape)}")
    if out is None:
        out = _new(stream, shape, x, dt)
    elif isinstance(out, torch.Tensor) and out.shape != shape:
        raise ValueError(f"out must have the shape {tuple(shape)}")
    od = _matrix("out", out, dt)
    _check("la_linear", _fn("la_linear")(xd, wd, bp, act, rd, od, _stream(stream, x)))
    return out


def causal_conv(x, weight, bias=None, activation="silu", state=None, lengths=None, out=None,
                return_state=False, stream=None):
    """la_causal_conv: depthwise causal convolution over a prompt.  x [B, n, D],
    weight [D, W] (W 2 to 4, the newest input meets the last column), bias
    [D]; activation "silu" or "none"; ``state`` [B, W−1, D] the inputs before
    the prompt (None: zeros); ``lengths`` [B] int32: later tokens are not read
    and give 0.  Returns out, or (out, state after the prompt)."""
    dt = _dtype_of(x)
    act = _act(activation)
    xd = _view3("x", x, dt)
    B, n, D = x.shape
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a [D, W] tensor")
    W = weight.shape[1]
    wp = _dense("weight", weight, dt, (D, W))
    bp = _dense("bias", bias, dt, (D,))
    sp = _dense("state", state, dt, (B, W - 1, D))
    lp = _dense("lengths", lengths, torch.int32, (B,))
    if out is None:
        out = _new(stream, (B, n, D), x, dt)
    od = _view3("out", out, dt)
    after = _new(stream, (B, max(W - 1, 0), D), x, dt) if return_state else None
    _check("la_causal_conv", _fn("la_causal_conv")(
        xd, wp, W, bp, act, sp, lp, od, after.data_ptr() if return_state else None,
        _stream(stream, x)))
    return (out, after) if return_state else out


def causal_conv_step(state, x, weight, bias=None, activation="silu", out=None, stream=None):
    """la_causal_conv_step: the convolution's next token.  state [B, W−1, D] is
    shifted in place; x [B, D].  Returns out [B, D]."""
    dt = _dtype_of(x)
    act = _act(activation)
    xd = _view2("x", x, dt)
    B, D = x.shape
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a [D, W] tensor")
    W = weight.shape[1]
    wp = _dense("weight", weight, dt, (D, W))
    bp = _dense("bias", bias, dt, (D,))
    if state is None:
        raise TypeError("state must be a torch.Tensor")
    sp = _dense("state", state, dt, (B, W - 1, D))
    if out is None:
        out = _new(stream, (B, D), x, dt)
    od = _view2("out", out, dt)
    _check("la_causal_conv_step", _fn("la_causal_conv_step")(
        sp, xd, wp, W, bp, act, od, _stream(stream, x)))
    return out


def _scan_args(x, dt, a, b, c, skip, gate, dt_bias, view):
    ty = _dtype_of(x)
    xd = view("x", x, ty)
    dd = view("dt", dt, ty)
    if not isinstance(a, torch.Tensor) or a.dim() != 2:
        raise ValueError("a must be a [D, S] tensor")
    D, S = x.shape[-1], a.shape[1]
    ap = _dense("a", a, torch.float32, (D, S))
    bd = view("b", b, ty)
    cd = view("c", c, ty)
    kp = _dense("skip", skip, torch.float32, (D,))
    gd = view("gate", gate, ty) if gate is not None else None
    tp = _dense("dt_bias", dt_bias, torch.float32, (D,))
    return ty, S, xd, dd, ap, bd, cd, kp, gd, tp


def selective_scan(x, dt, a, b, c, skip=None, gate=None, dt_bias=None, softplus=True, state=None,
                   lengths=None, out=None, return_state=False, stream=None):
    """la_selective_scan: h ← exp(Δ·a)·h + Δ·x·b, out = (Σ c·h + skip·x)·silu(gate)
    with Δ = softplus(dt + dt_bias) (or dt + dt_bias).  x, dt, gate [B, n, D]
    and b, c [B, n, S] bf16 or fp32; a [D, S], skip [D], dt_bias [D] and
    ``state`` [B, D, S] fp32; ``lengths`` [B] int32: later tokens are not read,
    leave the state alone and give 0.  S is 8, 16, 32 or 64.  Returns out, or
    (out, state after the prompt)."""
    ty, S, xd, dd, ap, bd, cd, kp, gd, tp = _scan_args(x, dt, a, b, c, skip, gate, dt_bias, _view3)
    B, n, D = x.shape
    sp = _dense("state", state, torch.float32, (B, D, S))
    lp = _dense("lengths", lengths, torch.int32, (B,))
    if out is None:
        out = _new(stream, (B, n, D), x, ty)
    od = _view3("out", out, ty)
    after = _new(stream, (B, D, S), x, torch.float32) if return_state else None
    _check("la_selective_scan", _fn("la_selective_scan")(
        xd, dd, ap, S, bd, cd, kp, gd, tp, int(bool(softplus)), sp, lp, od,
        after.data_ptr() if return_state else None, _stream(stream, x)))
    return (out, after) if return_state else out


def selective_step(state, x, dt, a, b, c, skip=None, gate=None, dt_bias=None, softplus=True,
                   out=None, stream=None):
    """la_selective_step: the recurrence's next token.  state [B, D, S] fp32 is
    updated in place; x, dt, gate [B, D]; b, c [B, S]; the rest as
    ``selective_scan``.  Returns out [B, D]."""
    ty, S, xd, dd, ap, bd, cd, kp, gd, tp = _scan_args(x, dt, a, b, c, skip, gate, dt_bias,
                                                       _view2)
    if state is None:
        raise TypeError("state must be a torch.Tensor")
    shape = x.shape
    sp = _dense("state", state, torch.float32, shape + (S,))
    if out is None:
        out = _new(stream, shape, x, ty)
    od = _view2("out", out, ty)
    _check("la_selective_step", _fn("la_selective_step")(
        sp, xd, dd, ap, S, bd, cd, kp, gd, tp, int(bool(softplus)), od, _stream(stream, x)))
    return out
