"""The state-space block's operators (``la_linear``, ``la_causal_conv``,
``la_causal_conv_step``, ``la_selective_scan``, ``la_selective_step`` in
include/linattn.h).

Arguments are checked and marshalled in C++ (``csrc/py_block.cpp``, built as
``la_block.so``): a decoding step's kernels are shorter than the same work in
Python.  Unlike the attention entry points these take strided views: the last
axis is contiguous, the others may have any stride that is a multiple of 16
bytes, so the parts of a projection's output are passed as slices.  With an
explicit ``stream`` the outputs are allocated for that stream.  An ``out`` that
is given lies on no input, except the same view where a function says so.

They have no backward.  Outputs of inputs that require a gradient carry a node that
raises when a gradient reaches it; such inputs are refused with a given ``out``,
and a state that is updated in place may not require one unless one of these
functions returned it (``torch.no_grad()`` lifts both).
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading

import torch

from . import build as _build
from ._binding import _check, load

_NAMES = ("la_linear", "la_causal_conv", "la_causal_conv_step", "la_selective_scan",
          "la_selective_step")
_lock = threading.Lock()
_ext = None


class _NoBackward(torch.autograd.Function):
    """Outputs as they are, behind a node that has no gradient to give."""

    @staticmethod
    def forward(ctx, name, outs, *inputs):
        ctx.name = name
        return outs[0] if len(outs) == 1 else outs

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.name} has no backward: a gradient reached its output "
                           "(call it under torch.no_grad(), or detach its inputs)")


def _no_backward(name, result, inputs):
    return _NoBackward.apply(name, result if isinstance(result, tuple) else (result,), *inputs)


def _load_ext():
    """The la_block module, bound to the loaded library's functions."""
    global _ext
    with _lock:
        if _ext is None:
            lib = load()
            path = _build.EXT_PATH
            if not os.path.exists(path):
                raise RuntimeError(f"la_block.so is not built ({path}); run "
                                   "`python -m causal_kernelized_linear_gb300.build`")
            if _build.ext_built_for() != _build._ext_target():
                raise RuntimeError(f"la_block.so is built for {_build.ext_built_for() or 'an unknown PyTorch'}, "
                                   f"this is {_build._ext_target()}; run "
                                   "`python -m causal_kernelized_linear_gb300.build`")
            loader = importlib.machinery.ExtensionFileLoader("la_block", path)
            ext = importlib.util.module_from_spec(
                importlib.util.spec_from_file_location("la_block", path, loader=loader))
            loader.exec_module(ext)
            ext.bind(_check, _no_backward, *[ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
                               for n in _NAMES])
            _ext = ext
    return _ext


def linear(x, weight, bias=None, activation="none", residual=None, out=None, stream=None):
    """la_linear: act(x·weightᵀ + bias) + residual.  x [..., K], weight [N, K],
    bias [N], residual [..., N], all bf16 or all fp32; activation "none",
    "relu", "silu", "gelu" or "softplus".  K and N are multiples of 8 (bf16)
    or 4 (fp32).  ``out`` may be ``residual``.  Returns out [..., N]."""
    return (_ext or _load_ext()).linear(x, weight, bias, activation, residual, out, stream)


def causal_conv(x, weight, bias=None, activation="silu", state=None, lengths=None, out=None,
                return_state=False, stream=None):
    """la_causal_conv: depthwise causal convolution over a prompt.  x [B, n, D],
    weight [D, W] (W 2 to 4, the newest input meets the last column), bias
    [D]; activation "silu" or "none"; ``state`` [B, W−1, D] the inputs before
    the prompt (None: zeros); ``lengths`` [B] int32: later tokens are not read
    and give 0.  Returns out, or (out, state after the prompt)."""
    return (_ext or _load_ext()).causal_conv(x, weight, bias, activation, state, lengths, out,
                                             return_state, stream)


def causal_conv_step(state, x, weight, bias=None, activation="silu", out=None, stream=None):
    """la_causal_conv_step: the convolution's next token.  state [B, W−1, D] is
    shifted in place; x [B, D]; ``out`` may be x.  Returns out [B, D]."""
    return (_ext or _load_ext()).causal_conv_step(state, x, weight, bias, activation, out, stream)


def selective_scan(x, dt, a, b, c, skip=None, gate=None, dt_bias=None, softplus=True, state=None,
                   lengths=None, out=None, return_state=False, stream=None):
    """la_selective_scan: h ← exp(Δ·a)·h + Δ·x·b, out = (Σ c·h + skip·x)·silu(gate)
    with Δ = softplus(dt + dt_bias) (or dt + dt_bias).  x, dt, gate [B, n, D]
    and b, c [B, n, S] bf16 or fp32; a [D, S], skip [D], dt_bias [D] and
    ``state`` [B, D, S] fp32; ``lengths`` [B] int32: later tokens are not read,
    leave the state alone and give 0.  S is 8, 16, 32 or 64.  ``out`` may be x, dt
    or gate.  Returns out, or (out, state after the prompt)."""
    return (_ext or _load_ext()).selective_scan(x, dt, a, b, c, skip, gate, dt_bias, softplus,
                                                state, lengths, out, return_state, stream)


def selective_step(state, x, dt, a, b, c, skip=None, gate=None, dt_bias=None, softplus=True,
                   out=None, stream=None):
    """la_selective_step: the recurrence's next token.  state [B, D, S] fp32 is
    updated in place; x, dt, gate [B, D]; b, c [B, S]; the rest as
    ``selective_scan``, out included.  Returns out [B, D]."""
    return (_ext or _load_ext()).selective_step(state, x, dt, a, b, c, skip, gate, dt_bias,
                                                softplus, out, stream)
