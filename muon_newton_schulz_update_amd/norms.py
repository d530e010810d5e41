"""Norms after and before a block, fused with the block's gate and the
residual's scale, with their gradient. Argument marshalling only, like the
package's other entry points; the kernels are reached through libmuon's C ABI
(include/libmuon.h).

    h = mu.rms_norm(x, gain)                                       # before the first block
    x, h = mu.residual_norm(x, block(h), post_gain=a, gate=g, scale=s, pre_gain=b)   # between two
    dx, dgain = mu.rms_norm_grad(x, dh, gain)
    grads = mu.residual_norm_grad(x, y, dx, dh, post_gain=a, gate=g, scale=s, pre_gain=b)
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import load_library
from .training import _checked, _describe, _handle_for, _one_stream_a_leaf


class NormParams(ctypes.Structure):
    _fields_ = [("post_gain", ctypes.c_void_p), ("pre_gain", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("post_norm", ctypes.c_int32), ("pre_norm", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class _GradPointers(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in ("x", "y", "post_gain", "gate", "scale", "pre_gain")]


class NormGrads(NamedTuple):
    """Gradients of `residual_norm`'s inputs; None for what was not given or not asked for."""
    x: torch.Tensor | None
    y: torch.Tensor | None
    post_gain: torch.Tensor | None
    gate: torch.Tensor | None
    scale: torch.Tensor | None
    pre_gain: torch.Tensor | None


_entries = None


def _entry(i: int) -> int:
    """Address of a C entry point, for the native binding."""
    global _entries
    if _entries is None:
        lib = load_library()
        _entries = [ctypes.cast(f, ctypes.c_void_p).value for f in (lib.residual_norm, lib.residual_norm_grad)]
    return _entries[i]


def _forward(x, y, post_gain, gate, scale, pre_gain, post_norm, pre_norm, eps, dtype, handle):
    h = _handle_for((x,), handle)
    status, out, hidden = _describe().residual_norm(_entry(0), h.ptr.value or 0, h.device, (x, y, post_gain, gate, scale, pre_gain),
                                                    post_norm, pre_norm, eps, dtype)
    h._check(status)
    return out, hidden


def _backward(x, y, post_gain, gate, scale, pre_gain, post_norm, pre_norm, eps, dout, dhidden, wanted, handle):
    h = _handle_for((x,), handle)
    status, grads = _describe().residual_norm_grad(_entry(1), h.ptr.value or 0, h.device, (x, y, post_gain, gate, scale, pre_gain),
                                                   dout, dhidden, wanted, post_norm, pre_norm, eps)
    h._check(status)
    return NormGrads(*grads)


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, post_gain, gate, scale, pre_gain, *options):
        post_norm, pre_norm, eps, dtype, handle = ctx.options = options
        _one_stream_a_leaf((x, y, post_gain, gate, scale, pre_gain))
        ctx.save_for_backward(x, y, post_gain, gate, scale, pre_gain)
        ctx.set_materialize_grads(False)
        return _forward(x, y, post_gain, gate, scale, pre_gain, post_norm, pre_norm, eps, dtype, handle)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, dhidden):
        # (a handle that was given serves the backward too; without one, the
        # thread that runs it has its own)
        post_norm, pre_norm, eps, _, handle = ctx.options
        none = (None,) * 11
        if dout is None and dhidden is None:
            return none
        dout, dhidden = (None if g is None else g.contiguous() for g in (dout, dhidden))
        return (*_backward(*ctx.saved_tensors, post_norm, pre_norm, eps, dout, dhidden, ctx.needs_input_grad[:6], handle),
                *none[6:])


def _differentiable(*tensors):
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def rms_norm(x: torch.Tensor, gain: torch.Tensor | None = None, *, eps: float = 1e-6, dtype: torch.dtype | None = None,
             handle=None) -> torch.Tensor:
    """x / sqrt(mean(x^2) + eps) * gain over the last dimension (libmuon
    `residual_norm` of x alone), of x's type or, for a float32 x, of a bfloat16
    dtype. Differentiable in x and gain, in reverse mode."""
    args = (x, None, None, None, None, gain, False, True, eps, None if dtype in (None, x.dtype) else dtype, handle)
    return (_ResidualNorm.apply if _differentiable(x, gain) else _forward)(*args)[1]


def rms_norm_grad(x: torch.Tensor, dhidden: torch.Tensor, gain: torch.Tensor | None = None, *, eps: float = 1e-6,
                  handle=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """(dx, dgain): gradient of `rms_norm` for the gradient dhidden of its result."""
    grads = _backward(x, None, None, None, None, gain, False, True, eps, None, dhidden, (True,) * 6, handle)
    return grads.x, grads.pre_gain


def residual_norm(x: torch.Tensor, y: torch.Tensor, *, post_norm: bool = True, post_gain: torch.Tensor | None = None,
                  gate: torch.Tensor | None = None, scale: torch.Tensor | None = None, pre_norm: bool = True,
                  pre_gain: torch.Tensor | None = None, eps: float = 1e-6,
                  handle=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """(out, hidden): the residual stream after a block, scale x + gate norm(y),
    and its norm, which the next block starts from (libmuon `residual_norm`).

    x, y: (..., D), D up to 16384, of one type, or y bfloat16 beside a float32 x;
    out has x's type, hidden y's. norm(y) = y / sqrt(mean(y^2) + eps) * post_gain,
    or y itself without post_norm; hidden likewise from out with pre_gain, None
    without pre_norm. Gains: (D,). gate: one value, (D,), or y's shape and type.
    scale: one value or (D,). Differentiable in every tensor, in reverse mode; the
    backward pass makes out again from x and y and keeps nothing else. A graph that
    captures it with its backward pass needs its leaves without eager results on
    other streams; `residual_norm_grad` has no such condition."""
    args = (x, y, post_gain, gate, scale, pre_gain, post_norm, pre_norm, eps, None, handle)
    return (_ResidualNorm.apply if _differentiable(x, y, post_gain, gate, scale, pre_gain) else _forward)(*args)


def residual_norm_grad(x: torch.Tensor, y: torch.Tensor, dout: torch.Tensor | None, dhidden: torch.Tensor | None, *,
                       post_norm: bool = True, post_gain: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                       scale: torch.Tensor | None = None, pre_norm: bool = True, pre_gain: torch.Tensor | None = None,
                       eps: float = 1e-6, handle=None) -> NormGrads:
    """Gradients of `residual_norm`'s tensors, each of its own type and shape, for
    the gradients of its results; one of the two may be None (zero)."""
    return _backward(x, y, post_gain, gate, scale, pre_gain, post_norm, pre_norm, eps, dout, dhidden, (True,) * 6, handle)


# ---------------------------------------------------------------------------
# host-only validation (no device needed); descriptors are MuonMatrix objects
# ---------------------------------------------------------------------------
def _params(post_gain, pre_gain, gate, scale, post_norm, pre_norm, eps):
    address = lambda m: None if m is None else ctypes.addressof(m)
    return ctypes.byref(NormParams(address(post_gain), address(pre_gain), address(gate), address(scale), post_norm,
                                   pre_norm, eps))


def _ref(m):
    return None if m is None else ctypes.byref(m)


def check_residual_norm_args(x, y=None, out=None, hidden=None, *, post_gain=None, pre_gain=None, gate=None, scale=None,
                             post_norm=1, pre_norm=1, eps=1e-6) -> tuple[int, str]:
    return _checked(load_library().muon_check_residual_norm_args, _ref(x), _ref(y),
                    _params(post_gain, pre_gain, gate, scale, post_norm, pre_norm, eps), _ref(out), _ref(hidden))


def check_residual_norm_grad_args(x, y=None, dout=None, dhidden=None, grads=None, *, post_gain=None, pre_gain=None,
                                  gate=None, scale=None, post_norm=1, pre_norm=1, eps=1e-6) -> tuple[int, str]:
    """grads: a dict of gradients by input ("x", "y", "post_gain", ...), or None."""
    pointers = None if grads is None else ctypes.byref(_GradPointers(**{k: ctypes.addressof(m) for k, m in grads.items()}))
    return _checked(load_library().muon_check_residual_norm_grad_args, _ref(x), _ref(y),
                    _params(post_gain, pre_gain, gate, scale, post_norm, pre_norm, eps), _ref(dout), _ref(dhidden), pointers)
