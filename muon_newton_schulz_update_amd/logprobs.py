"""Log probabilities of given tokens under a language-model head, with the
distribution's entropy and its likeliest tokens, and the gradient of the first
two. Argument marshalling only, like the package's other entry points; the
kernels are reached through libmuon's C ABI (include/libmuon.h).

    out = mu.linear_logprobs(hidden, head, tokens, top=5)          # no logits are stored
    out.logprobs, out.entropy, out.top_logprobs, out.top_tokens    # the first two differentiable
    dhidden, dhead = mu.linear_logprobs_grad(hidden, head, tokens, out.stats, grad_logprobs=g, grad_entropy=e)
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import load_library
from .training import _checked, _describe, _handle_for, _one_stream_a_leaf, _scalar


class LogProbConfig(ctypes.Structure):
    _fields_ = [("top", ctypes.c_int32), ("softcap", ctypes.c_float), ("ignore_index", ctypes.c_int64)]


class LogProbs(NamedTuple):
    """Float32, of the tokens' shape; top_logprobs and top_tokens (int64) with one dimension more, None with top 0.
    stats, the tokens' shape and 4, is what `linear_logprobs_grad` needs of the call."""
    logprobs: torch.Tensor
    entropy: torch.Tensor
    top_logprobs: torch.Tensor | None
    top_tokens: torch.Tensor | None
    stats: torch.Tensor


def _head_args(hidden, weight, targets, top, softcap, ignore_index, handle):
    if hidden.dim() < 1 or targets.shape != hidden.shape[:-1]:
        raise ValueError(f"targets of shape {tuple(targets.shape)} for hidden states of {tuple(hidden.shape)}")
    if weight.dim() != 2:
        raise ValueError(f"weight: expected a 2-D tensor, got shape {tuple(weight.shape)}")
    if targets.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"targets: dtype {targets.dtype} is not int64 or int32")
    if not targets.is_contiguous():
        raise ValueError("targets must be contiguous")
    h = _handle_for((weight, hidden), handle)
    if targets.numel() and targets.get_device() != h.device:
        raise ValueError(f"targets: expected a tensor on GPU {h.device}, got {targets.device}")
    return h, LogProbConfig(int(top), float(softcap), int(ignore_index))


def _call(hidden, weight, targets, top, softcap, ignore_index, handle):
    h, cfg = _head_args(hidden, weight, targets, top, softcap, ignore_index, handle)
    words, at = _describe().pack_rows((hidden, weight), ("hidden", "weight"), h.device)
    device = torch.device("cuda", h.device)
    new = lambda *more, dtype=torch.float32: torch.empty((*targets.shape, *more), device=device, dtype=dtype)
    stats = new(4)
    logprobs, entropy = _describe().empty(h.device, targets), _describe().empty(h.device, targets)
    top_logprobs = top_tokens = None
    if cfg.top > 0:
        top_logprobs, top_tokens = new(cfg.top), new(cfg.top, dtype=torch.int64)
    h._check(h._lib.linear_logprobs(h.ptr, at, at + len(words) // 2, targets.data_ptr(), targets.element_size(),
                                    ctypes.byref(cfg), logprobs.data_ptr(), entropy.data_ptr(), stats.data_ptr(),
                                    top_logprobs.data_ptr() if cfg.top > 0 else None,
                                    top_tokens.data_ptr() if cfg.top > 0 else None))
    return logprobs, entropy, top_logprobs, top_tokens, stats


def linear_logprobs_grad(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, stats: torch.Tensor, *,
                         grad_logprobs: torch.Tensor | None = None, grad_entropy: torch.Tensor | None = None,
                         ignore_index: int = -100, softcap: float = 0.0, dhidden: torch.Tensor | None | bool = None,
                         dweight: torch.Tensor | None | bool = None, handle=None):
    """(dhidden, dweight): gradient of sum(grad_logprobs * logprobs + grad_entropy *
    entropy) of `linear_logprobs` on the same inputs, whose stats it takes
    (libmuon `linear_logprobs_grad`). It takes the logits again, a piece of
    tokens at a time; a piece's gradient of them (2 bytes each, float32 4) takes up
    to 1 GiB of the handle. grad_logprobs, grad_entropy: float32, one a token;
    one of them may be None. dhidden, dweight: tensors to write to; False leaves
    that gradient out (and its product)."""
    h, cfg = _head_args(hidden, weight, targets, 0, softcap, ignore_index, handle)
    d, n = h.device, targets.numel()
    native = _describe()
    at_stats = _scalar(stats, "stats", d, 4 * n)
    go = [_scalar(g, what, d, n) for g, what in ((grad_logprobs, "grad_logprobs"), (grad_entropy, "grad_entropy"))]
    outs = []
    for out, like, what in ((dhidden, hidden, "dhidden"), (dweight, weight, "dweight")):
        if out is None:
            out = native.empty(d, like, like)
        elif out is False:
            out = None
        elif out.shape != like.shape:
            raise ValueError(f"{what} of shape {tuple(out.shape)} for {tuple(like.shape)}")
        outs.append(out)
    words, at = native.pack_rows((hidden, weight, *outs), ("hidden", "weight", "dhidden", "dweight"), d)
    size = len(words) // 4
    h._check(h._lib.linear_logprobs_grad(h.ptr, at, at + size, targets.data_ptr(), targets.element_size(), ctypes.byref(cfg),
                                         at_stats, *go, *(None if o is None else at + size * (2 + i) for i, o in enumerate(outs))))
    return tuple(outs)


class _LinearLogProbs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, targets, top, softcap, ignore_index, handle):
        _one_stream_a_leaf((hidden, weight))
        out = _call(hidden, weight, targets, top, softcap, ignore_index, handle)
        ctx.options = (softcap, ignore_index, handle)
        ctx.save_for_backward(hidden, weight, targets, out[4])
        ctx.mark_non_differentiable(*(t for t in out[2:] if t is not None))
        ctx.set_materialize_grads(False)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_logprobs, grad_entropy, *_):
        # (a handle that was given serves the backward too; without one, the
        # thread that runs it has its own)
        softcap, ignore_index, handle = ctx.options
        if grad_logprobs is None and grad_entropy is None:
            return (None,) * 7
        hidden, weight, targets, stats = ctx.saved_tensors
        grads = (None if g is None else g.contiguous() for g in (grad_logprobs, grad_entropy))
        need = ctx.needs_input_grad
        dh, dw = linear_logprobs_grad(hidden, weight, targets, stats, **dict(zip(("grad_logprobs", "grad_entropy"), grads)),
                                      ignore_index=ignore_index, softcap=softcap, dhidden=None if need[0] else False,
                                      dweight=None if need[1] else False, handle=handle)
        return dh, dw, None, None, None, None, None


def linear_logprobs(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, *, top: int = 0,
                    ignore_index: int = -100, softcap: float = 0.0, handle=None) -> LogProbs:
    """Log probabilities of the tokens `targets` under the logits hidden weight^T,
    the entropy of each token's distribution, and its `top` (up to 32) likeliest
    tokens with their log probabilities, in falling order, equal logits by rising
    token (libmuon `linear_logprobs`). No logits are stored.

    hidden: (..., D), targets: (...) int64 or int32, weight: (V, D). Tokens whose
    target is ignore_index have zeros, and -1 for their alternatives. logprobs and
    entropy are differentiable in hidden and weight, in reverse mode: the
    backward pass takes the logits again (`linear_logprobs_grad`). A graph that
    captures it with its backward pass needs its leaves without eager results on
    other streams; the gradient's own call has no such condition."""
    if torch.is_grad_enabled() and (hidden.requires_grad or weight.requires_grad):
        return LogProbs(*_LinearLogProbs.apply(hidden, weight, targets, top, softcap, ignore_index, handle))
    return LogProbs(*_call(hidden, weight, targets, top, softcap, ignore_index, handle))


# ---------------------------------------------------------------------------
# host-only validation (no device needed); descriptors are MuonMatrix objects
# ---------------------------------------------------------------------------
def _ref(m):
    return None if m is None else ctypes.byref(m)


def check_logprob_args(hidden, weight, targets=4096, target_bytes=8, cfg: LogProbConfig | None = None, logprobs=1 << 20,
                       entropy=None, stats=None, top_logprobs=None, top_tokens=None) -> tuple[int, str]:
    return _checked(load_library().muon_check_logprob_args, _ref(hidden), _ref(weight), targets, target_bytes, _ref(cfg),
                    logprobs, entropy, stats, top_logprobs, top_tokens)


def check_logprob_grad_args(hidden, weight, targets=4096, target_bytes=8, cfg: LogProbConfig | None = None, stats=1 << 20,
                            grad_logprobs=1 << 16, grad_entropy=None, dhidden=None, dweight=None) -> tuple[int, str]:
    return _checked(load_library().muon_check_logprob_grad_args, _ref(hidden), _ref(weight), targets, target_bytes,
                    _ref(cfg), stats, grad_logprobs, grad_entropy, _ref(dhidden), _ref(dweight))
