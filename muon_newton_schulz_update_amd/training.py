"""The rest of a training step around the Muon update: the head's softmax
cross entropy with its gradient, the global gradient norm with clipping, and
AdamW for the parameters Muon does not take. Argument marshalling only, like
the package's other entry points; the kernels are reached through libmuon's C
ABI (include/libmuon.h).

    loss = mu.linear_cross_entropy(hidden, head, targets)      # differentiable
    loss, dhidden, dhead = mu.linear_cross_entropy_grad(hidden, head, targets)
    norm, coef = mu.grad_norm(grads, max_norm=1.0)             # both stay on the device
    mu.adamw_update(grads, exp_avgs, exp_avg_sqs, weights, step=1, lr=3e-3, grad_scale=coef)
    norm = mu.clip_grad_norm(matrix_grads, 1.0)                # in place
"""
from __future__ import annotations

import ctypes
from typing import Sequence

import torch

from . import MuonMatrix, get_handle, load_library

REDUCTIONS = {"none": 0, "sum": 1, "mean": 2}


class AdamWConfig(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float), ("step", ctypes.c_int64),
                ("step_at", ctypes.c_void_p), ("lr_at", ctypes.c_void_p)]


class LossConfig(ctypes.Structure):
    _fields_ = [("reduction", ctypes.c_int32), ("softcap", ctypes.c_float), ("ignore_index", ctypes.c_int64)]


# ---------------------------------------------------------------------------
# descriptors: packed natively (csrc/describe.cpp) into bytes, whose address
# the C ABI takes. A matrix keeps its row stride; anything else (a vector, a
# contiguous tensor of more dimensions) is one row.
# ---------------------------------------------------------------------------
_native = None


def _describe():
    global _native
    if _native is None:
        try:
            from . import _describe as module
        except ImportError as e:
            raise RuntimeError("the _describe extension is missing or does not load: build it with "
                               f"`python -m muon_newton_schulz_update_amd.build` ({e})") from e
        _native = module
    return _native


def _handle_for(tensors, handle):
    if handle is None:
        device = _describe().device_of(tensors)
        handle = get_handle(None if device < 0 else device)
    stream = torch._C._cuda_getCurrentRawStream(handle.device)
    if stream != handle._stream:
        handle._bind_stream()
    return handle


def _scalar(t: torch.Tensor | None, what: str, device: int, n: int | None = None, dtype=torch.float32):
    if t is None:
        return None
    if t.dtype != dtype or t.get_device() != device:
        raise ValueError(f"{what}: expected {dtype} on GPU {device}, got {t.dtype} on {t.device}")
    if t.numel() != (1 if n is None else n) or not t.is_contiguous():
        raise ValueError(f"{what}: expected {1 if n is None else n} contiguous values, got shape {tuple(t.shape)}")
    return t.data_ptr()


# ---------------------------------------------------------------------------
# gradient norm and clipping
# ---------------------------------------------------------------------------
def grad_norm(grads: Sequence[torch.Tensor], *, max_norm: float | None = None, handle=None):
    """Global 2-norm of a list of gradients (libmuon `muon_grad_norm`), a
    float32 scalar on the device. With max_norm also the clipping coefficient
    min(1, max_norm / (norm + 1e-6)): (norm, coef), for `adamw_update`'s
    grad_scale. Nothing waits for the GPU."""
    grads = list(grads)
    h = _handle_for(grads, handle)
    native = _describe()
    words = native.pack(grads, "grads", h.device)
    norm = native.empty(h.device)
    if max_norm is None:
        h._check(h._lib.muon_grad_norm(h.ptr, len(grads), words, 0.0, norm.data_ptr(), None))
        return norm
    coef = native.empty(h.device)
    h._check(h._lib.muon_grad_norm(h.ptr, len(grads), words, max_norm, norm.data_ptr(), coef.data_ptr()))
    return norm, coef


def clip_grad_norm(grads: Sequence[torch.Tensor], max_norm: float, *, out: Sequence[torch.Tensor] | None = None,
                   handle=None) -> torch.Tensor:
    """Scale gradients so that their global norm is at most max_norm (libmuon
    `muon_clip_grad_norm`), in place or into `out`, and return the norm before
    clipping. In place, nothing is written when the norm is within the limit."""
    grads = list(grads)
    h = _handle_for(grads, handle)
    native = _describe()
    words = native.pack(grads, "grads", h.device)
    outs = None if out is None else native.pack(out, "out", h.device, grads, "grads")
    norm, coef = native.empty(h.device), native.empty(h.device)
    h._check(h._lib.muon_clip_grad_norm(h.ptr, len(grads), words, outs, max_norm, norm.data_ptr(), coef.data_ptr()))
    return norm


def scale(tensors: Sequence[torch.Tensor], coef: torch.Tensor, *, out: Sequence[torch.Tensor] | None = None,
          handle=None) -> None:
    """Multiply tensors by a scalar that lives on the device (libmuon
    `muon_scale`), in place or into `out`."""
    tensors = list(tensors)
    h = _handle_for(tensors, handle)
    pack = _describe().pack
    words = pack(tensors, "tensors", h.device)
    outs = None if out is None else pack(out, "out", h.device, tensors, "tensors")
    h._check(h._lib.muon_scale(h.ptr, len(tensors), words, outs, _scalar(coef, "coef", h.device)))


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------
_adamw_default = None


def _adamw_defaults() -> AdamWConfig:
    global _adamw_default
    if _adamw_default is None:
        cfg = AdamWConfig()
        load_library().muon_adamw_config_default(ctypes.byref(cfg))
        _adamw_default = cfg
    return _adamw_default


def adamw_update(grads: Sequence[torch.Tensor], exp_avgs: Sequence[torch.Tensor],
                 exp_avg_sqs: Sequence[torch.Tensor], weights: Sequence[torch.Tensor], *, step: int | torch.Tensor,
                 lr: float | torch.Tensor | None = None, beta1: float | None = None, beta2: float | None = None,
                 eps: float | None = None, weight_decay: float | None = None,
                 grad_scale: torch.Tensor | None = None,
                 copies: Sequence[torch.Tensor | None] | None = None, handle=None) -> None:
    """One AdamW step in place (libmuon `adamw_update`); what is not given has
    the library's default. grad_scale: a float32 device scalar that multiplies
    every gradient (`grad_norm`'s coefficient). step (int64) and lr (float32) may
    be one-element tensors on the device, read when the kernel runs: a captured
    graph repeats numbers, and counts its steps with tensors. copies[i], when
    given, receives the new weight's 32-bit value rounded to its own type, for a
    model that computes on 16-bit copies of 32-bit weights (a float32 copy of a
    bfloat16 weight is the value that the weight was rounded from)."""
    weights = list(weights)
    h = _handle_for(weights, handle)
    d, pack = h.device, _describe().pack
    w = pack(weights, "weights", d)
    lists = [pack(x, what, d, weights, "weights") for x, what in
             ((grads, "grads"), (exp_avgs, "exp_avgs"), (exp_avg_sqs, "exp_avg_sqs"))]
    cp = None if copies is None else pack(copies, "copies", d, weights, "weights")
    z = _adamw_defaults()
    step_at = lr_at = None
    if isinstance(step, torch.Tensor):
        step, step_at = 1, _scalar(step, "step", d, dtype=torch.int64)
    if isinstance(lr, torch.Tensor):
        lr, lr_at = None, _scalar(lr, "lr", d)
    cfg = AdamWConfig(z.lr if lr is None else lr, z.beta1 if beta1 is None else beta1,
                      z.beta2 if beta2 is None else beta2, z.eps if eps is None else eps,
                      z.weight_decay if weight_decay is None else weight_decay, step, step_at, lr_at)
    h._check(h._lib.adamw_update(h.ptr, len(weights), *lists, w, cp, ctypes.byref(cfg),
                                 _scalar(grad_scale, "grad_scale", d)))


# ---------------------------------------------------------------------------
# head cross entropy
# ---------------------------------------------------------------------------
def _matrix(t: torch.Tensor, what: str, device: int):
    if t.dim() != 2:
        raise ValueError(f"{what}: expected a 2-D tensor, got shape {tuple(t.shape)}")
    return _describe().pack((t,), what, device)


def _loss_call(hidden, weight, targets, ignore_index, reduction, softcap, grad_out, dhidden, dweight, grad, handle):
    if reduction not in REDUCTIONS:
        raise ValueError(f"unknown reduction {reduction!r}")
    if hidden.dim() < 1 or targets.shape != hidden.shape[:-1]:
        raise ValueError(f"targets of shape {tuple(targets.shape)} for hidden states of {tuple(hidden.shape)}")
    if targets.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"targets: dtype {targets.dtype} is not int64 or int32")
    if not targets.is_contiguous():
        raise ValueError("targets must be contiguous")
    h = _handle_for((weight, hidden), handle)
    d = h.device
    if targets.numel() and targets.get_device() != d:
        raise ValueError(f"targets: expected a tensor on GPU {d}, got {targets.device}")
    hid = hidden if hidden.dim() == 2 else hidden.view(-1, hidden.shape[-1])
    n = hid.shape[0]
    native = _describe()
    loss = native.empty(d, targets if reduction == "none" else None)
    cfg = LossConfig(REDUCTIONS[reduction], float(softcap), int(ignore_index))
    args = (h.ptr, _matrix(hid, "hidden", d), _matrix(weight, "weight", d), targets.data_ptr(),
            targets.element_size(), ctypes.byref(cfg))
    if not grad:
        h._check(h._lib.linear_cross_entropy(*args, loss.data_ptr()))
        return loss, None, None
    go = _scalar(grad_out, "grad_out", d, n if reduction == "none" else None)
    dh = dw = None
    if dhidden is not False:
        if dhidden is None:
            dhidden = native.empty(d, hidden, hidden)
        elif dhidden.shape != hidden.shape:
            raise ValueError(f"dhidden of shape {tuple(dhidden.shape)} for hidden states of {tuple(hidden.shape)}")
        dh = _matrix(dhidden if dhidden.dim() == 2 else dhidden.view(-1, dhidden.shape[-1]), "dhidden", d)
    if dweight is not False:
        if dweight is None:
            dweight = native.empty(d, weight, weight)
        dw = _matrix(dweight, "dweight", d)
    h._check(h._lib.linear_cross_entropy_grad(*args, go, loss.data_ptr(), dh, dw))
    return loss, dhidden if dh is not None else None, dweight if dw is not None else None


def linear_cross_entropy_grad(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, *,
                              ignore_index: int = -100, reduction: str = "mean", softcap: float = 0.0,
                              grad_out: torch.Tensor | None = None, dhidden: torch.Tensor | None | bool = None,
                              dweight: torch.Tensor | None | bool = None, handle=None):
    """(loss, dhidden, dweight): softmax cross entropy of the logits hidden
    weight^T against targets, and its gradient, in one call (libmuon
    `linear_cross_entropy_grad`). Pieces of tokens at a time: what is kept of a
    piece's logits (2 bytes each, float32 4) takes up to 1 GiB of the handle.

    hidden: (..., D), targets: (...) int64 or int32, weight: (V, D). grad_out
    (float32, on the device): one value that multiplies the gradient, or with
    reduction "none" one a token. dhidden, dweight: tensors to write to; False
    leaves that gradient out (and its product)."""
    return _loss_call(hidden, weight, targets, ignore_index, reduction, softcap, grad_out, dhidden, dweight, True,
                      handle)


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, targets, ignore_index, reduction, softcap, handle):
        need_h, need_w = ctx.needs_input_grad[:2]
        ctx.opts = (ignore_index, reduction, softcap, need_h, need_w, handle)
        if reduction == "none":
            # the gradient's weights come with backward: it takes the logits again
            ctx.save_for_backward(hidden, weight, targets)
            return _loss_call(hidden, weight, targets, ignore_index, reduction, softcap, None, None, None, False,
                              handle)[0]
        loss, dh, dw = _loss_call(hidden, weight, targets, ignore_index, reduction, softcap, None,
                                  None if need_h else False, None if need_w else False, True, handle)
        # (saved as tensors are, so that hooks on saved tensors see them; the graph
        # lets go of them before it hands on what backward returns, which is then
        # taken as it is, without a copy)
        ctx.taken = False
        ctx.save_for_backward(dh, dw)
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out):
        # (a handle that was given serves the backward too; without one, the
        # thread that runs it has its own)
        ignore_index, reduction, softcap, need_h, need_w, handle = ctx.opts
        grad_out = grad_out.contiguous()
        if reduction == "none":
            hidden, weight, targets = ctx.saved_tensors
            _, dh, dw = _loss_call(hidden, weight, targets, ignore_index, reduction, softcap, grad_out,
                                   None if need_h else False, None if need_w else False, True, handle)
        else:
            if ctx.taken:
                raise RuntimeError("linear_cross_entropy: the gradient was taken before (it is scaled in place)")
            dh, dw = ctx.saved_tensors
            ctx.taken = True
            scale([g for g in (dh, dw) if g is not None], grad_out, handle=handle)
        return dh, dw, None, None, None, None, None


def linear_cross_entropy(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, *,
                         ignore_index: int = -100, reduction: str = "mean", softcap: float = 0.0,
                         handle=None) -> torch.Tensor:
    """Softmax cross entropy of the logits hidden weight^T against targets,
    float32: one value ("mean" over the tokens whose target is not
    ignore_index, "sum") or one a token ("none", 0 where ignored). The loss
    alone stores no logits; a call that computes the gradient keeps a piece's, as
    `linear_cross_entropy_grad` says.

    Differentiable in hidden and weight, in reverse mode (a tensor with a
    forward-mode tangent is refused). "mean" and "sum" compute the gradient with
    the loss, so one backward per forward; backward multiplies it by grad_out in
    place, which rounds a bfloat16 gradient once more unless that is a power of
    two (`linear_cross_entropy_grad` takes grad_out before its one rounding).
    "none" computes the gradient in backward, logits and all. A handle that is
    given serves both; without one each uses its own thread's."""
    if torch.is_grad_enabled() and (hidden.requires_grad or weight.requires_grad):
        return _LinearCrossEntropy.apply(hidden, weight, targets, ignore_index, reduction, softcap, handle)
    return _loss_call(hidden, weight, targets, ignore_index, reduction, softcap, None, None, None, False, handle)[0]


# ---------------------------------------------------------------------------
# host-only validation (no device needed); descriptors may be MuonMatrix objects
# ---------------------------------------------------------------------------
def _descriptors(xs):
    if xs is None:
        return None
    arr = (MuonMatrix * max(1, len(xs)))()
    for i, x in enumerate(xs):
        arr[i] = x
    return arr


def _checked(call, *args):
    buf = ctypes.create_string_buffer(256)
    rc = call(*args, buf, 256)
    return rc, buf.value.decode()


def check_norm_args(grads, out=None, max_norm: float = 1.0, norm=4096, coef=None) -> tuple[int, str]:
    """Rules of grad_norm (out None: the list is only read) or of clip_grad_norm into `out`; in place, where the list
    is written, `out` is the list itself."""
    return _checked(load_library().muon_check_norm_args, len(grads), _descriptors(grads), _descriptors(out), max_norm,
                    norm, coef)


def check_adamw_args(grads, exp_avgs, exp_avg_sqs, weights, copies=None, cfg: AdamWConfig | None = None,
                     grad_scale=None) -> tuple[int, str]:
    lib = load_library()
    if cfg is None:
        cfg = AdamWConfig()
        lib.muon_adamw_config_default(ctypes.byref(cfg))
    return _checked(lib.muon_check_adamw_args, len(weights), _descriptors(grads), _descriptors(exp_avgs),
                    _descriptors(exp_avg_sqs), _descriptors(weights), _descriptors(copies), ctypes.byref(cfg),
                    grad_scale)


def check_loss_args(hidden, weight, targets=4096, target_bytes=8, cfg: LossConfig | None = None, grad_out=None,
                    loss=1 << 20, dhidden=None, dweight=None) -> tuple[int, str]:
    ref = lambda m: ctypes.byref(m) if m is not None else None
    return _checked(load_library().muon_check_loss_args, ref(hidden), ref(weight), targets, target_bytes, ref(cfg),
                    grad_out, loss, ref(dhidden), ref(dweight))
