"""Softmax cross entropy of hidden states under a frozen output head, over
libqlora.so: loss and gradient in one pass over the vocabulary, without the
logits.

:func:`linear_cross_entropy_fwd` gives each token's loss (evaluation),
:func:`linear_cross_entropy_grad` the gradient of the hidden states as well
(:func:`linear_cross_entropy_units` for one that is multiplied later), and
:func:`linear_cross_entropy` is the differentiable form.  The head is frozen, as
every weight here: there is no dW.  Formulas, rounding and limits:
include/qlora.h.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import qlora, rows
from .rotary import check_vector
from .rows import DTYPES, _first, _out, _stream

_F32 = (torch.float32,)


def _matrix(t, name: str, k: int | None = None):
    """(pointer, row stride, rows, columns) of a 16-bit matrix with contiguous rows."""
    _, (m, n), _ = _first(t, name)
    if k is not None and n != k:
        raise ValueError(f"{name} has {n} columns, not {k}")
    if n > 1 and t.stride(1) != 1 and m:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    ld = t.stride(0) if m > 1 else n
    if ld < n:
        raise ValueError(f"{name}: rows must not overlap (stride {ld} for {n} columns)")
    return t.data_ptr(), ld, m, n


def workspace_bytes(m: int, k: int, v: int, gradient: bool) -> int:
    return int(qlora.lib().qlora_cross_entropy_workspace_bytes(m, k, v, gradient))


def _call(X, W, targets, ignore_index, dloss, gradient, dX, ws, units=False):
    x, ldx, m, k = _matrix(X, "X")
    dt, dev = X.dtype, X.device
    w, ldw, v, _ = _matrix(W, "W", k)
    if W.dtype != dt:
        raise TypeError(f"W must be {dt}, got {W.dtype}")
    if W.device != dev:
        raise ValueError(f"W must be on {dev}")
    t = check_vector(targets, (torch.int64,), m, "targets", dev)
    g = None if dloss is None else check_vector(dloss, _F32, m, "dloss", dev)
    if not isinstance(ignore_index, int):
        raise TypeError("ignore_index must be a whole number")
    loss, lse = (torch.empty(m, dtype=torch.float32, device=dev) for _ in range(2))
    if gradient:
        dX = _out(dX, X.shape, dt, "dX", dev)
    L = qlora.lib()
    wst, wsn = qlora._ws(L.qlora_cross_entropy_workspace_bytes(m, k, v, gradient), dev, ws)
    rest = DTYPES[dt], None if wst is None else wst.data_ptr(), wsn, _stream(dev)
    if units:
        unit = torch.empty(m, dtype=torch.float32, device=dev)
        st = L.qlora_cross_entropy_units(x, ldx, w, ldw, t, m, k, v, ignore_index, loss.data_ptr(), lse.data_ptr(),
                                         dX.data_ptr(), unit.data_ptr(), *rest)
        if st:
            qlora._check(st, "qlora_cross_entropy_units")
        return loss, lse, dX, unit
    st = L.qlora_cross_entropy(x, ldx, w, ldw, t, m, k, v, ignore_index, g, loss.data_ptr(), lse.data_ptr(),
                               dX.data_ptr() if gradient else None, *rest)
    if st:
        qlora._check(st, "qlora_cross_entropy")
    return loss, lse, dX


def linear_cross_entropy_fwd(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, *, ignore_index: int = -100,
                             ws: torch.Tensor | None = None):
    """X [tokens, width], W [vocabulary, width] (bf16 or fp16), targets int64
    [tokens].  Returns (loss, lse), fp32 [tokens]: the losses are 0 where the
    target is ignore_index."""
    loss, lse, _ = _call(X, W, targets, ignore_index, None, False, None, ws)
    return loss, lse


def linear_cross_entropy_grad(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, dloss: torch.Tensor | None = None, *,
                              ignore_index: int = -100, dX: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """Returns (loss, lse, dX) with dX the gradient of sum(dloss loss); dloss
    (fp32 [tokens]) None: ones.  ``dX`` may be X (overwritten)."""
    return _call(X, W, targets, ignore_index, dloss, True, dX, ws)


def linear_cross_entropy_units(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, *, ignore_index: int = -100,
                               dX: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """Returns (loss, lse, dX, unit): dX as for losses that count once, its rows
    times unit (fp32 [tokens], powers of two) so that small ones keep their digits
    until ``scale_rows(dX, g / unit)``."""
    return _call(X, W, targets, ignore_index, None, True, dX, ws, True)


def scale_rows(X: torch.Tensor, g: torch.Tensor, Y: torch.Tensor | None = None) -> torch.Tensor:
    """g[:, None] * X for a contiguous 16-bit matrix and fp32 g, rounded once."""
    dt, (m, k), dev = _first(X, "X")
    if not X.is_contiguous():
        raise ValueError("X must be contiguous")
    Y = _out(Y, X.shape, dt, "Y", dev)
    st = qlora.lib().qlora_scale_rows(X.data_ptr(), check_vector(g, _F32, m, "g", dev), m, k, Y.data_ptr(), DTYPES[dt],
                                      _stream(dev))
    if st:
        qlora._check(st, "qlora_scale_rows")
    return Y


def reduce_losses(loss: torch.Tensor, targets: torch.Tensor, mean: bool, *, ignore_index: int = -100) -> torch.Tensor:
    """fp32 [2]: the sum or mean of the losses whose target is not ignore_index, and
    what one of them counts in it.  In one launch, for captured graphs too."""
    if not isinstance(loss, torch.Tensor) or loss.dim() != 1 or not loss.is_cuda:
        raise ValueError("loss must be a vector on the GPU")
    m, dev = loss.shape[0], loss.device
    p, t = check_vector(loss, _F32, m, "loss", dev), check_vector(targets, (torch.int64,), m, "targets", dev)
    out = torch.empty(2, dtype=torch.float32, device=dev)
    st = qlora.lib().qlora_loss_sum(p, t, m, ignore_index, bool(mean), out.data_ptr(), _stream(dev))
    if st:
        qlora._check(st, "qlora_loss_sum")
    return out


class LinearCrossEntropyFunction(torch.autograd.Function):
    """(X [tokens, width], W, targets) -> losses, or their sum or mean.  The gradient
    is made in the forward, for losses that count once, and the backward multiplies
    its rows.  In fp16 it is kept in units of each row: a loss scale that comes
    only from above would find small gradients rounded to nothing."""

    @staticmethod
    def forward(ctx, X, W, targets, ignore_index: int, reduction: str, gradient: bool):
        unit = None
        if gradient and X.dtype == torch.float16:
            loss, _, dX, unit = linear_cross_entropy_units(X, W, targets, ignore_index=ignore_index)
        elif gradient:
            loss, _, dX = linear_cross_entropy_grad(X, W, targets, ignore_index=ignore_index)
        else:
            loss, _ = linear_cross_entropy_fwd(X, W, targets, ignore_index=ignore_index)
        both = None if reduction == "none" else reduce_losses(loss, targets, reduction == "mean", ignore_index=ignore_index)
        if gradient:
            ctx.save_for_backward(dX, unit, targets, None if both is None else both[1])
            ctx.ignore_index = ignore_index
        return loss if both is None else both[0]

    @staticmethod
    @qlora._once
    def backward(ctx, dloss):
        dX, unit, targets, weight = ctx.saved_tensors
        if weight is not None:
            dloss = (dloss * weight).expand(dX.shape[0])
        # ignored tokens get none whatever comes: an infinite loss scale, or the mean of no losses
        g = dloss.masked_fill(targets == ctx.ignore_index, 0.0)
        if unit is not None:
            g = g / unit
        return scale_rows(dX, g.contiguous()), None, None, None, None, None


def linear_cross_entropy(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, *, ignore_index: int = -100,
                         reduction: str = "mean") -> torch.Tensor:
    """Differentiable loss of hidden states X [..., width] with targets [...]:
    ``reduction`` "none", "sum" or "mean" (over the targets that are not
    ignore_index).  A gradient for X only."""
    if reduction not in ("none", "sum", "mean"):
        raise ValueError(f"unknown reduction {reduction!r}")
    for t, name in ((X, "X"), (W, "W"), (targets, "targets")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    if W.requires_grad and torch.is_grad_enabled():
        raise ValueError("W is frozen: it has no gradient (detach it, or set requires_grad to False)")
    if X.dim() < 1 or targets.shape != X.shape[:-1]:
        raise ValueError(f"targets must have shape {tuple(X.shape[:-1])}, got {tuple(targets.shape)}")
    n = math.prod(targets.shape)
    flat = targets.reshape(n).contiguous()
    gradient = X.requires_grad and torch.is_grad_enabled()
    loss = LinearCrossEntropyFunction.apply(rows._rows_of(X, X.shape[-1]), W, flat, ignore_index, reduction, gradient)
    return loss.reshape(targets.shape) if reduction == "none" else loss


def _bind(L: ctypes.CDLL) -> None:
    i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    sig = {
        "qlora_cross_entropy_workspace_bytes": (sz, [i64, i64, i64, i32]),
        "qlora_cross_entropy": (i32, [vp, i64, vp, i64, vp, i64, i64, i64, i64, vp, vp, vp, vp, i32, vp, sz, vp]),
        "qlora_cross_entropy_units": (i32, [vp, i64, vp, i64, vp, i64, i64, i64, i64, vp, vp, vp, vp, i32, vp, sz, vp]),
        "qlora_loss_sum": (i32, [vp, vp, i64, i64, i32, vp, vp]),
        "qlora_scale_rows": (i32, [vp, vp, i64, i64, vp, i32, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
