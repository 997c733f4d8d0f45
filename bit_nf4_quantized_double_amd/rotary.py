"""Rotary positions of queries and keys over libqlora.so.

:func:`rotate` turns both in one launch (in place, if asked to), and
:func:`rotate_bwd` gradients back; :func:`rotary` is the differentiable form.
:func:`frequencies` makes the angles, also for contexts longer than the trained
one.  Formulas, rounding and limits: include/qlora.h.

Queries and keys are bf16 or fp16 [tokens, heads, head_dim] whose last dimension
is contiguous; tokens and heads may be apart in any way (slices of a projection's
output, a cache).  Positions are int32 or int64 [tokens]; however large, the
angle is exact.
"""

from __future__ import annotations

import ctypes
import math
from fractions import Fraction

import torch

from . import qlora
from .rows import DTYPES, _stream

# 2^320 / (2 pi), to 256 bits and more
_PER_RADIAN = round(Fraction(2**320) / (2 * Fraction(
    "3.1415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679821480865")))


def _turns(f: float) -> int:
    """f radians as a signed 64-bit fraction of a turn, to the nearest."""
    m, e = math.frexp(f)
    up = 320 - 64 + 53 - e  # f = m 2^e, m a multiple of 2^-53
    n = int(m * 2.0**53) * _PER_RADIAN
    t = (n + (1 << (up - 1))) >> up if up > 0 else n << -up
    t &= 2**64 - 1
    return t - 2**64 if t >= 2**63 else t



class Frequencies:
    """Angles in radians a position, one for each pair, and the factor that turned
    pairs are multiplied by.  Kept as 64-bit fractions of a turn, in which
    position times frequency is exact modulo a turn."""

    def __init__(self, f, factor: float = 1.0, device="cuda"):
        f = torch.as_tensor(f, dtype=torch.float64, device="cpu")
        if f.dim() != 1 or not bool(torch.isfinite(f).all()):
            raise ValueError("f must be a vector of finite frequencies")
        if not math.isfinite(factor):
            raise ValueError("factor must be finite")
        self.turns = torch.tensor([_turns(x) for x in f.tolist()], dtype=torch.int64, device=device)
        self.rot, self.factor = 2 * f.shape[0], float(factor)


def frequencies(rot: int, base: float = 10000.0, *, scaling: str | None = None, by: float = 1.0, trained: int = 4096,
                low: float = 1.0, high: float = 32.0, device="cuda") -> Frequencies:
    """f_i = base^(-2 i / rot), for contexts ``by`` times the ``trained`` one by

    None       no change
    "linear"   positions divided: f / by
    "base"     a larger base: base by^(rot / (rot - 2)), which keeps the fastest
               pair and divides the slowest by ``by``
    "blended"  f / by for pairs that make fewer than ``low`` turns over the trained
               context, f for those that make more than ``high``, linear in the turns
               between; turned pairs are lengthened by 0.1 ln by + 1
    """
    if rot < 0 or rot % 2:
        raise ValueError("rot must be even")
    if not (by >= 1.0 and math.isfinite(by)) or not base > 0:
        raise ValueError("by must be at least 1, base positive")
    if scaling not in (None, "linear", "base", "blended"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling == "base" and rot > 2:
        base = base * by ** (rot / (rot - 2))
    f = base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / max(rot, 1))
    if scaling == "linear":
        f = f / by
    if scaling != "blended":
        return Frequencies(f, 1.0, device)
    if not (0 <= low < high):
        raise ValueError("low must be below high")
    keep = ((trained * f / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
    return Frequencies(f / by * (1 - keep) + f * keep, 0.1 * math.log(by) + 1.0, device)


class CHeads(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


def check_heads(t, name: str, dtype=None, shape=None, device=None) -> CHeads:
    """A [tokens, heads, head_dim] tensor of a type, shape and device as the library takes it."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is None:
        if t.dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"{name} must be bf16 or fp16, got {t.dtype}")
    elif t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {t.dim()} dimensions")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (there is no CPU path)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    n, h, d = t.shape
    if d > 1 and t.stride(2) != 1 and t.numel():
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return CHeads(t.data_ptr(), t.stride(0) if n > 1 else 0, t.stride(1) if h > 1 else 0)


def check_vector(t, types, n: int, name: str, device) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in types:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in types)}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} elements, got {tuple(t.shape)}")
    return t.data_ptr()


def _turn(Q, K, positions, freqs: Frequencies, interleaved: bool, inverse: bool, Q_out, K_out):
    q = check_heads(Q, "Q")
    dev, dt = Q.device, Q.dtype
    n, h, d = Q.shape
    hk = 0
    k = CHeads()
    if K is not None:
        if not isinstance(K, torch.Tensor) or K.dim() != 3:
            raise ValueError("K must be a [tokens, heads, head_dim] tensor")
        hk = K.shape[1]
        k = check_heads(K, "K", dt, (n, hk, d), dev)
    elif K_out is not None:
        raise ValueError("K_out without K")
    if not isinstance(freqs, Frequencies):
        raise TypeError("freqs must be Frequencies")
    if freqs.rot > d:
        raise ValueError(f"{freqs.rot} values to turn in heads of {d}")
    p = check_vector(positions, (torch.int32, torch.int64), n, "positions", dev)
    f = check_vector(freqs.turns, (torch.int64,), freqs.rot // 2, "freqs.turns", dev)
    Q_out = torch.empty(n, h, d, dtype=dt, device=dev) if Q_out is None else Q_out
    qo = check_heads(Q_out, "Q_out", dt, Q.shape, dev)
    ko = CHeads()
    if K is not None:
        K_out = torch.empty(n, hk, d, dtype=dt, device=dev) if K_out is None else K_out
        ko = check_heads(K_out, "K_out", dt, K.shape, dev)
    r = ctypes.byref
    st = qlora.lib().qlora_rope(r(q), h, r(k), hk, n, d, freqs.rot, interleaved, p, positions.dtype == torch.int64, f,
                                freqs.factor, inverse, r(qo), r(ko), DTYPES[dt], _stream(dev))
    if st:
        qlora._check(st, "qlora_rope")
    return Q_out, K_out


def rotate(Q: torch.Tensor, K: torch.Tensor | None, positions: torch.Tensor, freqs: Frequencies, *,
           interleaved: bool = False, Q_out: torch.Tensor | None = None, K_out: torch.Tensor | None = None):
    """Returns (Q, K) turned to their positions.  ``Q_out`` and ``K_out`` may be Q
    and K (in place), not each other or K and Q.  K may be None."""
    return _turn(Q, K, positions, freqs, bool(interleaved), False, Q_out, K_out)


def rotate_bwd(dQ: torch.Tensor, dK: torch.Tensor | None, positions: torch.Tensor, freqs: Frequencies, *,
               interleaved: bool = False, Q_out: torch.Tensor | None = None, K_out: torch.Tensor | None = None):
    """The gradients of :func:`rotate`'s inputs from those of its outputs."""
    return _turn(dQ, dK, positions, freqs, bool(interleaved), True, Q_out, K_out)


def _last_contiguous(t: torch.Tensor) -> torch.Tensor:
    return t if t.shape[-1] <= 1 or t.stride(-1) == 1 else t.contiguous()


class RotaryFunction(torch.autograd.Function):
    """(Q, K or None) -> both turned."""

    @staticmethod
    def forward(ctx, Q, K, positions, freqs: Frequencies, interleaved: bool):
        ctx.save_for_backward(positions)
        ctx.freqs, ctx.interleaved = freqs, interleaved
        ctx.set_materialize_grads(False)
        return rotate(_last_contiguous(Q), None if K is None else _last_contiguous(K), positions, freqs,
                      interleaved=interleaved)

    @staticmethod
    @qlora._once
    def backward(ctx, dQ, dK):
        positions, = ctx.saved_tensors
        both = [None if g is None else _last_contiguous(g) for g in (dQ, dK)]
        if both[0] is None and both[1] is not None:  # the queries' output is not used
            return None, rotate_bwd(both[1], None, positions, ctx.freqs, interleaved=ctx.interleaved)[0], None, None, None
        if both[0] is None:
            return None, None, None, None, None
        dq, dk = rotate_bwd(both[0], both[1], positions, ctx.freqs, interleaved=ctx.interleaved)
        return dq, dk, None, None, None


def rotary(Q: torch.Tensor, K: torch.Tensor | None, positions: torch.Tensor, freqs: Frequencies,
           interleaved: bool = False):
    """Differentiable :func:`rotate`."""
    return RotaryFunction.apply(Q, K, positions, freqs, bool(interleaved))


def _bind(L: ctypes.CDLL) -> None:
    i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    H = ctypes.POINTER(CHeads)
    L.qlora_rope.restype = i32
    L.qlora_rope.argtypes = [H, i64, H, i64, i64, i64, i64, i32, vp, i32, vp, ctypes.c_float, i32, H, H, i32, vp]
