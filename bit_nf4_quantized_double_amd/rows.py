"""Row-wise operators of a decoder block over libqlora.so: RMS norm with the
residual's addition, SwiGLU, and rows quantized to 8 bits.

The 16-bit forms have backward passes (and autograd wrappers); the 8-bit ones
(``*_int8``) write the operand of the int8 product (:mod:`.int8`).  Formulas,
rounding and limits: include/qlora.h.  As in :mod:`.qlora`, PyTorch supplies
memory and the stream; there is no CPU path.

Inputs are bf16 or fp16 matrices whose last dimension is contiguous; their
rows may be further apart (a slice of a wider matrix).
"""

from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass

import torch

from . import qlora

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # QLORA_BF16 / F16 / F32
MAX_NORM_WIDTH = 32768


# The current device and its current stream as plain numbers: the same as
# torch.cuda.current_device() and current_stream().cuda_stream, without the
# Stream object whose making costs as much as a small call's whole checks.
_device_index = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream(device) -> int:
    """The current stream of the device the tensors are on, which has to be
    the current device: the library launches there."""
    index = _device_index()
    if device.index != index:
        raise ValueError(f"the tensors are on {device}, the current device is cuda:{index}")
    return _raw_stream(index)


# Small calls are bound by the host: each check below passes on its first
# line for the usual argument, and only says what is wrong when that fails.

def _first(t, name: str, types=(torch.bfloat16, torch.float16)):
    """(dtype, shape, device) that a call's other matrices have to match."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dtype, shape = t.dtype, t.shape
    if dtype not in types:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in types)}, got {dtype}")
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D, got {len(shape)} dimensions")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (there is no CPU path)")
    return dtype, shape, t.device


def _mat(t, dtype, shape, name: str, device):
    """(pointer, row stride) of a matrix with contiguous rows."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr(), shape[1]
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (there is no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    m, k = shape
    if k > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    ld = t.stride(0) if m > 1 else k
    if ld < k:
        raise ValueError(f"{name}: rows must not overlap (stride {ld} for {k} columns)")
    return t.data_ptr(), ld


def _vec(t, types, n: int, name: str, device) -> int:
    """Pointer of a contiguous vector of n elements."""
    if isinstance(t, torch.Tensor) and t.dtype in types and t.shape == (n,) and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in types:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in types)}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    raise ValueError(f"{name} must be a contiguous vector of {n} elements, got {tuple(t.shape)}")


def _out(t, shape, dtype, name: str, device, like=None):
    """A caller's output buffer (checked), or a new one (`like`: a tensor of
    that shape, type and device, to make it from sooner)."""
    if t is None:
        if like is not None and like.is_contiguous():
            return torch.empty_like(like)
        return torch.empty(*shape, dtype=dtype, device=device)  # sooner than with a tuple
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


@dataclass(slots=True)
class Int8Rows:
    """Rows in 8 bits, a scale each, in the layout the int8 product reads."""
    codes: torch.Tensor  # uint8 [qlora_int8_rows_bytes(m, k)], opaque
    scale: torch.Tensor  # float32 [m]
    m: int
    k: int
    dtype: torch.dtype   # of the values they were made from (fp32 ones count as bf16)

    def nbytes(self) -> int:
        return self.codes.numel() + 4 * self.scale.numel()


def _new_rows(m: int, k: int, dtype, device) -> Int8Rows:
    # the rows' bytes (checked against the library's own count in the tests)
    nbytes = (m + 15) // 16 * 16 * ((k + 127) // 128 * 128)
    return Int8Rows(torch.empty(nbytes, dtype=torch.uint8, device=device),
                    torch.empty(m, dtype=torch.float32, device=device), m, k, dtype)


def check_rows(q, device=None) -> Int8Rows:
    if not isinstance(q, Int8Rows):
        raise TypeError("expected Int8Rows")
    codes, scale, m = q.codes, q.scale, q.m
    if device is None:
        device = codes.device
    nbytes = (m + 15) // 16 * 16 * ((q.k + 127) // 128 * 128)
    if not (codes.dtype is torch.uint8 and codes.shape == (nbytes,) and codes.device == device and codes.is_contiguous()):
        _vec(codes, (torch.uint8,), nbytes, "codes", device)
    if not (scale.dtype is torch.float32 and scale.shape == (m,) and scale.device == device and scale.is_contiguous()):
        _vec(scale, (torch.float32,), m, "scale", device)
    if not codes.is_cuda:
        raise ValueError("codes must be GPU tensors (there is no CPU path)")
    return q


def quantize_rows(X: torch.Tensor, col_scale: torch.Tensor | None = None) -> Int8Rows:
    """bf16, fp16 or fp32 [M, K] -> Int8Rows; col_scale (fp32 [K]) multiplies
    the columns first."""
    dt, (m, k), dev = _first(X, "X", tuple(DTYPES))
    p, ld = _mat(X, dt, X.shape, "X", dev)
    c = None if col_scale is None else _vec(col_scale, (torch.float32,), k, "col_scale", dev)
    q = _new_rows(m, k, torch.bfloat16 if dt == torch.float32 else dt, dev)
    st = qlora.lib().qlora_int8_quantize_rows(p, DTYPES[dt], ld, m, k, c, q.codes.data_ptr(), q.scale.data_ptr(),
                                              _stream(dev))
    if st:
        qlora._check(st, "qlora_int8_quantize_rows")
    return q


def dequant_rows(q: Int8Rows, out: torch.Tensor | None = None, dtype=None) -> torch.Tensor:
    """The values of Int8Rows as a 16-bit [M, K] tensor (``dtype``, or the
    type they were made from)."""
    check_rows(q)
    dev = q.codes.device
    dtype = dtype or (q.dtype if out is None else out.dtype)
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError("dequant_rows produces bf16 or fp16")
    out = _out(out, (q.m, q.k), dtype, "out", dev)
    st = qlora.lib().qlora_int8_dequant_rows(q.codes.data_ptr(), q.scale.data_ptr(), q.m, q.k, out.data_ptr(),
                                             DTYPES[dtype], _stream(dev))
    if st:
        qlora._check(st, "qlora_int8_dequant_rows")
    return out


def _norm_args(X, gamma, residual, H):
    dt, shape, dev = _first(X, "X")
    m, k = shape
    p, ld = _mat(X, dt, shape, "X", dev)
    g = _vec(gamma, (dt, torch.float32), k, "gamma", dev)
    if residual is None:
        if H is not None:
            raise ValueError("H is written only with a residual (without one it is X)")
        return dt, m, k, dev, (p, ld, None, 0, g, DTYPES[gamma.dtype], m, k), X
    r, ldr = _mat(residual, dt, shape, "residual", dev)
    return dt, m, k, dev, (p, ld, r, ldr, g, DTYPES[gamma.dtype], m, k), _out(H, shape, dt, "H", dev, X)


def rms_norm_fwd(X: torch.Tensor, gamma: torch.Tensor, eps: float, residual: torch.Tensor | None = None, *,
                 H: torch.Tensor | None = None, Y: torch.Tensor | None = None):
    """h = X + residual, Y = h gamma / sqrt(mean h^2 + eps).  Returns
    (Y, h, rstd); without a residual h is X itself.  ``H`` may be X or the
    residual (updated in place)."""
    dt, m, k, dev, args, h = _norm_args(X, gamma, residual, H)
    Y = _out(Y, (m, k), dt, "Y", dev, X)
    rstd = torch.empty(m, dtype=torch.float32, device=dev)
    st = qlora.lib().qlora_rms_norm_fwd(*args, eps, None if residual is None else h.data_ptr(), Y.data_ptr(),
                                        rstd.data_ptr(), DTYPES[dt], _stream(dev))
    if st:
        qlora._check(st, "qlora_rms_norm_fwd")
    return Y, h, rstd


def rms_norm_int8(X: torch.Tensor, gamma: torch.Tensor, eps: float, residual: torch.Tensor | None = None, *,
                  H: torch.Tensor | None = None):
    """The norm of :func:`rms_norm_fwd` in 8 bits.  Returns (Int8Rows, h)."""
    dt, m, k, dev, args, h = _norm_args(X, gamma, residual, H)
    q = _new_rows(m, k, dt, dev)
    st = qlora.lib().qlora_rms_norm_int8(*args, eps, None if residual is None else h.data_ptr(), q.codes.data_ptr(),
                                         q.scale.data_ptr(), DTYPES[dt], _stream(dev))
    if st:
        qlora._check(st, "qlora_rms_norm_int8")
    return q, h


def rms_norm_bwd(dY: torch.Tensor, H: torch.Tensor, rstd: torch.Tensor, gamma: torch.Tensor,
                 dH: torch.Tensor | None = None, *, dX: torch.Tensor | None = None,
                 dgamma: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """Returns (dX, dgamma fp32 [K]); dX is the residual's gradient too.
    ``dH``: the gradient that reaches h by itself, added to dX."""
    dt, shape, dev = _first(dY, "dY")
    m, k = shape
    dy, lddy = _mat(dY, dt, shape, "dY", dev)
    h, ldh = _mat(H, dt, shape, "H", dev)
    dh, lddh = (None, 0) if dH is None else _mat(dH, dt, shape, "dH", dev)
    g = _vec(gamma, (dt, torch.float32), k, "gamma", dev)
    rs = _vec(rstd, (torch.float32,), m, "rstd", dev)
    dX = _out(dX, shape, dt, "dX", dev, dY)
    dgamma = _out(dgamma, (k,), torch.float32, "dgamma", dev)
    L = qlora.lib()
    wst, wsn = qlora._ws(L.qlora_rms_norm_bwd_workspace_bytes(m, k), dev, ws)
    st = L.qlora_rms_norm_bwd(dy, lddy, h, ldh, rs, g, DTYPES[gamma.dtype], dh, lddh, m, k, dX.data_ptr(),
                              dgamma.data_ptr(), DTYPES[dt], None if wst is None else wst.data_ptr(), wsn,
                              _stream(dev))
    if st:
        qlora._check(st, "qlora_rms_norm_bwd")
    return dX, dgamma


def _swiglu_args(G, U):
    dt, shape, dev = _first(G, "gate")
    g, ldg = _mat(G, dt, shape, "gate", dev)
    u, ldu = _mat(U, dt, shape, "up", dev)
    return dt, shape, dev, (g, ldg, u, ldu, *shape)


def swiglu_fwd(G: torch.Tensor, U: torch.Tensor, *, Y: torch.Tensor | None = None) -> torch.Tensor:
    """silu(G) * U in 16 bits."""
    dt, shape, dev, args = _swiglu_args(G, U)
    Y = _out(Y, shape, dt, "Y", dev, G)
    st = qlora.lib().qlora_swiglu_fwd(*args, Y.data_ptr(), DTYPES[dt], _stream(dev))
    if st:
        qlora._check(st, "qlora_swiglu_fwd")
    return Y


def swiglu_int8(G: torch.Tensor, U: torch.Tensor) -> Int8Rows:
    """silu(G) * U in 8 bits."""
    dt, shape, dev, args = _swiglu_args(G, U)
    q = _new_rows(*shape, dt, dev)
    st = qlora.lib().qlora_swiglu_int8(*args, q.codes.data_ptr(), q.scale.data_ptr(), DTYPES[dt], _stream(dev))
    if st:
        qlora._check(st, "qlora_swiglu_int8")
    return q


def swiglu_bwd(dY: torch.Tensor, G: torch.Tensor, U: torch.Tensor, *, dG: torch.Tensor | None = None,
               dU: torch.Tensor | None = None):
    """Returns (dG, dU)."""
    dt, shape, dev, args = _swiglu_args(G, U)
    dy, lddy = _mat(dY, dt, shape, "dY", dev)
    dG, dU = _out(dG, shape, dt, "dG", dev, G), _out(dU, shape, dt, "dU", dev, G)
    st = qlora.lib().qlora_swiglu_bwd(dy, lddy, *args, dG.data_ptr(), dU.data_ptr(), DTYPES[dt], _stream(dev))
    if st:
        qlora._check(st, "qlora_swiglu_bwd")
    return dG, dU


def _rows_of(t: torch.Tensor, width: int) -> torch.Tensor:
    """[..., width] as a matrix with contiguous rows."""
    t = t.reshape(math.prod(t.shape[:-1]), width)  # not -1, which rows of no values leave open
    return t if (width <= 1 or t.stride(1) == 1) and (t.shape[0] <= 1 or t.stride(0) >= width) else t.contiguous()


def _new(shape, like: torch.Tensor) -> torch.Tensor:
    return torch.empty(shape, dtype=like.dtype, device=like.device)


def _same_shape(t, shape, name: str) -> None:
    """Before anything is reshaped to a matrix: afterwards a tensor of another
    shape may have as many rows, and would be paired up wrongly."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


class RMSNormFunction(torch.autograd.Function):
    """(X, residual or None, gamma) -> (Y, h)."""

    @staticmethod
    def forward(ctx, X, residual, gamma, eps: float):
        if residual is not None:
            _same_shape(residual, X.shape, "residual")
        k = X.shape[-1]
        X2 = _rows_of(X, k)
        R2 = None if residual is None else _rows_of(residual, k)
        # outputs are made in their own shape: views of others could not be modified in place
        Y = _new(X.shape, X)
        h = None if residual is None else _new(X.shape, X)
        _, H, rstd = rms_norm_fwd(X2, gamma, eps, R2, H=None if h is None else _rows_of(h, k), Y=_rows_of(Y, k))
        ctx.save_for_backward(H if h is None else h, rstd, gamma)
        ctx.has_residual = residual is not None
        # an output that nothing reads has no gradient: it comes as None, not as a tensor of zeros
        ctx.set_materialize_grads(False)
        return Y, h  # without a residual h is X, which is not returned as an output

    @staticmethod
    @qlora._once
    def backward(ctx, dY, dh):
        h, rstd, gamma = ctx.saved_tensors
        k = h.shape[-1]
        if dY is None:  # h alone is read: its gradient passes through
            return dh, (dh if ctx.has_residual else None), (torch.zeros_like(gamma) if ctx.needs_input_grad[2] else None), None
        dX, dgamma = rms_norm_bwd(_rows_of(dY, k), _rows_of(h, k), rstd, gamma, None if dh is None else _rows_of(dh, k))
        dX = dX.reshape(dY.shape)
        return dX, (dX if ctx.has_residual else None), (dgamma.to(gamma.dtype) if ctx.needs_input_grad[2] else None), None


class RMSNorm(torch.nn.Module):
    """RMS norm; ``forward(x, residual)`` also returns the new residual
    stream, as (y, h)."""

    def __init__(self, width: int, eps: float = 1e-5, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.eps = float(eps)
        self.weight = torch.nn.Parameter(torch.ones(width, dtype=dtype, device=device))

    def forward(self, x, residual=None):
        y, h = RMSNormFunction.apply(x, residual, self.weight, self.eps)
        return y if residual is None else (y, h)


class SwiGLUFunction(torch.autograd.Function):
    """silu(G) * U."""

    @staticmethod
    def forward(ctx, G, U):
        _same_shape(U, G.shape, "up")
        k = G.shape[-1]
        G2, U2 = _rows_of(G, k), _rows_of(U, k)
        ctx.save_for_backward(G2, U2)
        Y = _new(G.shape, G)
        swiglu_fwd(G2, U2, Y=_rows_of(Y, k))
        return Y

    @staticmethod
    @qlora._once
    def backward(ctx, dY):
        G, U = ctx.saved_tensors
        dG, dU = swiglu_bwd(_rows_of(dY, G.shape[-1]), G, U)
        return dG.reshape(dY.shape), dU.reshape(dY.shape)


def swiglu(G: torch.Tensor, U: torch.Tensor) -> torch.Tensor:
    """Differentiable silu(G) * U."""
    return SwiGLUFunction.apply(G, U)


def _bind(L: ctypes.CDLL) -> None:
    i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    norm = [vp, i64, vp, i64, vp, i32, i64, i64, ctypes.c_float]
    sig = {
        "qlora_int8_rows_bytes": (sz, [i64, i64]),
        "qlora_int8_quantize_rows": (i32, [vp, i32, i64, i64, i64, vp, vp, vp, vp]),
        "qlora_int8_dequant_rows": (i32, [vp, vp, i64, i64, vp, i32, vp]),
        "qlora_rms_norm_bwd_workspace_bytes": (sz, [i64, i64]),
        "qlora_rms_norm_fwd": (i32, norm + [vp, vp, vp, i32, vp]),
        "qlora_rms_norm_int8": (i32, norm + [vp, vp, vp, i32, vp]),
        "qlora_rms_norm_bwd": (i32, [vp, i64, vp, i64, vp, vp, i32, vp, i64, i64, i64, vp, vp, i32, vp, sz, vp]),
        "qlora_swiglu_fwd": (i32, [vp, i64, vp, i64, i64, i64, vp, i32, vp]),
        "qlora_swiglu_int8": (i32, [vp, i64, vp, i64, i64, i64, vp, vp, i32, vp]),
        "qlora_swiglu_bwd": (i32, [vp, i64, vp, i64, vp, i64, i64, i64, vp, vp, i32, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
