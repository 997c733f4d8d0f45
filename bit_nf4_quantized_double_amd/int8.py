"""Matrix product in 8-bit integers over libqlora.so: a frozen weight in int8
with a scale for each output channel, activations quantized with a scale for
each token.

The form to serve a merged model in where 4 bits are too few or the product is
bound by arithmetic: ``quantize_weight(qlora.merge(...))`` gives the weight,
:func:`linear_fwd` the product, and the norm and SwiGLU of :mod:`.rows` write
its operand directly.  :func:`linear_bwd` passes gradients through the frozen
layer.  Formulas, rounding and limits: include/qlora.h.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import qlora, rows
from .rows import DTYPES, Int8Rows, _first, _mat, _out, _stream, _vec


class _CInt8Weight(ctypes.Structure):
    _fields_ = [("n_out", ctypes.c_int64), ("k_in", ctypes.c_int64), ("codes", ctypes.c_void_p),
                ("codes_t", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


@dataclass
class Int8Weight:
    """A frozen weight in int8, a scale for each output channel."""
    codes: torch.Tensor           # uint8 [qlora_int8_weight_bytes(n_out, k_in)], opaque
    scale: torch.Tensor           # float32 [n_out]
    n_out: int
    k_in: int
    codes_t: torch.Tensor | None = None  # the transpose's codes, for the backward

    def _c(self) -> _CInt8Weight:
        dev = self.codes.device
        t = self.codes_t
        return _CInt8Weight(self.n_out, self.k_in,
                            _vec(self.codes, (torch.uint8,), weight_bytes(self.n_out, self.k_in), "codes", dev),
                            None if t is None else _vec(t, (torch.uint8,), weight_bytes(self.k_in, self.n_out),
                                                        "codes_t", dev),
                            _vec(self.scale, (torch.float32,), self.n_out, "scale", dev))

    def nbytes(self) -> int:
        n = self.codes.numel() + 4 * self.scale.numel()
        return n + (0 if self.codes_t is None else self.codes_t.numel())


def weight_bytes(n_out: int, k_in: int) -> int:
    """Bytes of a weight's codes (qlora_int8_weight_bytes)."""
    return (n_out + 31) // 32 * 32 * ((k_in + 127) // 128 * 128)


def _transposed(w: Int8Weight) -> Int8Weight:
    t = torch.empty(weight_bytes(w.k_in, w.n_out), dtype=torch.uint8, device=w.codes.device)
    cw = w._c()
    st = qlora.lib().qlora_int8_transpose_weight(ctypes.byref(cw), t.data_ptr(), _stream(w.codes.device))
    if st:
        qlora._check(st, "qlora_int8_transpose_weight")
    w.codes_t = t
    return w


def quantize_weight(W: torch.Tensor, transposed: bool = False) -> Int8Weight:
    """fp32, bf16 or fp16 [n_out, k_in] -> Int8Weight.  ``transposed``: also
    lay out the transpose, which linear_bwd reads."""
    dt, (n, k), dev = _first(W, "W", tuple(DTYPES))
    p, ld = _mat(W, dt, W.shape, "W", dev)
    w = Int8Weight(torch.empty(weight_bytes(n, k), dtype=torch.uint8, device=dev),
                   torch.empty(n, dtype=torch.float32, device=dev), n, k)
    st = qlora.lib().qlora_int8_quantize_weight(p, DTYPES[dt], ld, n, k, w.codes.data_ptr(), w.scale.data_ptr(),
                                                _stream(dev))
    if st:
        qlora._check(st, "qlora_int8_quantize_weight")
    return _transposed(w) if transposed else w


def weight_from_codes(codes: torch.Tensor, scale: torch.Tensor, transposed: bool = False) -> Int8Weight:
    """int8 codes [n_out, k_in] and fp32 scales [n_out] from elsewhere (a
    checkpoint) -> Int8Weight with W = scale[:, None] * codes."""
    dt, (n, k), dev = _first(codes, "codes", (torch.int8,))
    p, ld = _mat(codes, dt, codes.shape, "codes", dev)
    _vec(scale, (torch.float32,), n, "scale", dev)
    w = Int8Weight(torch.empty(weight_bytes(n, k), dtype=torch.uint8, device=dev), scale.clone(), n, k)
    st = qlora.lib().qlora_int8_pack_weight(p, ld, n, k, w.codes.data_ptr(), _stream(dev))
    if st:
        qlora._check(st, "qlora_int8_pack_weight")
    return _transposed(w) if transposed else w


def dequant_weight(w: Int8Weight, out: torch.Tensor | None = None, dtype=torch.bfloat16) -> torch.Tensor:
    """The weight's values as a 16-bit [n_out, k_in] tensor."""
    dtype = dtype if out is None else out.dtype
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("dequant_weight produces bf16 or fp16")
    dev = w.codes.device
    out = _out(out, (w.n_out, w.k_in), dtype, "out", dev)
    cw = w._c()
    st = qlora.lib().qlora_int8_dequant_weight(ctypes.byref(cw), out.data_ptr(), DTYPES[dtype], _stream(dev))
    if st:
        qlora._check(st, "qlora_int8_dequant_weight")
    return out


def workspace_bytes(op: int, m: int, n_out: int, k_in: int) -> int:
    """Of linear_fwd (qlora.QLORA_OP_FWD) or linear_bwd (QLORA_OP_BWD)."""
    return int(qlora.lib().qlora_int8_workspace_bytes(op, m, n_out, k_in))


def plan(op: int, m: int, n_out: int, k_in: int, compute_units: int = 0) -> dict:
    """How the library runs a product (qlora_int8_plan)."""
    out = (ctypes.c_int64 * 3)()
    qlora._check(qlora.lib().qlora_int8_plan(op, m, n_out, k_in, compute_units, out), "qlora_int8_plan")
    return {"kernel": "tile" if out[0] == 256 else f"few{out[0]}", "splits": out[1], "quantizes_rows": bool(out[2])}


def linear_fwd(w: Int8Weight, X, bias: torch.Tensor | None = None, *, Y: torch.Tensor | None = None,
               ws: torch.Tensor | None = None) -> torch.Tensor:
    """Y = X W^T + bias.  X: a bf16 or fp16 matrix [M, k_in], quantized on the
    way in, or Int8Rows.  Y has X's type."""
    L = qlora.lib()
    cw = w._c()
    dev = w.codes.device
    if isinstance(X, Int8Rows):
        rows.check_rows(X, dev)
        m, dt = X.m, X.dtype
        if X.k != w.k_in:
            raise ValueError(f"X has {X.k} columns, the weight {w.k_in}")
    else:
        dt, shape, _ = _first(X, "X")
        m = shape[0]
        p, ld = _mat(X, dt, (m, w.k_in), "X", dev)
    b = None if bias is None else _vec(bias, (dt,), w.n_out, "bias", dev)
    Y = _out(Y, (m, w.n_out), dt, "Y", dev)
    if isinstance(X, Int8Rows):
        wst, wsn = qlora._ws(L.qlora_int8_rows_workspace_bytes(m, w.n_out, w.k_in), dev, ws)
        st = L.qlora_int8_linear_rows(ctypes.byref(cw), X.codes.data_ptr(), X.scale.data_ptr(), m, b, Y.data_ptr(),
                                      DTYPES[dt], None if wst is None else wst.data_ptr(), wsn, _stream(dev))
        if st:
            qlora._check(st, "qlora_int8_linear_rows")
        return Y
    wst, wsn = qlora._ws(L.qlora_int8_workspace_bytes(qlora.QLORA_OP_FWD, m, w.n_out, w.k_in), dev, ws)
    st = L.qlora_int8_linear_fwd(ctypes.byref(cw), p, ld, m, b, Y.data_ptr(), DTYPES[dt],
                                 None if wst is None else wst.data_ptr(), wsn, _stream(dev))
    if st:
        qlora._check(st, "qlora_int8_linear_fwd")
    return Y


def linear_bwd(w: Int8Weight, dY: torch.Tensor, *, dX: torch.Tensor | None = None,
               ws: torch.Tensor | None = None) -> torch.Tensor:
    """dX = dY W, with dY times the channels' scales quantized on the way in
    (the forward's rounding to 8 bits is passed straight through).  The weight
    needs its transpose.  There is no dW."""
    L = qlora.lib()
    cw = w._c()
    dt, shape, dev = _first(dY, "dY")
    m = shape[0]
    p, ld = _mat(dY, dt, (m, w.n_out), "dY", w.codes.device)
    dX = _out(dX, (m, w.k_in), dt, "dX", dev)
    wst, wsn = qlora._ws(L.qlora_int8_workspace_bytes(qlora.QLORA_OP_BWD, m, w.n_out, w.k_in), dev, ws)
    st = L.qlora_int8_linear_bwd(ctypes.byref(cw), p, ld, m, dX.data_ptr(), DTYPES[dt],
                                 None if wst is None else wst.data_ptr(), wsn, _stream(dev))
    if st:
        qlora._check(st, "qlora_int8_linear_bwd")
    return dX


class Int8LinearFunction(torch.autograd.Function):
    """Autograd wrapper: gradients for X and the bias; no grad for W.  X may be
    Int8Rows, through which no gradient passes."""

    @staticmethod
    def forward(ctx, X, bias, w: Int8Weight):
        ctx.w, ctx.bias_dtype = w, None if bias is None else bias.dtype
        if isinstance(X, Int8Rows):
            return linear_fwd(w, X, bias)
        if X.shape[-1] != w.k_in:  # a reshape to rows of k_in values could hide it
            raise ValueError(f"X has {X.shape[-1]} columns, the weight {w.k_in}")
        ctx.xshape = X.shape
        Y = rows._new((*X.shape[:-1], w.n_out), X)
        linear_fwd(w, rows._rows_of(X, w.k_in), bias, Y=rows._rows_of(Y, w.n_out))
        return Y

    @staticmethod
    @qlora._once
    def backward(ctx, dY):
        dY2 = rows._rows_of(dY, ctx.w.n_out)
        dX = linear_bwd(ctx.w, dY2).reshape(ctx.xshape) if ctx.needs_input_grad[0] else None
        db = dY2.sum(0, dtype=torch.float32).to(ctx.bias_dtype) if ctx.needs_input_grad[1] else None
        return dX, db, None


class Int8Linear(torch.nn.Module):
    """nn.Linear replacement with a frozen int8 weight.  ``transposed``: lay
    out what the backward needs."""

    def __init__(self, weight: torch.Tensor, bias: torch.Tensor | None = None, transposed: bool = False):
        super().__init__()
        self.w = quantize_weight(weight, transposed)
        self.bias = None if bias is None else torch.nn.Parameter(bias)

    def forward(self, X):
        if isinstance(X, Int8Rows) and not (torch.is_grad_enabled() and self.bias is not None and self.bias.requires_grad):
            return linear_fwd(self.w, X, self.bias)  # nothing to differentiate: without the wrapper's cost
        return Int8LinearFunction.apply(X, self.bias, self.w)


def _bind(L: ctypes.CDLL) -> None:
    i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    W = ctypes.POINTER(_CInt8Weight)
    sig = {
        "qlora_int8_weight_bytes": (sz, [i64, i64]),
        "qlora_int8_workspace_bytes": (sz, [i32, i64, i64, i64]),
        "qlora_int8_rows_workspace_bytes": (sz, [i64, i64, i64]),
        "qlora_int8_quantize_weight": (i32, [vp, i32, i64, i64, i64, vp, vp, vp]),
        "qlora_int8_pack_weight": (i32, [vp, i64, i64, i64, vp, vp]),
        "qlora_int8_transpose_weight": (i32, [W, vp, vp]),
        "qlora_int8_dequant_weight": (i32, [W, vp, i32, vp]),
        "qlora_int8_linear_fwd": (i32, [W, vp, i64, i64, vp, vp, i32, vp, sz, vp]),
        "qlora_int8_linear_rows": (i32, [W, vp, vp, i64, vp, vp, i32, vp, sz, vp]),
        "qlora_int8_plan": (i32, [i32, i64, i64, i64, i32, ctypes.POINTER(i64)]),
        "qlora_debug_int8_linear_rows": (i32, [W, vp, vp, i64, vp, vp, i32, i32, i32, vp, sz, vp]),
        "qlora_int8_linear_bwd": (i32, [W, vp, i64, i64, vp, i32, vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
