"""Attention of packed sequences over libqlora.so, for training, prompts and
single tokens over a cache.

:func:`attention_fwd` and :func:`attention_bwd` are the two passes,
:func:`attention` the differentiable form.  Formulas, masks, rounding and limits:
include/qlora.h.

Q is bf16 or fp16 [tokens, heads, head_dim], K and V [tokens, kv_heads, head_dim],
the sequences' tokens one after another; ``cu_q`` and ``cu_k`` (int32 [sequences +
1], on the GPU) say where each begins and ends, and ``lengths_q``, ``lengths_k``
(int32 [sequences]) how much of that is used, where it is not all: a padded batch
[n, room, heads, d] is its view [n * room, heads, d] with ``cu = room * arange(n +
1)``.  Under a causal mask a sequence's queries are its last tokens: one query
over a cache is the next token.
"""

from __future__ import annotations

import ctypes

import torch

from . import qlora
from .rotary import CHeads, check_heads, check_vector
from .rows import DTYPES, _stream

MAX_HEAD_DIM = 128
_I32 = (torch.int32,)


class _CAttention(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("tokens_q", "tokens_k", "batch", "heads", "kv_heads", "head_dim")] + [
        (n, ctypes.c_void_p) for n in ("cu_q", "cu_k", "len_q", "len_k")] + [
        ("scale", ctypes.c_float), ("causal", ctypes.c_int), ("zero_rest", ctypes.c_int), ("dtype", ctypes.c_int)]


def _describe(Q, K, V, cu_q, cu_k, lengths_q, lengths_k, causal, scale, zero_rest):
    """(descriptor, Q, K, V as the library takes them)."""
    q = check_heads(Q, "Q")
    dt, dev = Q.dtype, Q.device
    tq, h, d = Q.shape
    k = check_heads(K, "K", dt, None, dev)
    tk, hk, dk = K.shape
    if dk != d:
        raise ValueError(f"K has heads of {dk}, Q of {d}")
    if hk == 0 or h % hk:
        raise ValueError(f"{h} heads of Q are no multiple of {hk} of K")
    if not 0 < d <= MAX_HEAD_DIM or d % 8:
        raise ValueError(f"heads of {d}: a multiple of 8 up to {MAX_HEAD_DIM} is needed")
    v = check_heads(V, "V", dt, K.shape, dev)
    if not isinstance(cu_q, torch.Tensor) or cu_q.dim() != 1 or cu_q.shape[0] < 1:
        raise ValueError("cu_q must be a vector of int32, one more than sequences")
    n = cu_q.shape[0] - 1
    if cu_k is None:
        if tk != tq:
            raise ValueError("without cu_k, K must have Q's tokens")
        cu_k = cu_q
        if lengths_k is None:
            lengths_k = lengths_q
    scale = d ** -0.5 if scale is None else float(scale)
    c = _CAttention(tq, tk, n, h, hk, d, check_vector(cu_q, _I32, n + 1, "cu_q", dev),
                    check_vector(cu_k, _I32, n + 1, "cu_k", dev),
                    None if lengths_q is None else check_vector(lengths_q, _I32, n, "lengths_q", dev),
                    None if lengths_k is None else check_vector(lengths_k, _I32, n, "lengths_k", dev),
                    scale, bool(causal), bool(zero_rest), DTYPES[dt])
    return c, q, k, v


def _new(shape, like):
    return torch.empty(shape, dtype=like.dtype, device=like.device)


def plan(Q, K, cu_q, compute_units: int = 0) -> dict:
    """How the library runs a forward (qlora_attention_plan)."""
    c, *_ = _describe(Q, K, K, cu_q, torch.zeros_like(cu_q), None, None, True, None, False)
    out = (ctypes.c_int64 * 2)()
    qlora._check(qlora.lib().qlora_attention_plan(ctypes.byref(c), compute_units, out), "qlora_attention_plan")
    return {"rows": out[0], "splits": out[1]}


def attention_fwd(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor | None = None,
                  *, lengths_q: torch.Tensor | None = None, lengths_k: torch.Tensor | None = None, causal: bool = True,
                  scale: float | None = None, O: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None):
    """Returns (O, lse fp32 [tokens, heads]).  ``cu_k`` None: the keys are at the
    queries' places.  ``scale``: head_dim^-1/2.  Tokens of no sequence: zeros (lse
    -inf) in new outputs; where O is given they stay as they are in both."""
    c, q, k, v = _describe(Q, K, V, cu_q, cu_k, lengths_q, lengths_k, causal, scale, O is None)
    dev = Q.device
    if O is None:
        O = _new(Q.shape, Q)
    o = check_heads(O, "O", Q.dtype, Q.shape, dev)
    if lse is None:
        lse = torch.empty(Q.shape[:2], dtype=torch.float32, device=dev)
    elif lse.dtype != torch.float32 or lse.shape != Q.shape[:2] or lse.device != dev or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 tensor of shape {tuple(Q.shape[:2])} on {dev}")
    L = qlora.lib()
    r = ctypes.byref
    wst, wsn = qlora._ws(L.qlora_attention_workspace_bytes(qlora.QLORA_OP_FWD, r(c)), dev, ws)
    st = L.qlora_attention_fwd(r(c), r(q), r(k), r(v), r(o), lse.data_ptr(), None if wst is None else wst.data_ptr(), wsn,
                               _stream(dev))
    if st:
        qlora._check(st, "qlora_attention_fwd")
    return O, lse


def attention_bwd(dO: torch.Tensor, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, O: torch.Tensor, lse: torch.Tensor,
                  cu_q: torch.Tensor, cu_k: torch.Tensor | None = None, *, lengths_q: torch.Tensor | None = None,
                  lengths_k: torch.Tensor | None = None, causal: bool = True, scale: float | None = None,
                  dQ: torch.Tensor | None = None, dK: torch.Tensor | None = None, dV: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None):
    """Returns (dQ, dK, dV) from the forward's O and lse.  Tokens of no sequence:
    zeros in new outputs; where dQ, dK and dV are given (all three) they stay as
    they are."""
    given = [g is not None for g in (dQ, dK, dV)]
    if any(given) and not all(given):
        raise ValueError("give all of dQ, dK and dV, or none")
    c, q, k, v = _describe(Q, K, V, cu_q, cu_k, lengths_q, lengths_k, causal, scale, dQ is None)
    dev, dt = Q.device, Q.dtype
    do = check_heads(dO, "dO", dt, Q.shape, dev)
    o = check_heads(O, "O", dt, Q.shape, dev)
    if not isinstance(lse, torch.Tensor) or lse.dtype != torch.float32 or lse.shape != Q.shape[:2] or lse.device != dev \
            or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 tensor of shape {tuple(Q.shape[:2])} on {dev}")
    if dQ is None:
        dQ, dK, dV = _new(Q.shape, Q), _new(K.shape, K), _new(V.shape, V)
    gq, gk, gv = (check_heads(t, n, dt, s, dev) for t, n, s in ((dQ, "dQ", Q.shape), (dK, "dK", K.shape), (dV, "dV", V.shape)))
    L = qlora.lib()
    r = ctypes.byref
    wst, wsn = qlora._ws(L.qlora_attention_workspace_bytes(qlora.QLORA_OP_BWD, r(c)), dev, ws)
    st = L.qlora_attention_bwd(r(c), r(do), r(q), r(k), r(v), r(o), lse.data_ptr(), r(gq), r(gk), r(gv),
                               None if wst is None else wst.data_ptr(), wsn, _stream(dev))
    if st:
        qlora._check(st, "qlora_attention_bwd")
    return dQ, dK, dV


def _aligned(t: torch.Tensor) -> torch.Tensor:
    """As the kernels read it: 16-byte rows of heads; a copy where it is not."""
    n, h, d = t.shape
    if t.numel() and (t.stride(2) != 1 or t.data_ptr() % 16 or (n > 1 and t.stride(0) % 8) or (h > 1 and t.stride(1) % 8)):
        t = t.contiguous()
        return t if t.data_ptr() % 16 == 0 else t.clone()
    return t


class AttentionFunction(torch.autograd.Function):
    """(Q, K, V) -> O."""

    @staticmethod
    def forward(ctx, Q, K, V, cu_q, cu_k, lengths_q, lengths_k, causal: bool, scale):
        for t, name in ((Q, "Q"), (K, "K"), (V, "V")):
            if not isinstance(t, torch.Tensor) or t.dim() != 3:
                raise ValueError(f"{name} must be a [tokens, heads, head_dim] tensor")
        Q, K, V = _aligned(Q), _aligned(K), _aligned(V)
        O, lse = attention_fwd(Q, K, V, cu_q, cu_k, lengths_q=lengths_q, lengths_k=lengths_k, causal=causal, scale=scale)
        ctx.save_for_backward(Q, K, V, O, lse, cu_q, cu_k, lengths_q, lengths_k)
        ctx.causal, ctx.scale = causal, scale
        return O

    @staticmethod
    @qlora._once
    def backward(ctx, dO):
        Q, K, V, O, lse, cu_q, cu_k, lengths_q, lengths_k = ctx.saved_tensors
        dQ, dK, dV = attention_bwd(_aligned(dO), Q, K, V, O, lse, cu_q, cu_k, lengths_q=lengths_q, lengths_k=lengths_k,
                                   causal=ctx.causal, scale=ctx.scale)
        return dQ, dK, dV, None, None, None, None, None, None


def attention(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor | None = None, *,
              lengths_q: torch.Tensor | None = None, lengths_k: torch.Tensor | None = None, causal: bool = True,
              scale: float | None = None) -> torch.Tensor:
    """Differentiable attention of packed sequences: O.  Gradients for Q, K and V."""
    return AttentionFunction.apply(Q, K, V, cu_q, cu_k, lengths_q, lengths_k, bool(causal), scale)


def _bind(L: ctypes.CDLL) -> None:
    i32, vp, sz = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    A, H = ctypes.POINTER(_CAttention), ctypes.POINTER(CHeads)
    sig = {
        "qlora_attention_workspace_bytes": (sz, [i32, A]),
        "qlora_attention_plan": (i32, [A, i32, ctypes.POINTER(ctypes.c_int64)]),
        "qlora_attention_fwd": (i32, [A, H, H, H, H, vp, vp, sz, vp]),
        "qlora_attention_bwd": (i32, [A, H, H, H, H, H, vp, H, H, H, vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
