"""Plain 64-bit reference of the row-wise operators and the int8 product.

Inputs are float64 arrays holding the exact values of the 16- or 32-bit
tensors the kernels read; nothing is rounded except where the operator's
definition rounds (codes to integers).
"""

from __future__ import annotations

import numpy as np

AMAX_FLOOR = 1e-30


def quantize_rows(x: np.ndarray):
    """(codes, scale): amax = max(max|x|, floor), scale = amax / 127, code =
    127 x / amax to nearest, ties to even.  Non-finite rows: codes 0, scale NaN."""
    m = x.shape[0]
    ok = np.isfinite(x).all(axis=1)
    v = np.where(ok[:, None], x, 0.0)
    amax = np.maximum(np.abs(v).max(axis=1) if x.shape[1] else np.zeros(m), AMAX_FLOOR)
    codes = np.rint(v * 127.0 / amax[:, None])
    return codes, np.where(ok, amax / 127.0, np.nan)


def rms_norm_fwd(h: np.ndarray, gamma: np.ndarray, eps: float):
    """(y, rstd) of the hidden state h as it is stored."""
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * gamma, rstd


def rms_norm_bwd(dy: np.ndarray, h: np.ndarray, gamma: np.ndarray, eps: float, dh: np.ndarray | None = None):
    """(dx, dgamma) for the outputs y and (with dh) h."""
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    hat, g = h * rstd, dy * gamma
    dx = rstd * (g - hat * (g * hat).mean(axis=1, keepdims=True))
    return dx if dh is None else dx + dh, (dy * hat).sum(axis=0)


def sigmoid(g: np.ndarray) -> np.ndarray:
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def swiglu_fwd(g: np.ndarray, u: np.ndarray) -> np.ndarray:
    return g * sigmoid(g) * u


def swiglu_bwd(dy: np.ndarray, g: np.ndarray, u: np.ndarray):
    s = sigmoid(g)
    return dy * u * s * (1.0 + g * (1.0 - s)), dy * g * s


def int8_linear(qx: np.ndarray, sx: np.ndarray, qw: np.ndarray, sw: np.ndarray | None, bias=None) -> np.ndarray:
    """sx[m] sw[n] sum_k qx[m][k] qw[n][k] + bias[n]; the sum is exact (every
    partial sum is a whole number below 2^53)."""
    y = (qx @ qw.T) * sx[:, None]
    if sw is not None:
        y = y * sw[None, :]
    return y if bias is None else y + bias[None, :]
