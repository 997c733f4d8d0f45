"""Plain fp64 reference of rotary positions, attention and the head's cross
entropy (numpy, one sequence and one head at a time; shares nothing with the
kernels)."""

import numpy as np


def rotate(x, positions, f, factor=1.0, interleaved=False, inverse=False):
    """x [tokens, heads, d], positions [tokens] whole numbers, f [r / 2] radians a position."""
    x = np.array(x, dtype=np.float64)
    f = np.asarray(f, dtype=np.float64)
    n = len(f)
    # the angle modulo a turn in extended precision: far positions have more radians than fp64 has digits for
    angle = np.remainder(np.asarray(positions, dtype=np.longdouble)[:, None] * f.astype(np.longdouble), 2 * np.pi)
    c, s = (np.asarray(t(angle), dtype=np.float64)[:, None, :] * factor for t in (np.cos, np.sin))
    s = -s if inverse else s
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def _seen(n, m, causal):
    i, j = np.arange(n)[:, None], np.arange(m)[None, :]
    return (j <= i + m - n) if causal else np.ones((n, m), dtype=bool)


def softmax_rows(q, k, scale, causal):
    """(P, lse, seen) of one head of one sequence; rows that see nothing are zeros."""
    seen = _seen(len(q), len(k), causal)
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.where(seen, scale * (q @ k.T), -np.inf)
        top = z.max(1, initial=-np.inf)
        e = np.where(seen, np.exp(z - np.where(np.isneginf(top), 0.0, top)[:, None]), 0.0)
        total = e.sum(1)
        lse = np.where(np.isneginf(top), 0.0, top) + np.log(total)
        p = np.where(total[:, None] > 0, e / total[:, None], 0.0)
    return p, np.where(total > 0, lse, -np.inf), seen


def attention_head(q, k, v, scale, causal, do=None):
    """O, lse and (with dO) dQ, dK, dV of one head of one sequence."""
    p, lse, _ = softmax_rows(q, k, scale, causal)
    o = p @ v
    if do is None:
        return o, lse
    dp = do @ v.T
    ds = p * (dp - (p * dp).sum(1, keepdims=True))
    return o, lse, scale * ds @ k, scale * ds.T @ q, p.T @ do


def cross_entropy(x, w, targets, ignore_index=-100, dloss=None):
    """loss, log-sum and the gradient of x: dloss (softmax - 1 at the target) W."""
    z = x @ w.T
    top = z.max(1)
    e = np.exp(z - top[:, None])
    total = e.sum(1)
    live = targets != ignore_index
    at = np.where(live, targets, 0)
    rows = np.arange(len(x))
    mine = e[rows, at]
    e[rows, at] = 0.0
    rest = e.sum(1)
    # log(total / mine) with mine apart: small losses keep their digits
    loss = np.where(live, np.log1p(rest / mine), 0.0)
    g = np.where(live, 1.0 if dloss is None else dloss, 0.0)
    dx = g[:, None] * ((e / total[:, None]) @ w - (rest / total)[:, None] * w[at])
    return loss, top + np.log(total), dx
