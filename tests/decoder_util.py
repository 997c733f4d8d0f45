"""References and error bounds of the attention tests.

Bounds.  U is a rounding to the 16-bit type (half a step), E = 2^-24 one in
fp32.  Scores are sums of d products in fp32: off by at most ds = (d + 8) E
scale sum |q k|, and p = exp(s - lse) by a relative 2 ds + 2^-20 (the exponential,
the reference's rounding, the sum of p: at most 64 additions in a row, and the
keys of a sequence in at most 64 tiles a factor of two larger than E each).
P is rounded to 16 bits as an operand, relative U (fp16: at least half its
smallest step, 2^-25, of the row's largest), and the output once more:

    |dO| <= sum_j p_j |v_j| (U + rel) + U |o|

Backward: delta is a sum over O as it is stored, so off by U sum |do o|, and dS
= p (dp - delta) by p (U sum |do o| + 2^-20 (sum |do v| + |delta|)) + (U + rel) |dS|;
dQ, dK and dV are sums of those times K, Q (or dO), rounded once.  The
exponential and the matrix operands have no subnormal values: a p or dS below
2^-126 may be zero, an error of at most FLUSH = 2^-126 in it, which counts where
every score of a row's other keys is 87 below the largest.  (fp16 operands
that a power of two keeps in range add less than 2^-37 of their bound.)
"""

import numpy as np
import torch

import oracle.decoder as ref
from rows_util import TINY, U, f64

E = 2.0 ** -24
FLUSH = 2.0 ** -126


def starts(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)


def cu(lengths):
    return torch.tensor(starts(lengths).tolist(), dtype=torch.int32, device="cuda")


def _head(q, k, v, scale, causal, dtype, do=None):
    """Reference and bound of each output of one head of one sequence."""
    u, d = U[dtype], q.shape[1]
    small = 2.0 ** -25 if dtype == torch.float16 else 0.0
    p, lse, seen = ref.softmax_rows(q, k, scale, causal)
    out = ref.attention_head(q, k, v, scale, causal, do)
    ds = (d + 8) * E * scale * np.where(seen, np.abs(q) @ np.abs(k).T, 0.0).max(1, initial=0.0)[:, None]
    rel = 2 * ds + 2.0 ** -20
    sv = seen @ np.abs(v)
    o_err = ((u + rel) * p) @ np.abs(v) + (small + FLUSH) * sv + u * np.abs(out[0])
    lse_err = ds[:, 0] + 2.0 ** -20 * (1 + np.abs(np.where(np.isinf(lse), 0.0, lse)))
    if do is None:
        return out, (o_err, lse_err)
    dp = do @ v.T
    adv, ado = np.abs(do) @ np.abs(v).T, (np.abs(do) * np.abs(out[0])).sum(1, keepdims=True)
    s = p * (dp - (p * dp).sum(1, keepdims=True))
    bound = 2 * d * np.abs(do).max(initial=0.0) * np.abs(v).max(initial=0.0)
    serr = p * (u * ado * 1.02 + 2.0 ** -20 * (adv + ado)) + (u + 2 * rel) * np.abs(s) + (small * 2.0 ** -12 * bound + FLUSH * (1 + adv + ado)) * seen
    perr = (u + 2 * rel) * p + (small * 2.0 ** -12 + 2 * FLUSH) * seen
    dq_err = scale * serr @ np.abs(k) + u * np.abs(out[2])
    dk_err = scale * serr.T @ np.abs(q)
    dv_err = perr.T @ np.abs(do)
    return out, (o_err, lse_err, dq_err, dk_err, dv_err)


def attention_reference(q, k, v, lq, lk, causal, scale=None, do=None, at_q=None, at_k=None):
    """{name: (reference, bound)} over all sequences and heads, from GPU tensors.
    at_q, at_k: where the sequences start (default: one after another)."""
    dtype = q.dtype
    (tq, h, d), (tk, hk, _) = q.shape, k.shape
    group, scale = h // hk, d ** -0.5 if scale is None else scale
    Q, K, V = f64(q), f64(k), f64(v)
    D = None if do is None else f64(do)
    at_q, at_k = starts(lq) if at_q is None else at_q, starts(lk) if at_k is None else at_k
    res = {"o": (np.zeros((tq, h, d)), np.zeros((tq, h, d))), "lse": (np.full((tq, h), -np.inf), np.zeros((tq, h)))}
    if do is not None:
        res.update(dq=(np.zeros((tq, h, d)), np.zeros((tq, h, d))), dk=(np.zeros((tk, hk, d)), np.zeros((tk, hk, d))),
                   dv=(np.zeros((tk, hk, d)), np.zeros((tk, hk, d))))
    for n, m, a, b in zip(lq, lk, at_q, at_k):
        for i in range(h):
            j, qs, ks = i // group, slice(a, a + n), slice(b, b + m)
            out, err = _head(Q[qs, i], K[ks, j], V[ks, j], scale, causal, dtype, None if D is None else D[qs, i])
            for x, y, name in zip(out, err, ("o", "lse", "dq", "dk", "dv")):
                r, e = res[name]
                if name in ("dk", "dv"):
                    r[ks, j] += x
                    e[ks, j] += y
                else:
                    r[qs, i], e[qs, i] = x, y
    if do is not None:
        for name in ("dk", "dv"):
            r, e = res[name]
            e += U[dtype] * (np.abs(r) + e)
    return res


def close(got, want, what=""):
    """A tensor against (reference, bound); infinities have to be equal."""
    r, e = want
    g = f64(got)
    tiny = TINY.get(got.dtype, 0.0)
    with np.errstate(invalid="ignore"):
        ok = (g == r) | (np.abs(g - r) <= e * (1 + 2.0 ** -6) + tiny)
    if not ok.all():
        at = tuple(np.argwhere(~ok)[0])
        raise AssertionError(f"{what}: {(~ok).sum()} of {ok.size} outside the bound, first at {at}: got {g[at]}, want "
                             f"{r[at]} within {e[at]}; rms error {np.sqrt(np.nanmean((g - r)[np.isfinite(r)] ** 2)):.3g}")
