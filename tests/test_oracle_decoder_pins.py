"""Pins of the 64-bit reference of rotary positions, attention and the head's cross
entropy: definitions written out by hand, gradients against central differences."""

import numpy as np
import pytest

import oracle.decoder as ref


def _central(f, x, step=1e-5):
    out = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += step
        lo[i] -= step
        out[i] = (f(hi) - f(lo)) / (2 * step)
    return out


def test_rotation():
    g = np.random.default_rng(0)
    x, f = g.normal(size=(5, 2, 8)), np.array([1.0, 0.1, 0.01])
    y = ref.rotate(x, np.arange(5), f)
    # a quarter turn, by hand; the last two values are not turned
    q = ref.rotate(x, [1] * 5, [np.pi / 2])
    assert np.allclose(q[..., 0], -x[..., 1]) and np.allclose(q[..., 1], x[..., 0]) and np.array_equal(q[..., 2:], x[..., 2:])
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 6:], x[..., 6:])
    # lengths of pairs, the inverse, and scores that depend on the distance alone
    assert np.allclose(np.hypot(y[..., :3], y[..., 3:6]), np.hypot(x[..., :3], x[..., 3:6]))
    assert np.allclose(ref.rotate(y, np.arange(5), f, inverse=True), x)
    a, b = x[:1], x[1:2]
    dot = lambda i, j: (ref.rotate(a, [i], f) * ref.rotate(b, [j], f)).sum()
    assert np.isclose(dot(3, 1), dot(1002, 1000))
    z = ref.rotate(x, np.arange(5), f, 2.0, interleaved=True)
    order = [0, 2, 4, 1, 3, 5, 6, 7]
    assert np.allclose(z[..., order][..., :6], ref.rotate(x[..., order], np.arange(5), f, 2.0)[..., :6])


@pytest.mark.parametrize("n,m,causal", [(4, 4, True), (3, 6, True), (5, 2, True), (3, 4, False), (1, 1, True)])
def test_attention(n, m, causal):
    g = np.random.default_rng(n + m)
    q, k, v, do = g.normal(size=(n, 6)), g.normal(size=(m, 6)), g.normal(size=(m, 6)), g.normal(size=(n, 6))
    o, lse, dq, dk, dv = ref.attention_head(q, k, v, 0.4, causal, do)
    for i in range(n):
        seen = [j for j in range(m) if not causal or j <= i + m - n]
        if not seen:
            assert not o[i].any() and lse[i] == -np.inf and not dq[i].any()
            continue
        e = np.array([np.exp(0.4 * q[i] @ k[j]) for j in seen])
        assert np.allclose(o[i], (e[:, None] * v[seen]).sum(0) / e.sum()) and np.isclose(lse[i], np.log(e.sum()))
    loss = lambda a, b, c: (ref.attention_head(a, b, c, 0.4, causal)[0] * do).sum()
    np.testing.assert_allclose(dq, _central(lambda t: loss(t, k, v), q), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(dk, _central(lambda t: loss(q, t, v), k), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(dv, _central(lambda t: loss(q, k, t), v), rtol=1e-6, atol=1e-8)


def test_cross_entropy():
    g = np.random.default_rng(2)
    x, w, y = g.normal(size=(4, 5)), g.normal(size=(7, 5)), np.array([2, 6, -100, 0])
    loss, lse, dx = ref.cross_entropy(x, w, y, dloss=np.array([1.0, 0.5, 9.0, 2.0]))
    z = x @ w.T
    want = np.log(np.exp(z).sum(1))
    assert np.allclose(lse, want) and loss[2] == 0 and not dx[2].any()
    assert np.allclose(loss[[0, 1, 3]], (want - z[np.arange(4), [2, 6, 0, 0]])[[0, 1, 3]])
    f = lambda t: (ref.cross_entropy(t, w, y)[0] * [1.0, 0.5, 9.0, 2.0]).sum()
    np.testing.assert_allclose(dx, _central(f, x), rtol=1e-6, atol=1e-8)
    # a target far above the rest: e^-40, which one minus a probability does not show
    big, _, _ = ref.cross_entropy(np.array([[40.0]]), np.array([[1.0], [0.0]]), np.array([0]))
    assert np.isclose(big[0], np.exp(-40.0), rtol=1e-12)
