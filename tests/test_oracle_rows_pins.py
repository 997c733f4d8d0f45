"""Pins of the 64-bit reference of the row-wise operators: gradients against
central differences, the quantizer against its definition."""

import numpy as np
import pytest

import oracle.rows as ref

EPS = 1e-5


def _central(f, x, step=1e-5):
    """d sum(f(x)) / dx entry by entry."""
    out = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += step
        lo[i] -= step
        out[i] = (f(hi) - f(lo)) / (2 * step)
    return out


@pytest.mark.parametrize("m,k", [(1, 1), (3, 7), (2, 16)])
def test_rms_norm_gradient_against_differences(m, k):
    g = np.random.default_rng(m + k)
    h, dy, dh, gamma = g.normal(size=(m, k)), g.normal(size=(m, k)), g.normal(size=(m, k)), g.normal(size=k)
    dx, dgamma = ref.rms_norm_bwd(dy, h, gamma, EPS, dh)
    # the error of a central difference: step^2 / 6 times a third derivative,
    # and the rounding of the two values over the step
    np.testing.assert_allclose(dx, _central(lambda v: (ref.rms_norm_fwd(v, gamma, EPS)[0] * dy + v * dh).sum(), h),
                               rtol=1e-6, atol=1e-6)
    np.testing.assert_allclose(dgamma, _central(lambda v: (ref.rms_norm_fwd(h, v, EPS)[0] * dy).sum(), gamma),
                               rtol=1e-6, atol=1e-6)


def test_swiglu_gradient_against_differences():
    g = np.random.default_rng(5)
    a, u, dy = g.normal(size=(3, 9)) * 3, g.normal(size=(3, 9)), g.normal(size=(3, 9))
    dg, du = ref.swiglu_bwd(dy, a, u)
    np.testing.assert_allclose(dg, _central(lambda v: (ref.swiglu_fwd(v, u) * dy).sum(), a), rtol=1e-6, atol=1e-6)
    np.testing.assert_allclose(du, _central(lambda v: (ref.swiglu_fwd(a, v) * dy).sum(), u), rtol=1e-6, atol=1e-6)


def test_sigmoid_ends():
    with np.errstate(over="raise"):
        s = ref.sigmoid(np.array([-1e4, -700.0, 0.0, 700.0, 1e4]))
    assert s[0] == 0 and s[2] == 0.5 and s[4] == 1


def test_quantizer():
    x = np.array([[0.0, 1.0, -2.0, 127.0], [0.0, 0.0, 0.0, 0.0], [1.0, np.inf, 0.0, 0.0], [np.nan, 1.0, 2.0, 3.0],
                  [0.5, 1.5, 2.5, 127.0]])
    codes, scale = ref.quantize_rows(x)
    assert np.array_equal(codes, [[0, 1, -2, 127], [0, 0, 0, 0], [0, 0, 0, 0], [0, 0, 0, 0], [0, 2, 2, 127]])
    assert scale[0] == 1 and scale[1] == 1e-30 / 127 and np.isnan(scale[2:4]).all()
    g = np.random.default_rng(0)
    x = g.normal(size=(20, 50))
    codes, scale = ref.quantize_rows(x)
    assert np.abs(codes).max() == 127
    assert (np.abs(codes * scale[:, None] - x) <= 0.5 * scale[:, None] * (1 + 1e-12)).all()


def test_product():
    g = np.random.default_rng(1)
    qx, qw = g.integers(-127, 128, (4, 30)), g.integers(-127, 128, (5, 30))
    sx, sw, b = g.random(4), g.random(5), g.random(5)
    want = (qx * sx[:, None]) @ (qw * sw[:, None]).T + b
    np.testing.assert_allclose(ref.int8_linear(qx.astype(float), sx, qw.astype(float), sw, b), want, rtol=1e-13)
