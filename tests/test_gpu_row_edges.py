"""Corners of the row-wise operators on the GPU: rows of no values,
gates far out, and more rows than a launch has in one dimension."""

import numpy as np
import pytest
import torch

import oracle.rows as ref
from bit_nf4_quantized_double_amd import int8, rows
from rows_util import E32, TINY, U, f64, need_gpu, rand

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
EPS = 1e-5


@pytest.mark.parametrize("m", [1, 3, 2000])
def test_norm_in_8_bits_of_no_values(m):
    """A row of no values is a row of zeros: its scale is the floor's, as the
    quantizer's and SwiGLU's, and a product of it is the bias."""
    need_gpu()
    x, g = torch.empty((m, 0), dtype=BF16, device="cuda"), torch.empty(0, dtype=BF16, device="cuda")
    want = rows.quantize_rows(x).scale
    for residual in (None, x):
        stale = torch.full((1 << 16,), float("nan"), device="cuda")
        del stale  # what a new buffer is likely to hold
        q, h = rows.rms_norm_int8(x, g, EPS, residual)
        assert h.shape == (m, 0)
        np.testing.assert_allclose(f64(q.scale), f64(want), rtol=2.0 ** -21)
        b = rand((40,), 2)
        w = int8.quantize_weight(torch.empty((40, 0), device="cuda"))
        assert torch.equal(int8.linear_fwd(w, q, b), b.expand(m, 40))
        stale = torch.full((m,), float("nan"), device="cuda")
        del stale
        _, _, rstd = rows.rms_norm_fwd(x, g, EPS, residual)
        np.testing.assert_allclose(f64(rstd), EPS ** -0.5, rtol=2.0 ** -21)


def test_swiglu_gates_whose_sigmoid_is_subnormal():
    """1 / (1 + e^-g) below 2^-126 is a number still, and its products with a
    large u or dY are ordinary ones.  The bound: half a spacing of the
    output's type and that of s, whose spacing there is 2^-149."""
    need_gpu()
    g = torch.tensor([[-86.0, -87.0, -87.5, -88.0, -88.5]], dtype=BF16, device="cuda")
    for c in (1.0, 1e4, 1e30):
        u = torch.full_like(g, c)
        G, C = f64(g), f64(u)
        s = ref.sigmoid(G)
        # e^-g through 2^(-g log2 e) in fp32: |g| 2^-24 and a few roundings
        def near(got, want, slope):
            err = np.abs(want) * (U[BF16] + (1 + np.abs(G)) * E32) + slope * 2.0 ** -149 + TINY[BF16]
            assert (np.abs(f64(got) - want) <= err).all(), (f64(got), want)
        near(rows.swiglu_fwd(g, u), ref.swiglu_fwd(G, C), np.abs(G) * C)
        dg, du = rows.swiglu_bwd(u, g, u)
        wg, wu = ref.swiglu_bwd(C, G, C)
        if c * c < 1e38:
            near(dg, wg, C * C * (1 + np.abs(G)))
        near(du, wu, np.abs(G) * C)


def _same(a, b):
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_more_rows_than_a_launch_dimension():
    """A row takes 64 threads or more, and a dimension of a launch fewer than
    2^32 threads: the rows around that edge and the last ones are those of
    calls of their own."""
    need_gpu()
    m, k = (1 << 26) + 70, 16
    x, g = rand((4099, k), 1).repeat(m // 4099 + 1, 1)[:m], rand((k,), 2)
    parts = [slice(0, 100), slice((1 << 26) - 50, (1 << 26) + 50), slice(m - 70, m)]
    y, _, rstd = rows.rms_norm_fwd(x, g, EPS)
    for p in parts:
        a, _, c = rows.rms_norm_fwd(x[p], g, EPS)
        _same((y[p], rstd[p]), (a, c))
    del rstd
    for call in (lambda t: rows.rms_norm_int8(t, g, EPS)[0], rows.quantize_rows, lambda t: rows.swiglu_int8(t, t)):
        q = call(x)
        v = rows.dequant_rows(q)
        for p in parts:
            few = call(x[p])
            assert torch.equal(v[p], rows.dequant_rows(few))
            assert torch.equal(q.scale[p], few.scale)
        del q, v


def test_more_8_bit_rows_and_outputs_than_a_launch_dimension():
    """Reading rows back, packing a weight and the product of few tokens take
    fewer threads a row; the values are exact, so all of them are compared."""
    need_gpu()
    m = (1 << 28) + 40
    x = (torch.arange(1, 252, device="cuda") - 126).to(BF16).repeat(m // 251 + 1)[:m].reshape(m, 1)
    assert torch.equal(rows.dequant_rows(rows.quantize_rows(x)), x)
    codes = x.to(torch.int8)
    w = int8.weight_from_codes(codes, torch.ones(m, device="cuda"))
    assert torch.equal(int8.dequant_weight(w), x)
    one = torch.tensor([[1.0], [-2.0]], dtype=BF16, device="cuda")
    y = int8.linear_fwd(w, one)
    assert torch.equal(y[0], x[:, 0]) and torch.equal(y[1], -2 * x[:, 0])
