"""Corners of the row-wise operators on the GPU: rows of no values."""

import numpy as np
import pytest
import torch

from bit_nf4_quantized_double_amd import int8, rows
from rows_util import f64, need_gpu, rand

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
