"""The int8 product on the GPU against the 64-bit reference (bounds:
rows_util).  The integer sum is exact, so the only errors are the scales'
products, the bias and the output's rounding."""

import ctypes

import numpy as np
import pytest
import torch

import oracle.rows as ref
from bit_nf4_quantized_double_amd import int8, qlora, rows
from rows_util import close16, codes_of, f64, need_gpu, rand, strided

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32

# (M, n_out, k_in): one of each; ragged tiles of outputs, tokens and the
# reduction; the few tokens' kernels and their edges (16, 17, 64, 65 tokens),
# which the plan takes for all of these forwards (tiles and splits:
# test_gpu_int8_plans.py)
SHAPES = [(1, 1, 1), (1, 33, 64), (2, 31, 100), (5, 130, 129), (16, 256, 256), (17, 64, 128), (16, 1000, 2500),
          (33, 96, 1000), (64, 520, 4096), (65, 520, 512), (100, 260, 300), (128, 128, 128), (150, 1000, 2500),
          (257, 513, 640), (300, 4096, 1024), (512, 256, 8192), (1, 8192, 4096), (3, 256, 28672), (700, 130, 65)]


def _weight(n, k, seed, dtype=F32):
    W = rand((n, k), seed, dtype, 0.02)
    return W, int8.quantize_weight(W, transposed=True)


def _product(q, w, got, bias=None):
    want = ref.int8_linear(codes_of(q), f64(q.scale), codes_of(w), f64(w.scale), None if bias is None else f64(bias))
    mag = np.abs(want) + (0 if bias is None else np.abs(f64(bias))[None, :])
    close16(got, want, mag, "Y")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear(m, n, k, dtype):
    need_gpu()
    W, w = _weight(n, k, n + k)
    want, scale = ref.quantize_rows(f64(W))
    np.testing.assert_allclose(f64(w.scale), scale, rtol=2.0 ** -22)
    assert (np.abs(codes_of(w) - f64(W) / scale[:, None]) <= 0.5 + 127 * 2.0 ** -22).all()
    x = rand((m, k), m + k, dtype)
    bias = rand((n,), 3, dtype)
    q = rows.quantize_rows(x)
    y = int8.linear_fwd(w, x)
    _product(q, w, y)
    _product(q, w, int8.linear_fwd(w, x, bias), bias)
    assert torch.equal(y, int8.linear_fwd(w, q))
    assert torch.equal(y, int8.linear_fwd(w, strided(x, 24, 8)))
    if qlora.lib().qlora_int8_rows_workspace_bytes(m, n, k):
        # without room for split sums the result is the same
        y2 = torch.full_like(y, float("nan"))
        cw = w._c()
        st = qlora.lib().qlora_int8_linear_rows(ctypes.byref(cw), q.codes.data_ptr(), q.scale.data_ptr(), m, None,
                                                y2.data_ptr(), rows.DTYPES[dtype], None, 0, qlora._stream())
        assert st == 0 and torch.equal(y, y2)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear_backward(m, n, k, dtype):
    need_gpu()
    _, w = _weight(n, k, n + k)
    dy = rand((m, n), m + n, dtype)
    q = rows.quantize_rows(dy, w.scale)
    want = ref.int8_linear(codes_of(q), f64(q.scale), codes_of(w).T, None)
    got = int8.linear_bwd(w, dy)
    close16(got, want, np.abs(want), "dX")
    # and it is the gradient of the forward, to the rounding of dY to 8 bits:
    # each entry of dY scale is off by at most half a step, so dX by at most
    # half a step times the sum of the codes' magnitudes
    true = f64(dy) @ (codes_of(w) * f64(w.scale)[:, None])
    bound = 0.501 * f64(q.scale)[:, None] * np.abs(codes_of(w)).sum(0)[None, :]
    assert (np.abs(want - true) <= bound + 1e-6 * np.abs(true)).all()


@pytest.mark.parametrize("n,k", [(1, 1), (31, 100), (64, 128), (130, 257), (1000, 2500)])
def test_weight_layouts(n, k):
    """Codes from elsewhere come back as they were, and so does the transpose."""
    need_gpu()
    g = torch.Generator(device="cuda")
    g.manual_seed(n + k)
    codes = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int16).to(torch.int8)
    scale = torch.rand(n, generator=g, device="cuda") + 0.5
    w = int8.weight_from_codes(codes, scale, transposed=True)
    L = qlora.lib()
    assert w.codes.numel() == L.qlora_int8_weight_bytes(n, k) and w.codes_t.numel() == L.qlora_int8_weight_bytes(k, n)
    assert np.array_equal(codes_of(w), f64(codes))
    t = int8.Int8Weight(w.codes_t, torch.ones(k, device="cuda"), k, n)
    assert np.array_equal(codes_of(t), f64(codes).T)
    wide = torch.full((n, k + 13), 77, dtype=torch.int8, device="cuda")
    wide[:, 5:5 + k] = codes
    assert np.array_equal(codes_of(int8.weight_from_codes(wide[:, 5:5 + k], scale)), f64(codes))
    for dtype in (BF16, F16):
        v = f64(codes) * f64(scale)[:, None]
        close16(int8.dequant_weight(w, dtype=dtype), v, np.abs(v))


def test_largest_sums():
    """Every product at its largest magnitude (a weight's codes go to -128):
    the int32 sum stays exact up to the longest reduction, at either sign."""
    need_gpu()
    k = 132104
    codes = torch.full((3, k), 127, dtype=torch.int8, device="cuda")
    codes[1] = -128
    codes[2, ::2] = -128
    w = int8.weight_from_codes(codes, torch.ones(3, device="cuda"), transposed=True)
    for m in (1, 20, 70):
        x = torch.full((m, k), 1.0, dtype=BF16, device="cuda")
        x[m - 1] = -1.0
        y = int8.linear_fwd(w, x)
        want = np.tile([127.0 * k, -128.0 * k, -0.5 * k], (m, 1)) * np.where(np.arange(m) == m - 1, -1.0, 1.0)[:, None]
        close16(y, want, np.abs(want))
    dy = torch.ones((2, 3), dtype=BF16, device="cuda")
    close16(int8.linear_bwd(w, dy), np.tile(f64(codes).sum(0), (2, 1)), 3 * 128.0)


def test_large_offsets():
    """More than 2^31 elements in and out: the last rows are those of a call of
    their own."""
    need_gpu()
    m, k, n = 270000, 128, 8200
    _, w = _weight(n, k, 1)
    x = rand((m, k), 2)
    y = int8.linear_fwd(w, x)
    assert y.numel() > 2 ** 31
    for at in (0, m // 2, m - 100):
        assert torch.equal(y[at:at + 100], int8.linear_fwd(w, x[at:at + 100].contiguous()))
    q = rows.quantize_rows(y)
    v = rows.dequant_rows(q)
    dx = int8.linear_bwd(w, y)
    assert torch.equal(v[-100:], rows.dequant_rows(rows.quantize_rows(y[-100:])))
    assert torch.equal(dx[-100:], int8.linear_bwd(w, y[-100:]))


def test_odd_rows():
    """A token with a NaN or an infinity gives NaN outputs and leaves the
    others alone; a zero token gives the bias."""
    need_gpu()
    for m in (7, 40, 200):
        _, w = _weight(100, 300, 1)
        x, b = rand((m, 300), 2), rand((100,), 3)
        clean = int8.linear_fwd(w, x, b)
        x2 = x.clone()
        x2[1, 5], x2[4, 299], x2[m - 1] = float("nan"), float("-inf"), 0
        y = int8.linear_fwd(w, x2, b)
        assert torch.isnan(y[[1, 4]]).all() and torch.equal(y[m - 1], b)
        keep = [i for i in range(m) if i not in (1, 4, m - 1)]
        assert torch.equal(y[keep], clean[keep])


def test_empty():
    need_gpu()
    _, w = _weight(40, 64, 1)
    assert int8.linear_fwd(w, torch.empty((0, 64), dtype=BF16, device="cuda")).shape == (0, 40)
    assert int8.linear_bwd(w, torch.empty((0, 40), dtype=BF16, device="cuda")).shape == (0, 64)
    none = int8.quantize_weight(torch.empty((0, 64), device="cuda"), transposed=True)
    assert int8.linear_fwd(none, rand((3, 64), 1)).shape == (3, 0)
    assert (int8.linear_bwd(none, torch.empty((3, 0), dtype=BF16, device="cuda")) == 0).all()
    thin = int8.quantize_weight(torch.empty((40, 0), device="cuda"), transposed=True)
    b = rand((40,), 2)
    x = torch.empty((3, 0), dtype=BF16, device="cuda")
    assert (int8.linear_fwd(thin, x) == 0).all() and torch.equal(int8.linear_fwd(thin, x, b), b.expand(3, 40))
    assert int8.linear_bwd(thin, rand((3, 40), 1)).shape == (3, 0)


def test_autograd():
    need_gpu()
    W = rand((48, 200), 1, F32, 0.02)
    lin = int8.Int8Linear(W, rand((48,), 2), transposed=True)
    x = rand((2, 3, 200), 3).requires_grad_()
    y = lin(x)
    d = rand((2, 3, 48), 4)
    y.backward(d)
    assert torch.equal(x.grad.reshape(6, 200), int8.linear_bwd(lin.w, d.reshape(6, 48)))
    close16(lin.bias.grad, f64(d).reshape(6, 48).sum(0), np.abs(f64(d)).reshape(6, 48).sum(0))
    with torch.no_grad():
        assert torch.equal(lin(rows.quantize_rows(x.reshape(6, 200))), y.reshape(6, 48))


def test_merged_weight():
    """The way to serve a trained layer: merge the adapter, quantize to 8 bits."""
    need_gpu()
    W = rand((256, 512), 1, F32, 0.02)
    w4 = qlora.quantize(W)
    A, B = rand((8, 512), 2, BF16, 512 ** -0.5), rand((256, 8), 3, BF16, 0.01)
    merged = qlora.merge(w4, A, B, 8, 16.0)
    w8 = int8.quantize_weight(merged)
    want, scale = ref.quantize_rows(f64(merged))
    assert np.array_equal(codes_of(w8), want)
    x = rand((40, 512), 4)
    y4, _ = qlora.linear_fwd(w4, x, A, B, 8, 16.0)
    y8 = int8.linear_fwd(w8, x)
    # 8-bit rounding of both operands: half a step each, as independent errors
    err = np.linalg.norm(f64(y8) - f64(y4)) / np.linalg.norm(f64(y4))
    assert err < 0.03


def test_refusals():
    need_gpu()
    _, w = _weight(40, 64, 1)
    x = rand((4, 64), 2)
    with pytest.raises(ValueError, match="shape"):
        int8.linear_fwd(w, rand((4, 65), 2))
    with pytest.raises(ValueError, match="columns"):
        int8.linear_fwd(w, rows.quantize_rows(rand((4, 65), 2)))
    with pytest.raises(TypeError, match="X must be"):
        int8.linear_fwd(w, x.float())
    with pytest.raises(TypeError, match="bias"):
        int8.linear_fwd(w, x, rand((40,), 1, F16))
    with pytest.raises(ValueError, match="bias"):
        int8.linear_fwd(w, x, rand((41,), 1))
    with pytest.raises(ValueError, match="Y must be"):
        int8.linear_fwd(w, x, Y=torch.empty((4, 41), dtype=BF16, device="cuda"))
    with pytest.raises(RuntimeError, match="transposed codes"):
        int8.linear_bwd(int8.quantize_weight(rand((40, 64), 1, F32)), rand((4, 40), 1))
    with pytest.raises(RuntimeError, match="132104"):
        int8.quantize_weight(rand((1, 132105), 1, F32))
    with pytest.raises(ValueError, match="codes"):
        int8.linear_fwd(int8.Int8Weight(w.codes[:-1], w.scale, 40, 64), x)
    with pytest.raises(TypeError, match="codes must be"):
        int8.weight_from_codes(x, w.scale)
