"""The int8 product by every kernel and split: named ones at small ragged sizes,
and the plan's own at sizes where it takes tiles and splits, against the 64-bit
reference (bounds: rows_util).  The integer sum is exact, so every kernel and
split gives the same bits."""

import ctypes

import numpy as np
import pytest
import torch

import oracle.rows as ref
from bit_nf4_quantized_double_amd import int8, qlora, rows
from rows_util import close16, codes_of, f64, need_gpu, rand
from test_gpu_int8_bounds import _both

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
KERNELS = (16, 32, 64, 256)  # tokens of a workgroup: few tokens' kernels, tiles of 256 x 128
SPLITS = (1, 2, 3, 4, 8)
# ragged tokens and outputs; whole ones; reductions of 2, 4, 6, 10 and 16 chunks
# of 64, whose splits hold odd numbers of them, one or none
SHAPES = [(1, 1, 1), (17, 33, 100), (70, 130, 257), (256, 128, 128), (257, 129, 640), (300, 260, 1000), (513, 392, 129)]


def _named(w, q, dtype, tokens, splits, bias=None):
    y = torch.full((q.m, w.n_out), float("nan"), dtype=dtype, device="cuda")
    # sums that a split leaves unwritten would show
    ws = torch.full((splits * q.m * (-(-w.n_out // 8) * 8),), 0x55555555, dtype=torch.int32, device="cuda")
    cw = w._c()
    st = qlora.lib().qlora_debug_int8_linear_rows(ctypes.byref(cw), q.codes.data_ptr(), q.scale.data_ptr(), q.m,
                                                  None if bias is None else bias.data_ptr(), y.data_ptr(),
                                                  rows.DTYPES[dtype], tokens, splits, ws.data_ptr(),
                                                  4 * ws.numel(), qlora._stream())
    qlora._check(st, "qlora_debug_int8_linear_rows")
    return y


def _reference(w, q, at=slice(None), bias=None):
    b = None if bias is None else f64(bias)
    want = ref.int8_linear(codes_of(q)[at], f64(q.scale)[at], codes_of(w), f64(w.scale), b)
    return want, np.abs(want) + (0 if b is None else np.abs(b)[None, :])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_every_kernel_and_split(m, n, k, bias, dtype):
    need_gpu()
    w = int8.quantize_weight(rand((n, k), n + k, F32, 0.02))
    q = rows.quantize_rows(rand((m, k), m + k, dtype))
    b = rand((n,), 3, dtype) if bias else None
    want, mag = _reference(w, q, bias=b)
    first = None
    for tokens in KERNELS:
        for splits in SPLITS:
            y = _named(w, q, dtype, tokens, splits, b)
            if first is None:
                close16(y, want, mag, "Y")
                first = y
            assert torch.equal(y, first), (tokens, splits)
    assert torch.equal(int8.linear_fwd(w, q, b), first)


# ordinary prompts, for which the plan takes tiles, or splits the reduction
PLANNED = [(512, 4096, 11008, "tile", 4), (200, 14336, 4096, "tile", 2), (200, 4096, 14336, "tile", 8),
           (900, 6000, 300, "tile", 1), (401, 8100, 8197, "tile", 2), (70, 500, 28672, "few64", 8),
           (1500, 3001, 4100, "tile", 1)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,n,k,kernel,splits", PLANNED)
def test_planned_products(m, n, k, kernel, splits, dtype):
    """Through the calls of a user, with a bias and without, against the
    reference in some rows and another kernel in all."""
    need_gpu()
    assert int8.plan(qlora.QLORA_OP_FWD, m, n, k, 256) == {"kernel": kernel, "splits": splits, "quantizes_rows": False}
    w = int8.quantize_weight(rand((n, k), n + k, F32, 0.02))
    x, b = rand((m, k), m + k, dtype), rand((n,), 3, dtype)
    q = rows.quantize_rows(x)
    at = sorted({0, 1, 15, 16, 63, 64, m // 2, *range(m - 9, m)})
    for bias in (None, b):
        y = int8.linear_fwd(w, x, bias)
        want, mag = _reference(w, q, at, bias)
        close16(y[at], want, mag, "Y")
        assert torch.equal(y, int8.linear_fwd(w, q, bias))
        assert torch.equal(y, _named(w, q, dtype, 16, 1, bias))


# dX: reductions over the outputs
BACKWARD = [(512, 256, 4100, "tile", 1), (300, 700, 260, "few64", 1), (600, 1000, 4100, "tile", 1), (200, 14336, 4096, "tile", 8),
            (200, 4099, 14300, "tile", 2), (2049, 1025, 2051, "tile", 1)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,n,k,kernel,splits", BACKWARD)
def test_planned_backward(m, n, k, kernel, splits, dtype):
    need_gpu()
    plan = int8.plan(qlora.QLORA_OP_BWD, m, n, k, 256)
    assert (plan["kernel"], plan["splits"]) == (kernel, splits)
    w = int8.quantize_weight(rand((n, k), n + k, F32, 0.02), transposed=True)
    dy = rand((m, n), m + n, dtype)
    q = rows.quantize_rows(dy, w.scale)
    dx = int8.linear_bwd(w, dy)
    at = sorted({0, 1, 15, 16, 63, 64, m // 2, *range(m - 9, m)})
    want = ref.int8_linear(codes_of(q)[at], f64(q.scale)[at], codes_of(w).T, None)
    close16(dx[at], want, np.abs(want), "dX")


@pytest.mark.parametrize("tokens", KERNELS)
@pytest.mark.parametrize("splits", [1, 4])
def test_odd_rows(tokens, splits):
    """A token with a NaN or an infinity gives NaN outputs and leaves the
    others alone; a zero token gives the bias."""
    need_gpu()
    m, n, k = 290, 200, 700
    w = int8.quantize_weight(rand((n, k), 1, F32, 0.02))
    x, b = rand((m, k), 2), rand((n,), 3)
    clean = _named(w, rows.quantize_rows(x), BF16, tokens, splits, b)
    x[1, 5], x[100, k - 1], x[m - 1] = float("nan"), float("-inf"), 0
    y = _named(w, rows.quantize_rows(x), BF16, tokens, splits, b)
    assert torch.isnan(y[[1, 100]]).all() and torch.equal(y[m - 1], b)
    keep = [i for i in range(m) if i not in (1, 100, m - 1)]
    assert torch.equal(y[keep], clean[keep])


def test_largest_sums():
    """Every product at its largest magnitude, through tiles and splits."""
    need_gpu()
    k = 132104
    codes = torch.full((130, k), 127, dtype=torch.int8, device="cuda")
    codes[1] = -128
    codes[129, ::2] = -128
    w = int8.weight_from_codes(codes, torch.ones(130, device="cuda"))
    x = torch.full((300, k), 1.0, dtype=BF16, device="cuda")
    x[299] = -1.0
    q = rows.quantize_rows(x)
    want = np.full((300, 130), 127.0 * k)
    want[:, 1], want[:, 129] = -128.0 * k, -0.5 * k
    want[299] *= -1
    for splits in (1, 3, 8):
        close16(_named(w, q, BF16, 256, splits), want, np.abs(want))


@pytest.mark.parametrize("m,n,k", [(200, 4096, 14336), (400, 512, 1000), (70, 500, 28672)])
def test_product_in_a_graph(m, n, k):
    """Captured once, replayed on new inputs: every replay is the eager result,
    with eager work in between (tiles and few tokens' kernel, split 8 ways, and
    unsplit)."""
    need_gpu()
    w = int8.quantize_weight(rand((n, k), 1, F32, 0.02))
    x = rand((m, k), 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        int8.linear_fwd(w, x)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = int8.linear_fwd(w, x)
    for seed in (3, 4, 5):
        x.copy_(rand((m, k), seed))
        want = int8.linear_fwd(w, x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,n,k", SHAPES + [(515, 1030, 300)])
def test_every_kernel_in_bounds(m, n, k, dtype):
    need_gpu()
    W, x, b = rand((n, k), 1, F32, 0.02), rand((m, k), 2, dtype), rand((n,), 3, dtype)

    def run():
        w, q = int8.quantize_weight(W), rows.quantize_rows(x)
        return [_named(w, q, dtype, t, s, b) for t in KERNELS for s in (1, 2, 3, 8)]

    _both(run)


@pytest.mark.parametrize("m,n,k", [(512, 4096, 11008), (401, 8100, 8197), (900, 6000, 300)])
def test_planned_products_in_bounds(m, n, k):
    need_gpu()
    W, x, b = rand((n, k), 1, F32, 0.02), rand((m, k), 2), rand((n,), 3)

    def run():
        w = int8.quantize_weight(W)
        return [int8.linear_fwd(w, x), int8.linear_fwd(w, x, b)]

    _both(run)
