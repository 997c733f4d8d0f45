"""The row-wise operators and the int8 product through the bounds-checked
build (libqlora_checked.so): the same bits as the normal build, and no access
outside a buffer.  Shapes: ragged ones and whole tiles of the few tokens'
kernels (tiles and splits: test_gpu_int8_plans.py), and rows of each width class
in small numbers (many rows: test_gpu_rows_many.py)."""

import pytest
import torch

from bit_nf4_quantized_double_amd import int8, qlora, rows
from rows_util import need_gpu, rand, strided

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _both(fn):
    torch.cuda.synchronize()
    ref = fn()
    torch.cuda.synchronize()
    with qlora.library(qlora.LIB_CHECKED_PATH):
        qlora.debug_oob_count(reset=True)
        got = fn()
        torch.cuda.synchronize()
        assert qlora.debug_oob_count(reset=True) == 0
    assert len(ref) == len(got)
    for i, (a, b) in enumerate(zip(ref, got)):
        ints = {2: torch.int16, 4: torch.int32}[a.element_size()]
        assert torch.equal(a.view(ints), b.view(ints)), i


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,k", [(1, 1), (3, 129), (17, 1000), (600, 333), (40, 2500), (5, 8192), (2, 16400), (2, 32800)])
def test_rows_in_bounds(m, k, dtype, apart):
    need_gpu()
    x, r, d, e = (rand((m, k), i, dtype) for i in range(4))
    if apart:
        x, r, d, e = (strided(t, 11, 3) for t in (x, r, d, e))
    g = rand((k,), 7, F32)

    def run():
        out = []
        for q in (rows.quantize_rows(x), rows.quantize_rows(x, g), rows.swiglu_int8(x, r)):
            out += [q.scale, rows.dequant_rows(q)]
        out += [rows.swiglu_fwd(x, r), *rows.swiglu_bwd(d, x, r)]
        if k <= rows.MAX_NORM_WIDTH:
            y, h, rstd = rows.rms_norm_fwd(x, g, 1e-5, r)
            q, h8 = rows.rms_norm_int8(x, g, 1e-5, r)
            out += [y, h, rstd, q.scale, rows.dequant_rows(q), h8, *rows.rms_norm_bwd(d, h, rstd, g, e)]
        return out

    _both(run)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 4096, 4096), (3, 130, 257), (16, 520, 2500), (17, 64, 100), (40, 33, 129),
                                   (64, 1000, 4096), (65, 100, 300), (130, 513, 640), (300, 2048, 1024),
                                   (512, 256, 8192), (1030, 300, 70)])
def test_product_in_bounds(m, n, k, dtype):
    need_gpu()
    W = rand((n, k), 1, F32, 0.02)
    x, dy, b = rand((m, k), 2, dtype), rand((m, n), 3, dtype), rand((n,), 4, dtype)

    def run():
        w = int8.quantize_weight(W, transposed=True)
        q = rows.quantize_rows(x)
        return [w.scale, int8.dequant_weight(w), int8.linear_fwd(w, x), int8.linear_fwd(w, q, b),
                int8.linear_bwd(w, dy)]

    _both(run)


def test_layouts_in_bounds():
    need_gpu()
    for n, k in ((1, 1), (33, 130), (257, 1000)):
        codes = torch.randint(-127, 128, (n, k), device="cuda", dtype=torch.int16).to(torch.int8)
        scale = torch.rand(n, device="cuda")

        def run():
            w = int8.weight_from_codes(codes, scale, transposed=True)
            t = int8.Int8Weight(w.codes_t, torch.ones(k, device="cuda"), k, n)
            return [int8.dequant_weight(w), int8.dequant_weight(t)]

        _both(run)
