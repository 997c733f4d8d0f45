"""Host-side checks of the entry points of the row-wise operators and the int8
product (CPU only): sizes, and arguments refused before anything is enqueued.
Device pointers are fake and never dereferenced."""

import ctypes
import os

import pytest

from bit_nf4_quantized_double_amd import int8, qlora, rows

INVALID, SHAPE, ALIGN, WORKSPACE = -1, -2, -3, -4
P = 0x10000        # aligned
P2 = 0x10002       # aligned to two bytes
P1 = 0x10001
BF16, F16, F32 = 0, 1, 2
BIG = 1 << 31


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(qlora.LIB_PATH):
        from bit_nf4_quantized_double_amd import build
        build.build(verbose=False)
    return qlora.lib()


def test_layout_sizes(L):
    for m, k in ((0, 5), (1, 1), (16, 128), (17, 129), (1000, 2500)):
        assert L.qlora_int8_rows_bytes(m, k) == -(-m // 16) * 16 * (-(-k // 128) * 128)
        assert L.qlora_int8_weight_bytes(m, k) == int8.weight_bytes(m, k)
    assert L.qlora_int8_rows_bytes(-1, 5) == 0 and L.qlora_int8_weight_bytes(5, -1) == 0


def test_workspace_sizes(L):
    # few enough tokens are quantized inside the product
    assert L.qlora_int8_workspace_bytes(qlora.QLORA_OP_FWD, 1, 4096, 4096) == 0
    for m, n, k in ((17, 130, 2500), (2048, 4096, 11008)):
        fwd = L.qlora_int8_workspace_bytes(qlora.QLORA_OP_FWD, m, n, k)
        bwd = L.qlora_int8_workspace_bytes(qlora.QLORA_OP_BWD, m, n, k)
        assert fwd >= L.qlora_int8_rows_bytes(m, k) + 4 * m + L.qlora_int8_rows_workspace_bytes(m, n, k)
        assert bwd >= L.qlora_int8_rows_bytes(m, n) + 4 * m + L.qlora_int8_rows_workspace_bytes(m, k, n)
    assert L.qlora_int8_workspace_bytes(7, 1, 1, 1) == 0 and L.qlora_int8_workspace_bytes(1, 0, 1, 1) == 0
    assert L.qlora_rms_norm_bwd_workspace_bytes(5, 64) >= 64 * 4  # a row of partial sums at least
    assert L.qlora_rms_norm_bwd_workspace_bytes(0, 64) == 0


def _w(n=64, k=64, codes=P, codes_t=P, scale=P):
    return ctypes.byref(int8._CInt8Weight(n, k, codes, codes_t, scale))


def test_weight_refusals(L):
    q = L.qlora_int8_quantize_weight
    assert q(None, F32, 64, 64, 64, P, P, 0) == INVALID
    assert q(P, 3, 64, 64, 64, P, P, 0) == INVALID
    assert q(P, F32, 63, 64, 64, P, P, 0) == INVALID
    assert q(P, F32, 64, -1, 64, P, P, 0) == INVALID
    assert q(P2, F32, 64, 64, 64, P, P, 0) == ALIGN
    assert q(P, F32, 64, 64, 64, P2, P, 0) == ALIGN
    assert q(P, F32, 64, 64, 64, None, P, 0) == INVALID
    assert q(P, F32, 132105, 64, 132105, P, P, 0) == SHAPE
    assert q(P, F32, 64, BIG, 64, P, P, 0) == SHAPE
    assert q(P, F32, 1 << 41, 64, 64, P, P, 0) == SHAPE
    assert q(None, F32, 64, 0, 64, None, None, 0) == 0
    p = L.qlora_int8_pack_weight
    assert p(None, 64, 64, 64, P, 0) == INVALID and p(P, 63, 64, 64, P, 0) == INVALID
    assert p(P, 64, 64, 64, P1, 0) == ALIGN and p(P, 1 << 41, 64, 64, P, 0) == SHAPE
    assert p(P, 64, 64, 132105, P, 0) == SHAPE and p(None, 64, 0, 64, None, 0) == 0
    assert L.qlora_int8_transpose_weight(None, P, 0) == INVALID
    assert L.qlora_int8_transpose_weight(_w(), None, 0) == INVALID
    assert L.qlora_int8_transpose_weight(_w(n=132105), P, 0) == SHAPE
    assert L.qlora_int8_dequant_weight(_w(), P, F32, 0) == INVALID
    assert L.qlora_int8_dequant_weight(_w(scale=None), P, BF16, 0) == INVALID
    assert L.qlora_int8_dequant_weight(_w(), P2, BF16, 0) == ALIGN


def test_row_refusals(L):
    q = L.qlora_int8_quantize_rows
    assert q(None, BF16, 64, 4, 64, None, P, P, 0) == INVALID
    assert q(P1, BF16, 64, 4, 64, None, P, P, 0) == ALIGN
    assert q(P, BF16, 64, 4, 64, P2, P, P, 0) == ALIGN
    assert q(P, BF16, 64, 4, 64, None, None, P, 0) == INVALID
    assert q(P, BF16, 132105, 4, 132105, None, P, P, 0) == SHAPE
    assert q(P, BF16, 64, -4, 64, None, P, P, 0) == INVALID
    assert q(None, BF16, 64, 0, 64, None, None, None, 0) == 0
    d = L.qlora_int8_dequant_rows
    assert d(None, P, 4, 64, P, BF16, 0) == INVALID and d(P, P, 4, 64, P2, BF16, 0) == ALIGN
    assert d(P, P, 4, 64, P, F32, 0) == INVALID and d(None, None, 0, 64, None, BF16, 0) == 0


def test_product_refusals(L):
    f, r, b = L.qlora_int8_linear_fwd, L.qlora_int8_linear_rows, L.qlora_int8_linear_bwd
    need = L.qlora_int8_workspace_bytes(1, 40, 64, 64)
    assert f(None, P, 64, 40, None, P, BF16, P, need, 0) == INVALID
    assert f(_w(), None, 64, 40, None, P, BF16, P, need, 0) == INVALID
    assert f(_w(), P, 64, 40, None, P, F32, P, need, 0) == INVALID
    assert f(_w(), P, 64, 40, P2, P, BF16, P, need, 0) == ALIGN
    assert f(_w(), P, 64, 40, None, P2, BF16, P, need, 0) == ALIGN
    assert f(_w(), P, 64, 40, None, P, BF16, None, 0, 0) == WORKSPACE
    assert f(_w(), P, 64, 40, None, P, BF16, P, 64, 0) == WORKSPACE
    assert f(_w(), P, 64, 40, None, P, BF16, P2, need, 0) == ALIGN
    assert f(_w(), P, 64, BIG, None, P, BF16, P, need, 0) == SHAPE
    assert f(_w(), None, 64, 0, None, None, BF16, None, 0, 0) == 0
    assert r(_w(), None, P, 40, None, P, BF16, None, 0, 0) == INVALID
    assert r(_w(), P, P, 40, None, P, BF16, P2, 1, 0) == ALIGN
    assert b(_w(codes_t=None), P, 64, 40, P, BF16, P, need, 0) == INVALID
    assert b"transposed" in L.qlora_last_error()
    assert b(_w(n=132105), P, 132105, 40, P, BF16, P, 1 << 30, 0) == SHAPE
    assert b(_w(), P, 64, 40, P, BF16, None, 0, 0) == WORKSPACE


def test_norm_refusals(L):
    f, i, b = L.qlora_rms_norm_fwd, L.qlora_rms_norm_int8, L.qlora_rms_norm_bwd
    for fn in (f, i):
        assert fn(None, 64, None, 0, P, BF16, 4, 64, 1e-5, P, P, P, BF16, 0) == INVALID
        assert fn(P, 64, None, 0, None, BF16, 4, 64, 1e-5, P, P, P, BF16, 0) == INVALID
        assert fn(P, 64, None, 0, P, F16, 4, 64, 1e-5, P, P, P, BF16, 0) == INVALID
        assert fn(P, 64, None, 0, P, BF16, 4, 64, 0.0, P, P, P, BF16, 0) == INVALID
        assert fn(P, 64, None, 0, P, BF16, 4, 64, float("inf"), P, P, P, BF16, 0) == INVALID
        assert fn(P, 64, P1, 64, P, BF16, 4, 64, 1e-5, P, P, P, BF16, 0) == ALIGN
        assert fn(P, 64, P, 63, P, BF16, 4, 64, 1e-5, P, P, P, BF16, 0) == INVALID
        assert fn(P, 64, P, 64, P, BF16, 4, 64, 1e-5, None, P, P, BF16, 0) == INVALID
        assert fn(P, 40000, None, 0, P, BF16, 4, 32769, 1e-5, P, P, P, BF16, 0) == SHAPE
        assert fn(None, 64, None, 0, P, BF16, 0, 64, 1e-5, None, None, None, BF16, 0) == 0
    need = L.qlora_rms_norm_bwd_workspace_bytes(4, 64)
    assert b(P, 64, P, 64, P, P, BF16, None, 0, 4, 64, P, P, BF16, None, 0, 0) == WORKSPACE
    assert b(P, 64, P, 64, P, P, BF16, None, 0, 4, 64, P, P, BF16, P, need - 1, 0) == WORKSPACE
    assert b(P, 64, P, 64, None, P, BF16, None, 0, 4, 64, P, P, BF16, P, need, 0) == INVALID
    assert b(P, 64, P, 64, P, P, BF16, None, 0, 4, 64, P, None, BF16, P, need, 0) == INVALID
    assert b(P, 64, P, 63, P, P, BF16, None, 0, 4, 64, P, P, BF16, P, need, 0) == INVALID


def test_swiglu_refusals(L):
    f, i, b = L.qlora_swiglu_fwd, L.qlora_swiglu_int8, L.qlora_swiglu_bwd
    assert f(None, 64, P, 64, 4, 64, P, BF16, 0) == INVALID and f(P, 64, P1, 64, 4, 64, P, BF16, 0) == ALIGN
    assert f(P, 64, P, 64, 4, 64, None, BF16, 0) == INVALID and f(P, 64, P, 64, 4, 64, P, F32, 0) == INVALID
    assert f(P, 1 << 20, P, 1 << 20, BIG - 1, 1 << 20, P, BF16, 0) == SHAPE
    assert i(P, 132105, P, 132105, 4, 132105, P, P, BF16, 0) == SHAPE
    assert i(P, 64, P, 64, 4, 64, P, None, BF16, 0) == INVALID
    assert b(None, 64, P, 64, P, 64, 4, 64, P, P, BF16, 0) == INVALID
    assert b(P, 64, P, 64, P, 64, 4, 64, P, None, BF16, 0) == INVALID
    assert f(None, 64, None, 64, 0, 64, None, BF16, 0) == 0


def test_cpu_tensors_are_refused():
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: rows.quantize_rows(x), lambda: rows.swiglu_fwd(x, x),
                 lambda: rows.rms_norm_fwd(x, x[0], 1e-5), lambda: int8.quantize_weight(x)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_norm_of_no_values_writes_nothing_without_a_place(L):
    """K = 0: nothing to write but rstd or the scales, and not even those when
    the caller has no place for them."""
    assert L.qlora_rms_norm_fwd(None, 0, None, 0, None, BF16, 4, 0, 1e-5, None, None, None, BF16, 0) == 0
    assert L.qlora_rms_norm_int8(None, 0, None, 0, None, BF16, 4, 0, 1e-5, None, None, None, BF16, 0) == 0
    assert L.qlora_rms_norm_fwd(None, 0, None, 0, None, BF16, 4, 0, 1e-5, None, None, P2, BF16, 0) == ALIGN
    assert L.qlora_rms_norm_int8(None, 0, None, 0, None, BF16, 4, 0, 1e-5, None, None, P2, BF16, 0) == ALIGN
