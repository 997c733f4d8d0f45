"""The int8 product's plan and the entry point that names a kernel, as far as
they run on the host (CPU only; device pointers are fake)."""

import ctypes
import os

import pytest

from bit_nf4_quantized_double_amd import int8, qlora

INVALID, SHAPE, ALIGN, WORKSPACE = -1, -2, -3, -4
P, P2, BF16 = 0x10000, 0x10002, 0
FWD, BWD = qlora.QLORA_OP_FWD, qlora.QLORA_OP_BWD


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(qlora.LIB_PATH):
        from bit_nf4_quantized_double_amd import build
        build.build(verbose=False)
    return qlora.lib()


def test_plan(L):
    assert int8.plan(FWD, 1, 4096, 4096, 256) == {"kernel": "few16", "splits": 1, "quantizes_rows": True}
    assert int8.plan(FWD, 16, 8192, 28672, 256)["quantizes_rows"] is False
    assert int8.plan(FWD, 8192, 14336, 4096, 256) == {"kernel": "tile", "splits": 1, "quantizes_rows": False}
    # dX of a layer is the product of its transpose
    for m, n, k in ((1, 300, 5000), (200, 4096, 14336), (2048, 4096, 11008)):
        assert int8.plan(BWD, m, n, k, 256) == int8.plan(FWD, m, k, n, 256)
    # the workspace has room for the sums of the splits
    for m, n, k in ((200, 4096, 14336), (70, 500, 28672), (512, 4096, 11008)):
        p = int8.plan(FWD, m, n, k)
        assert L.qlora_int8_rows_workspace_bytes(m, n, k) == (p["splits"] * m * -(-n // 8) * 8 * 4 if p["splits"] > 1 else 0)


def test_plan_refusals(L):
    out = (ctypes.c_int64 * 3)()
    assert L.qlora_int8_plan(FWD, 1, 1, 1, 0, None) == INVALID
    assert L.qlora_int8_plan(7, 1, 1, 1, 0, out) == INVALID
    assert L.qlora_int8_plan(FWD, -1, 1, 1, 0, out) == INVALID
    assert L.qlora_int8_plan(FWD, 1, 1 << 31, 1, 0, out) == SHAPE


def test_named_kernel_refusals(L):
    w = ctypes.byref(int8._CInt8Weight(64, 64, P, None, P))
    f = L.qlora_debug_int8_linear_rows
    need = 2 * 40 * 64 * 4
    for tokens, splits in ((0, 1), (48, 1), (128, 1), (64, 0), (64, -1), (256, 65)):
        assert f(w, P, P, 40, None, P, BF16, tokens, splits, P, 1 << 30, 0) == INVALID
    assert f(w, P, P, 40, None, P, BF16, 256, 2, None, 0, 0) == WORKSPACE
    assert f(w, P, P, 40, None, P, BF16, 256, 2, P, need - 1, 0) == WORKSPACE
    assert f(w, P, P, 40, None, P, BF16, 256, 2, P2, need, 0) == ALIGN
    assert f(None, P, P, 40, None, P, BF16, 256, 1, None, 0, 0) == INVALID
    assert f(w, None, P, 40, None, P, BF16, 256, 1, None, 0, 0) == INVALID
    assert f(w, P, P, 40, P2, P, BF16, 256, 1, None, 0, 0) == ALIGN
    assert f(w, None, None, 0, None, None, BF16, 256, 1, None, 0, 0) == 0
