"""The row-wise operators with many rows, where several rows share a wave and
the norm's backward takes several turns, against the 64-bit reference (bounds:
rows_util)."""

import numpy as np
import pytest
import torch

import oracle.rows as ref
from bit_nf4_quantized_double_amd import rows
from rows_util import E32, close16, codes_of, f64, need_gpu, rand, strided
from test_gpu_int8_bounds import _both

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5

# From 1024 rows on (four for each of 256 compute units) 8-bit rows share waves.
# Rows that fill no group of four; widths at both ends of each number of threads
# and pieces a row has there, and ragged ones
WIDTHS = [16, 1000, 1024, 1025, 2048, 2500, 4096, 4100, 8192, 8200, 12288, 12300, 16384]
WIDER = [16390, 32768, 32800]  # in registers for the quantizer and SwiGLU; read twice


def _rows_of(k):
    return 1027 if k > 4096 else 1030


def _some(m):
    """Rows compared with the reference: of every place in a group, and the ends."""
    return sorted({*range(0, m, 13), *range(m - 9, m)})


def _fewer(call, m):
    """The same rows in calls of few enough that each has a wave of its own."""
    step = -(-m // 3)
    return [call(slice(i, i + step)) for i in range(0, m, step)]


def _codes_match(q, parts, exact_scale):
    assert np.array_equal(codes_of(q), np.concatenate([codes_of(p) for p in parts]))
    scale = np.concatenate([f64(p.scale) for p in parts])
    if exact_scale:
        assert np.array_equal(f64(q.scale), scale)
    else:  # the sums of squares are added up in another order
        np.testing.assert_allclose(f64(q.scale), scale, rtol=E32)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("k", WIDTHS + WIDER)
def test_quantize_rows(k, dtype):
    need_gpu()
    m = _rows_of(k)
    x = rand((m, k), m * 7 + k, dtype)
    q = rows.quantize_rows(x)
    at = _some(m)
    want, scale = ref.quantize_rows(f64(x[at]))
    got = codes_of(q)[at]
    np.testing.assert_allclose(f64(q.scale)[at], scale, rtol=2.0 ** -22)
    if dtype != F32:  # 127 x is exact in fp32, and so are the codes
        assert np.array_equal(got, want)
    else:
        assert (np.abs(got - f64(x[at]) / scale[:, None]) <= 0.5 + 127 * 2.0 ** -22).all()
    _codes_match(q, _fewer(lambda s: rows.quantize_rows(x[s]), m), True)


@pytest.mark.parametrize("k", [1000, 4100, 12300])
def test_quantize_rows_column_scale_and_strides(k):
    need_gpu()
    m = _rows_of(k)
    x, c = rand((m, k), 1), rand((k,), 2, F32, 0.01)
    at = _some(m)
    q = rows.quantize_rows(x, c)
    values = f64(x[at]) * f64(c)
    _, scale = ref.quantize_rows(values)
    np.testing.assert_allclose(f64(q.scale)[at], scale, rtol=2.0 ** -22 + 2.0 ** -24)
    assert (np.abs(codes_of(q)[at] - values / scale[:, None]) <= 0.5 + 127 * (2.0 ** -23 + 2.0 ** -22)).all()
    apart = rows.quantize_rows(strided(x, 11, 3), c)
    assert np.array_equal(codes_of(q), codes_of(apart)) and torch.equal(q.scale, apart.scale)


def test_quantize_rows_with_odd_ones():
    """A row with an infinity or a NaN is NaN and leaves its neighbours alone."""
    need_gpu()
    for k in (1000, 2500, 8200, 12300, 20000):
        x = rand((1027, k), k)
        clean = rows.quantize_rows(x)
        x[5, 0], x[6, k - 1], x[1026, k // 2], x[9] = float("nan"), float("inf"), float("-inf"), 0
        q = rows.quantize_rows(x)
        bad = [5, 6, 1026]
        assert np.isnan(f64(q.scale)[bad]).all() and (codes_of(q)[bad + [9]] == 0).all()
        keep = np.setdiff1d(np.arange(1027), bad + [9])
        assert np.array_equal(codes_of(q)[keep], codes_of(clean)[keep])
        assert np.array_equal(f64(q.scale)[keep], f64(clean.scale)[keep])


@pytest.mark.parametrize("dtype,gdtype", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("k", WIDTHS + WIDER[:2])
def test_rms_norm(k, residual, dtype, gdtype):
    need_gpu()
    m = _rows_of(k)
    x, g = rand((m, k), m + k, dtype), (1 + 0.1 * rand((k,), 5, F32)).to(gdtype)
    r = rand((m, k), m + k + 1, dtype) if residual else None
    y, h, rstd = rows.rms_norm_fwd(x, g, EPS, r)
    q, h8 = rows.rms_norm_int8(x, g, EPS, r)
    at = _some(m)
    if residual:
        close16(h[at], f64(x[at]) + f64(r[at]), np.abs(f64(x[at])) + np.abs(f64(r[at])), "h")
        assert torch.equal(h, h8)
    want, rs = ref.rms_norm_fwd(f64(h[at]), f64(g), EPS)
    np.testing.assert_allclose(f64(rstd)[at], rs, rtol=E32)
    close16(y[at], want, np.abs(want), "y")
    codes, (exact, scale) = codes_of(q), ref.quantize_rows(want)
    np.testing.assert_allclose(f64(q.scale)[at], scale, rtol=E32 + 2.0 ** -22)
    assert (np.abs(codes[at] - want / scale[:, None]) <= 0.5 + 127 * (2 * E32 + 2.0 ** -22)).all()
    if dtype == gdtype == BF16:
        # the codes do not depend on rstd, and 127 h gamma is exact in fp32 (7 + 8 + 8 bits): so are they, in all rows
        v = h.double() * g.double()
        assert np.array_equal(codes, f64(torch.round(127 * v / v.abs().amax(1, keepdim=True))))
    _codes_match(q, _fewer(lambda s: rows.rms_norm_int8(x[s], g, EPS, None if r is None else r[s])[0], m), False)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("k", WIDTHS + WIDER)
def test_swiglu(k, dtype):
    need_gpu()
    m = _rows_of(k)
    both = torch.cat([rand((m, k), 1, dtype, 3.0), rand((m, k), 2, dtype)], dim=1)
    g, u = both[:, :k], both[:, k:]
    q = rows.swiglu_int8(g, u)
    at = _some(m)
    G = f64(g[at])
    want = ref.swiglu_fwd(G, f64(u[at]))
    _, scale = ref.quantize_rows(want)
    slack = E32 * (1 + np.abs(G).max())
    np.testing.assert_allclose(f64(q.scale)[at], scale, rtol=slack)
    assert (np.abs(codes_of(q)[at] - want / scale[:, None]) <= 0.5 + 127 * 2 * slack).all()
    _codes_match(q, _fewer(lambda s: rows.swiglu_int8(g[s], u[s]), m), True)


# (rows, width) of the norm's backward: 256 workgroups that take two, three or
# more turns each, at every number of threads a row can have; the last turns
# partly filled; two pieces a thread (16400)
TURNS = [(9000, 8), (9000, 640), (5000, 1500), (2100, 2500), (1100, 4096), (1300, 8000), (700, 8195), (600, 16384), (600, 16400)]


@pytest.mark.parametrize("dtype,gdtype", [(BF16, BF16), (F16, F32), (BF16, F32)])
@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("m,k", TURNS)
def test_rms_norm_backward(m, k, stream, dtype, gdtype):
    need_gpu()
    x, g, dy = rand((m, k), m + k, dtype), (1 + 0.1 * rand((k,), 5, F32)).to(gdtype), rand((m, k), 3, dtype)
    dh = rand((m, k), 4, dtype) if stream else None
    _, h, rstd = rows.rms_norm_fwd(x, g, EPS)
    dx, dgamma = rows.rms_norm_bwd(dy, h, rstd, g, dh)
    want, wg = ref.rms_norm_bwd(f64(dy), f64(h), f64(g), EPS, None if dh is None else f64(dh))
    hat = np.abs(f64(h)) * f64(rstd)[:, None]
    gg = np.abs(f64(dy) * f64(g))
    mag = f64(rstd)[:, None] * (gg + hat * (gg * hat).mean(1, keepdims=True))
    close16(dx, want, mag + (0 if dh is None else np.abs(f64(dh))), "dx")
    # a sum over m rows, in groups and then over the groups
    bound = (E32 + m * 2.0 ** -24) * (np.abs(f64(dy)) * hat).sum(0)
    assert (np.abs(f64(dgamma) - wg) <= bound).all()
    again = rows.rms_norm_bwd(dy, h, rstd, g, dh)
    assert torch.equal(dx, again[0]) and torch.equal(dgamma, again[1])
    # in the buffers of its inputs: a later turn's rows are read before an earlier one's are written
    dy2 = dy.clone()
    got = rows.rms_norm_bwd(dy2, h, rstd, g, dh, dX=dy2)
    assert torch.equal(dy2, dx) and torch.equal(got[1], dgamma)
    if dh is not None:
        dh2 = dh.clone()
        got = rows.rms_norm_bwd(dy, h, rstd, g, dh2, dX=dh2)
        assert torch.equal(dh2, dx) and torch.equal(got[1], dgamma)


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("m,k", [(1027, 16), (1027, 1000), (1027, 2500), (1027, 4100), (1027, 8200), (1027, 12300),
                                 (1027, 16384), (1027, 20001), (1027, 32800), (9000, 8), (5000, 1500), (600, 16400)])
def test_in_bounds(m, k, apart):
    need_gpu()
    x, r, d, e = (rand((m, k), i) for i in range(4))
    if apart:
        x, r, d, e = (strided(t, 11, 3) for t in (x, r, d, e))

    def run():
        out = []
        for g in (rand((k,), 7, F32), rand((k,), 7)):
            if k <= rows.MAX_NORM_WIDTH:
                _, h, rstd = rows.rms_norm_fwd(x, g, EPS, r)
                q, _ = rows.rms_norm_int8(x, g, EPS, r)
                out += [q.scale, rows.dequant_rows(q), *rows.rms_norm_bwd(d, h, rstd, g, e)]
        for q in (rows.quantize_rows(x), rows.swiglu_int8(x, r)):
            out += [q.scale, rows.dequant_rows(q)]
        return out

    _both(run)
