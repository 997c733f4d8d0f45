"""RMS norm, SwiGLU and the row quantizer on the GPU against the 64-bit
reference (bounds: rows_util)."""

import numpy as np
import pytest
import torch

import oracle.rows as ref
from bit_nf4_quantized_double_amd import int8, qlora, rows
from rows_util import E32, close16, codes_of, f64, need_gpu, rand, strided

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5

# (rows, width): one row; one value; widths that are no multiple of 8, 16 or
# 128; each number of threads a row can have, and its edge; more rows than
# compute units (several rows a workgroup)
SHAPES = [(1, 1), (3, 7), (1, 64), (17, 100), (5, 128), (300, 333), (16, 1000), (33, 1024), (1030, 1040), (7, 2048),
          (600, 2500), (1, 4096), (130, 4100), (9, 8192), (2, 8208), (3, 16384), (2, 20001)]
LONG = [(2, 32768), (2, 32784), (3, 50001)]  # rows held in registers, and read twice


def quantized(values: np.ndarray, q, slack: float, exact: bool):
    """Codes and scales of quantized rows.  `slack`: the relative error of the
    values the kernel quantized (0 for inputs that are exact in fp32)."""
    want, scale = ref.quantize_rows(values)
    got = codes_of(q)
    np.testing.assert_allclose(f64(q.scale), scale, rtol=slack + 2.0 ** -22)
    if exact:
        assert np.array_equal(got, want)
        return
    # a code is the nearest integer of a quotient that is off by at most the
    # values' and the amax's error and two roundings
    quotient = values / scale[:, None]
    assert (np.abs(got - quotient) <= 0.5 + 127 * (2 * slack + 2.0 ** -22)).all()
    assert np.abs(got).max(initial=0) <= 127


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("m,k", SHAPES + LONG)
def test_quantize_rows(m, k, dtype):
    need_gpu()
    x = rand((m, k), m * 7 + k, dtype)
    q = rows.quantize_rows(x)
    assert q.codes.numel() == qlora.lib().qlora_int8_rows_bytes(m, k)
    quantized(f64(x), q, 0.0, exact=dtype != F32)


@pytest.mark.parametrize("m,k", [(1, 1), (5, 100), (40, 2500), (2, 40000)])
def test_quantize_rows_column_scale(m, k):
    need_gpu()
    x, c = rand((m, k), 1), rand((k,), 2, F32, 0.01)
    quantized(f64(x) * f64(c), rows.quantize_rows(x, c), 2.0 ** -24, exact=False)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_quantize_exact_ties(dtype):
    """Half the amax is 63.5: ties go to the even code, at every exponent and
    for every odd amax."""
    need_gpu()
    amax = torch.arange(129, 256, 2, dtype=torch.float64)
    e = torch.arange(-10, 8, dtype=torch.float64)
    a = (amax[:, None] * 2.0 ** e[None, :]).reshape(-1, 1) / 128
    x = torch.cat([a, -a / 2, a / 2, a / 4, a * 0], dim=1).to(dtype).cuda()
    quantized(f64(x), rows.quantize_rows(x), 0.0, exact=True)


@pytest.mark.parametrize("k", [5, 300, 40000])
def test_quantize_extremes(k):
    """Zero rows, tiny and huge rows, and rows with infinities or NaN."""
    need_gpu()
    x = rand((8, k), 3, F32)
    x[0] = 0
    x[1] *= 1e-36  # below the floor on amax
    x[2] = x[2] / x[2].abs().max() * 3.4e38  # 127 x overflows fp32
    x[3, k // 2] = float("inf")
    x[4, 0] = float("-inf")
    x[5, k - 1] = float("nan")
    x[6] = float("nan")
    x[7] = 1e-45
    q = rows.quantize_rows(x)
    s = f64(q.scale)
    assert np.isnan(s[3:7]).all() and np.isfinite(s[[0, 1, 2, 7]]).all()
    codes = codes_of(q)
    assert (codes[3:7] == 0).all() and (codes[0] == 0).all() and (codes[7] == 0).all()
    live = f64(x)[[0, 1, 2, 7]]
    want, scale = ref.quantize_rows(live)
    np.testing.assert_allclose(s[[0, 1, 2, 7]], scale, rtol=2.0 ** -22)
    assert (np.abs(codes[[0, 1, 2, 7]] - live / scale[:, None]) <= 0.5 + 127 * 2.0 ** -22).all()
    v = f64(rows.dequant_rows(q))
    assert np.isnan(v[3:7]).all() and (v[0] == 0).all()


@pytest.mark.parametrize("pad,offset", [(8, 8), (16, 0), (3, 1), (1, 0)])
@pytest.mark.parametrize("m,k", [(5, 96), (20, 1000)])
def test_strided_inputs(m, k, pad, offset):
    """Slices of wider matrices give the bits of their contiguous copies."""
    need_gpu()
    x, r, d, e = (rand((m, k), i) for i in range(4))
    g = rand((k,), 9)
    xs, rs_, ds, es = (strided(t, pad, offset) for t in (x, r, d, e))
    q, qs = rows.quantize_rows(x), rows.quantize_rows(xs)
    assert np.array_equal(codes_of(q), codes_of(qs)) and torch.equal(q.scale, qs.scale)
    for a, b in zip(rows.rms_norm_fwd(x, g, EPS, r), rows.rms_norm_fwd(xs, g, EPS, rs_)):
        assert torch.equal(a, b)
    y, h, rstd = rows.rms_norm_fwd(x, g, EPS, r)
    for a, b in zip(rows.rms_norm_bwd(d, h, rstd, g, e), rows.rms_norm_bwd(ds, strided(h, pad, offset), rstd, g, es)):
        assert torch.equal(a, b)
    assert torch.equal(rows.swiglu_fwd(x, r), rows.swiglu_fwd(xs, rs_))
    for a, b in zip(rows.swiglu_bwd(d, x, r), rows.swiglu_bwd(ds, xs, rs_)):
        assert torch.equal(a, b)
    q, qs = rows.swiglu_int8(x, r), rows.swiglu_int8(xs, rs_)
    assert np.array_equal(codes_of(q), codes_of(qs)) and torch.equal(q.scale, qs.scale)


def _hidden(x, r, dtype):
    """The stored hidden state and its bound: exact sum, rounded to the type."""
    h = f64(x) + f64(r)
    return torch.from_numpy(h).to(dtype), h


@pytest.mark.parametrize("dtype,gdtype", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("m,k", SHAPES + LONG[:1])
def test_rms_norm(m, k, residual, dtype, gdtype):
    need_gpu()
    x, g = rand((m, k), m + k, dtype), (1 + 0.1 * rand((k,), 5, F32)).to(gdtype)
    r = rand((m, k), m + k + 1, dtype) if residual else None
    y, h, rstd = rows.rms_norm_fwd(x, g, EPS, r)
    q, h8 = rows.rms_norm_int8(x, g, EPS, r)
    if residual:
        exact = f64(x) + f64(r)
        close16(h, exact, np.abs(f64(x)) + np.abs(f64(r)), "h")
        assert torch.equal(h, h8)
    else:
        assert h is x and h8 is x
    want, rs = ref.rms_norm_fwd(f64(h), f64(g), EPS)
    np.testing.assert_allclose(f64(rstd), rs, rtol=E32)
    close16(y, want, np.abs(want), "y")
    quantized(want, q, E32, exact=False)


@pytest.mark.parametrize("dtype,gdtype", [(BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("m,k", SHAPES + LONG[:1])
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


@pytest.mark.parametrize("m,k", [(1, 640), (3, 640), (5, 2048), (3, 8)])
def test_rms_norm_backward_last_row_infinite(m, k):
    """An infinite dY in the last row reaches dgamma as that infinity, also
    where its workgroup has places for rows past it."""
    need_gpu()
    h, g, dy = rand((m, k), 1).abs() + 1, rand((k,), 2), rand((m, k), 3)
    _, _, rstd = rows.rms_norm_fwd(h, g, EPS)
    _, wg = ref.rms_norm_bwd(f64(dy), f64(h), f64(g), EPS)
    dy[m - 1, 5] = float("inf")
    dg = f64(rows.rms_norm_bwd(dy, h, rstd, g)[1])
    assert dg[5] == np.inf
    rest = np.arange(k) != 5
    bound = (E32 + m * 2.0 ** -24) * (np.abs(f64(dy)) * f64(h) * f64(rstd)[:, None]).sum(0)
    assert (np.abs(dg - wg)[rest] <= bound[rest]).all()


@pytest.mark.parametrize("m,k", [(1, 7), (16, 645), (33, 640), (2, 8195), (1, 16384), (1, 16400)])
def test_rms_norm_backward_few_rows(m, k):
    """Few rows, where one workgroup writes dgamma itself, or its sum for a
    second kernel: nothing before or past dgamma is written."""
    need_gpu()
    x, g, dy = rand((m, k), 1), rand((k,), 2), rand((m, k), 3)
    _, h, rstd = rows.rms_norm_fwd(x, g, EPS)
    got = []
    for off in (0, 4):
        buf = torch.full((k + 32,), -7.0, device="cuda")
        rows.rms_norm_bwd(dy, h, rstd, g, dgamma=buf[off : off + k])
        assert (buf[:off] == -7).all() and (buf[off + k :] == -7).all()
        got.append(f64(buf[off : off + k]))
    _, wg = ref.rms_norm_bwd(f64(dy), f64(h), f64(g), EPS)
    bound = (E32 + m * 2.0 ** -24) * (np.abs(f64(dy) * f64(h)) * f64(rstd)[:, None]).sum(0)
    for dg in got:
        assert (np.abs(dg - wg) <= bound).all()


def test_rms_norm_in_place():
    """The residual stream updated in its own buffer, and dX in dH's and dY's."""
    need_gpu()
    x, r, g = rand((37, 1000), 1), rand((37, 1000), 2), rand((1000,), 3)
    y, h, rstd = rows.rms_norm_fwd(x, g, EPS, r)
    r2, x2 = r.clone(), x.clone()
    y2, h2, _ = rows.rms_norm_fwd(x, g, EPS, r2, H=r2)
    assert h2 is r2 and torch.equal(h, r2) and torch.equal(y, y2)
    q, h3 = rows.rms_norm_int8(x2, g, EPS, r, H=x2)
    assert h3 is x2 and torch.equal(h, x2)
    dy, dh = rand((37, 1000), 4), rand((37, 1000), 5)
    dx, dg = rows.rms_norm_bwd(dy, h, rstd, g, dh)
    dh2, dy2 = dh.clone(), dy.clone()
    assert torch.equal(rows.rms_norm_bwd(dy, h, rstd, g, dh2, dX=dh2)[0], dx) and torch.equal(dh2, dx)
    got = rows.rms_norm_bwd(dy2, h, rstd, g, dh, dX=dy2)
    assert torch.equal(dy2, dx) and torch.equal(got[1], dg)


def test_rms_norm_odd_values():
    """Zero rows, rows with NaN or infinity, and squares beyond fp32."""
    need_gpu()
    x = rand((6, 500), 1)
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 499] = float("inf")
    x[3] *= 1e25
    x[4] *= 1e-30
    g = torch.ones(500, dtype=BF16, device="cuda")
    y, _, rstd = rows.rms_norm_fwd(x, g, EPS)
    q, _ = rows.rms_norm_int8(x, g, EPS)
    v = f64(rows.dequant_rows(q))
    assert (f64(y)[0] == 0).all() and (v[0] == 0).all()
    assert np.isnan(f64(y)[1]).all() and np.isnan(v[1]).all()
    assert np.isnan(v[2]).all() and f64(rstd)[2] == 0
    assert f64(rstd)[3] == 0 and (f64(y)[3] == 0).all() and np.isnan(v[3]).all()
    want, _ = ref.rms_norm_fwd(f64(x)[4:], f64(g), EPS)
    close16(y[4:], want, np.abs(want))
    assert np.isfinite(v[4:]).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,k", SHAPES + LONG)
def test_swiglu(m, k, dtype):
    need_gpu()
    g, u, dy = rand((m, k), 1, dtype, 3.0), rand((m, k), 2, dtype), rand((m, k), 3, dtype)
    G, Uf, D = f64(g), f64(u), f64(dy)
    want = ref.swiglu_fwd(G, Uf)
    # e^-g through 2^(-g log2 e): the rounding of the exponent is |g| 2^-24
    grow = 1 + np.abs(G)
    close16(rows.swiglu_fwd(g, u), want, np.abs(want) * grow, "y")
    dg, du = rows.swiglu_bwd(dy, g, u)
    wg, wu = ref.swiglu_bwd(D, G, Uf)
    s = ref.sigmoid(G)
    close16(dg, wg, np.abs(D * Uf) * s * (1 + np.abs(G)) * grow, "dgate")
    close16(du, wu, np.abs(wu) * grow, "dup")
    q = rows.swiglu_int8(g, u)
    _, scale = ref.quantize_rows(want)
    slack = E32 * (1 + np.abs(G).max())
    np.testing.assert_allclose(f64(q.scale), scale, rtol=slack)
    assert (np.abs(codes_of(q) - want / scale[:, None]) <= 0.5 + 127 * 2 * slack).all()


def test_swiglu_far_gates():
    """Gates far out: e^-g overflows or vanishes."""
    need_gpu()
    g = torch.tensor([[-300.0, -90.0, -20.0, 0.0, 20.0, 90.0, 300.0, float("nan")]], dtype=BF16, device="cuda")
    u = torch.ones_like(g)
    y = f64(rows.swiglu_fwd(g, u))[0]
    dg, du = (f64(t)[0] for t in rows.swiglu_bwd(u, g, u))
    assert y[0] == 0 and y[3] == 0 and (y[4:7] == f64(g)[0, 4:7]).all() and np.isnan(y[7])
    assert np.isfinite(dg[:7]).all() and (dg[4:7] == 1).all() and dg[3] == 0.5 and du[3] == 0
    assert np.isnan(f64(rows.swiglu_int8(g, u).scale)[0])


def test_empty():
    """No rows, and rows of no values."""
    need_gpu()
    g = torch.ones(64, dtype=BF16, device="cuda")
    for m, k in ((0, 64), (3, 0), (0, 0)):
        x = torch.empty((m, k), dtype=BF16, device="cuda")
        gam = g[:k]
        q = rows.quantize_rows(x)
        assert q.codes.numel() == qlora.lib().qlora_int8_rows_bytes(m, k) and f64(q.scale).shape == (m,)
        if k == 0 and m:
            np.testing.assert_allclose(f64(q.scale), 1e-30 / 127, rtol=1e-6)
        assert rows.dequant_rows(q).shape == (m, k)
        y, h, rstd = rows.rms_norm_fwd(x, gam, EPS, x)
        assert y.shape == (m, k)
        dx, dg = rows.rms_norm_bwd(x, h, rstd, gam)
        assert dx.shape == (m, k) and (dg == 0).all()
        assert rows.swiglu_fwd(x, x).shape == (m, k)
        assert rows.swiglu_bwd(x, x, x)[0].shape == (m, k)
        rows.swiglu_int8(x, x)
        rows.rms_norm_int8(x, gam, EPS)


def test_autograd():
    """The modules' gradients are those of the formulas, through views and with
    both outputs used, and with only the residual stream used."""
    need_gpu()
    norm = rows.RMSNorm(96, EPS)
    with torch.no_grad():
        norm.weight.copy_(rand((96,), 1))
    x, r = rand((2, 5, 96), 2).requires_grad_(), rand((2, 5, 96), 3).requires_grad_()
    y, h = norm(x, r)
    dy, dh = rand((2, 5, 96), 4), rand((2, 5, 96), 5)
    torch.autograd.backward([y, h], [dy, dh])
    gam = f64(norm.weight)
    want, wg = ref.rms_norm_bwd(f64(dy).reshape(10, 96), f64(h).reshape(10, 96), gam, EPS, f64(dh).reshape(10, 96))
    mag = np.abs(want) + np.abs(f64(dh)).reshape(10, 96) + 8 * np.abs(f64(dy)).reshape(10, 96)
    close16(x.grad.reshape(10, 96), want, mag)
    assert torch.equal(x.grad, r.grad)
    close16(norm.weight.grad, wg, 10 * np.abs(f64(dy)).reshape(10, 96).sum(0) * 4)
    x.grad = r.grad = None
    _, h = norm(x, r)
    h.backward(dh)
    assert torch.equal(x.grad, dh)
    x.grad = None
    norm(x).backward(dy)
    want, _ = ref.rms_norm_bwd(f64(dy).reshape(10, 96), f64(x).reshape(10, 96), gam, EPS)
    close16(x.grad.reshape(10, 96), want, 8 * np.abs(f64(dy)).reshape(10, 96))
    both = rand((3, 4, 2 * 40), 6).requires_grad_()
    out = rows.swiglu(both[..., :40], both[..., 40:])
    d = rand((3, 4, 40), 7)
    out.backward(d)
    b = f64(both).reshape(12, 80)
    wg, wu = ref.swiglu_bwd(f64(d).reshape(12, 40), b[:, :40], b[:, 40:])
    m = np.abs(f64(d)).reshape(12, 40) * (1 + np.abs(b[:, :40])) ** 2 * (1 + np.abs(b[:, 40:]))
    close16(both.grad.reshape(12, 80)[:, :40], wg, m)
    close16(both.grad.reshape(12, 80)[:, 40:], wu, m)


def test_large_offsets():
    """More than 2^31 elements: the last rows are those of a call of their own."""
    need_gpu()
    m, k = 530000, 4096
    x = rand((m, 64), 1).repeat(1, 64)
    g = rand((k,), 2)
    assert x.numel() > 2 ** 31
    y, h, rstd = rows.rms_norm_fwd(x, g, EPS, x)
    a, b, c = rows.rms_norm_fwd(x[-50:], g, EPS, x[-50:])
    assert torch.equal(y[-50:], a) and torch.equal(h[-50:], b) and torch.equal(rstd[-50:], c)
    dx, _ = rows.rms_norm_bwd(y, h, rstd, g)
    assert torch.equal(dx[-50:], rows.rms_norm_bwd(a, b, c, g)[0])
    del dx, h
    s = rows.swiglu_fwd(x, y)
    assert torch.equal(s[-50:], rows.swiglu_fwd(x[-50:], a))
    dg, du = rows.swiglu_bwd(s, x, y)
    want = rows.swiglu_bwd(s[-50:], x[-50:], a)
    assert torch.equal(dg[-50:], want[0]) and torch.equal(du[-50:], want[1])


def test_refusals():
    need_gpu()
    x, g = rand((4, 64), 1), rand((64,), 2)
    y, h, rstd = rows.rms_norm_fwd(x, g, EPS)
    with pytest.raises(ValueError, match="GPU"):
        rows.quantize_rows(x.cpu())
    with pytest.raises(TypeError, match="must be"):
        rows.rms_norm_fwd(x.float(), g, EPS)
    with pytest.raises(TypeError, match="gamma"):
        rows.rms_norm_fwd(x, g.half(), EPS)
    with pytest.raises(ValueError, match="gamma"):
        rows.rms_norm_fwd(x, g[:32], EPS)
    with pytest.raises(ValueError, match="residual"):
        rows.rms_norm_fwd(x, g, EPS, x[:2])
    with pytest.raises(TypeError, match="residual"):
        rows.rms_norm_fwd(x, g, EPS, x.half())
    with pytest.raises(ValueError, match="H is written only"):
        rows.rms_norm_fwd(x, g, EPS, H=x)
    with pytest.raises(RuntimeError, match="eps"):
        rows.rms_norm_fwd(x, g, 0.0)
    with pytest.raises(RuntimeError, match="eps"):
        rows.rms_norm_int8(x, g, float("nan"))
    with pytest.raises(ValueError, match="last dimension"):
        rows.quantize_rows(rand((64, 4), 3).t())
    with pytest.raises(ValueError, match="overlap"):
        rows.quantize_rows(x[:1].expand(4, 64))
    with pytest.raises(ValueError, match="2-D"):
        rows.quantize_rows(x[0])
    with pytest.raises(ValueError, match="up"):
        rows.swiglu_fwd(x, x[:, :32])
    with pytest.raises(ValueError, match="Y must be"):
        rows.swiglu_fwd(x, x, Y=torch.empty_like(x).t())
    with pytest.raises(RuntimeError, match="QLORA_MAX_NORM_WIDTH"):
        rows.rms_norm_fwd(rand((1, 32769), 1), rand((32769,), 2), EPS)
    with pytest.raises(RuntimeError, match="132104"):
        rows.quantize_rows(rand((1, 132105), 1))
    with pytest.raises(ValueError, match="rstd"):
        rows.rms_norm_bwd(x, h, rstd[:2], g)
    with pytest.raises(ValueError, match="codes"):
        q = rows.quantize_rows(x)
        rows.dequant_rows(rows.Int8Rows(q.codes[:100], q.scale, 4, 64, BF16))


def test_other_stream():
    """A call on a side stream runs there, after what that stream waits for."""
    need_gpu()
    s = torch.cuda.Stream()
    x = rand((2000, 4096), 1)
    g = rand((4096,), 2)
    y, _, _ = rows.rms_norm_fwd(x, g, EPS)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        x2 = x * 2
        y2, _, _ = rows.rms_norm_fwd(x2, g, 4 * EPS)
    torch.cuda.current_stream().wait_stream(s)
    # doubling x and scaling eps with it changes no bit of y
    assert torch.equal(y, y2)
