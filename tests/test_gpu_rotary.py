"""Rotary positions against 64 bits: pairs, parts of heads, far positions,
strides, in place, gradients.

Bound: the angle is off by at most 2^-26 turns (its fp32 remainder) and sine and
cosine by 2^-22 each, so a result before rounding by (|a| + |b|) factor 2^-21;
then one rounding to 16 bits.
"""

import numpy as np
import pytest
import torch

import oracle.decoder as ref
from bit_nf4_quantized_double_amd import rotary
from rows_util import TINY, U, f64, need_gpu, rand

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def _check(got, x, positions, f, factor, interleaved, inverse=False):
    want = ref.rotate(f64(x), positions, f, factor, interleaved, inverse)
    n = len(f)
    mag = np.zeros_like(want)
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    both = np.abs(f64(x)[..., a]) + np.abs(f64(x)[..., b])
    mag[..., a] = mag[..., b] = both * abs(factor) * 2.0 ** -21
    bound = U[got.dtype] * np.abs(want) + mag * 1.01 + TINY[got.dtype]
    bound[..., 2 * n:] = 0.0  # what is not turned is copied
    bad = ~(np.abs(f64(got) - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[0], f64(got)[bad][0], want[bad][0])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("t,h,hk,d,rot", [(1, 1, 0, 2, 2), (1, 32, 8, 128, 128), (7, 3, 1, 64, 32), (300, 10, 2, 80, 32),
                                          (5, 2, 2, 96, 96), (17, 4, 4, 48, 34), (3, 1, 1, 9, 6), (33, 5, 5, 24, 0),
                                          (40, 70, 3, 128, 64), (0, 4, 2, 64, 64), (9000, 1, 1, 16, 16)])
def test_against_64_bits(t, h, hk, d, rot, interleaved, dtype):
    need_gpu()
    q, k = rand((t, h, d), 1, dtype), rand((t, hk, d), 2, dtype) if hk else None
    pos = torch.randint(0, 5000, (t,), device="cuda", dtype=torch.int32)
    freqs = rotary.frequencies(rot)
    f = 10000.0 ** (-2.0 * np.arange(rot // 2) / max(rot, 1))
    for call, inverse in ((rotary.rotate, False), (rotary.rotate_bwd, True)):
        a, b = call(q, k, pos, freqs, interleaved=interleaved)
        _check(a, q, pos.cpu().numpy(), f, 1.0, interleaved, inverse)
        if hk:
            _check(b, k, pos.cpu().numpy(), f, 1.0, interleaved, inverse)
        else:
            assert b is None


@pytest.mark.parametrize("scaling,by", [(None, 1.0), ("linear", 4.0), ("base", 4.0), ("blended", 8.0)])
@pytest.mark.parametrize("far", [131072, 2 ** 20, 2 ** 31 - 1, 2 ** 45])
def test_far_positions(scaling, by, far):
    need_gpu()
    x = rand((64, 2, 128), 3)
    pos = far - torch.arange(64, device="cuda", dtype=torch.int64) * 7919 % far
    freqs = rotary.frequencies(128, scaling=scaling, by=by)
    i = np.arange(64)
    base = 10000.0 * by ** (128 / 126) if scaling == "base" else 10000.0
    f, factor = base ** (-2.0 * i / 128), 1.0
    if scaling == "linear":
        f = f / by
    if scaling == "blended":
        keep = np.clip((4096 * f / (2 * np.pi) - 1) / 31, 0, 1)
        f, factor = f / by * (1 - keep) + f * keep, 0.1 * np.log(by) + 1
    # what the tensor holds: f to 2^-53 of itself, which at 2^45 positions is 2^-8 radians
    turns = [int(t) % 2 ** 64 for t in freqs.turns.tolist()]
    assert np.allclose([t * 2.0 ** -64 * 2 * np.pi for t in turns], f, rtol=1e-12, atol=0)
    angle = np.array([[(int(p) * t % 2 ** 64) * 2.0 ** -64 for t in turns] for p in pos.tolist()]) * 2 * np.pi
    c, s = np.cos(angle)[:, None] * factor, np.sin(angle)[:, None] * factor
    y, _ = rotary.rotate(x, None, pos, freqs)
    X = f64(x)
    want = np.concatenate([X[..., :64] * c - X[..., 64:] * s, X[..., 64:] * c + X[..., :64] * s], -1)
    both = np.abs(X[..., :64]) + np.abs(X[..., 64:])
    bound = U[BF16] * np.abs(want) + np.concatenate([both, both], -1) * factor * 2.0 ** -21
    assert (np.abs(f64(y) - want) <= bound).all()
    if far <= 2 ** 20:
        _check(y, x, pos.cpu().numpy(), f, factor, False)


def test_negative_and_32_bit_positions():
    need_gpu()
    x = rand((9, 2, 64), 1)
    pos = torch.arange(-4, 5, device="cuda")
    a, _ = rotary.rotate(x, None, pos, rotary.frequencies(64))
    b, _ = rotary.rotate(x, None, pos.int(), rotary.frequencies(64))
    c, _ = rotary.rotate_bwd(x, None, -pos, rotary.frequencies(64))
    assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("offset", [0, 8, 1])
@pytest.mark.parametrize("interleaved", [False, True])
def test_slices_and_in_place(offset, interleaved):
    """Slices of a projection's output, 16-byte aligned and not, in place too; what
    is between them stays."""
    need_gpu()
    t, h, hk, d = 50, 6, 2, 64
    wide = rand((t, (h + 2 * hk) * d + offset), 1)
    q = wide[:, offset:offset + h * d].view(t, h, d) if offset == 0 else wide[:, offset:offset + h * d].unflatten(1, (h, d))
    k = wide[:, offset + h * d:offset + (h + hk) * d].unflatten(1, (hk, d))
    pos = torch.arange(t, device="cuda")
    freqs = rotary.frequencies(32)
    a, b = rotary.rotate(q.contiguous(), k.contiguous(), pos, freqs, interleaved=interleaved)
    c, e = rotary.rotate(q, k, pos, freqs, interleaved=interleaved)
    assert torch.equal(a, c) and torch.equal(b, e)
    before = wide.clone()
    rotary.rotate(q, k, pos, freqs, interleaved=interleaved, Q_out=q, K_out=k)
    assert torch.equal(q, a) and torch.equal(k, b)
    assert torch.equal(wide[:, :offset], before[:, :offset])
    assert torch.equal(wide[:, offset + (h + hk) * d:], before[:, offset + (h + hk) * d:])


def test_offsets_past_32_bits():
    """Tokens so far apart that their offsets need more than 32 bits, in place."""
    need_gpu()
    t, h, d, far = 2200, 2, 64, 1 << 20
    x, f = rand((t, h, d), 1), rotary.frequencies(d)
    p = torch.arange(t, device="cuda")
    want, _ = rotary.rotate(x, None, p, f)
    y = torch.empty((t - 1) * far + h * d, dtype=x.dtype, device="cuda").as_strided((t, h, d), (far, d, 1))
    y.copy_(x)
    rotary.rotate(y, None, p, f, Q_out=y)
    assert torch.equal(y, want)


def test_autograd():
    """The gradient is the inverse rotation, also where one output is not used."""
    need_gpu()
    q, k = rand((20, 4, 64), 1).requires_grad_(), rand((20, 2, 64), 2).requires_grad_()
    pos, freqs = torch.arange(20, device="cuda") * 100, rotary.frequencies(64)
    dq, dk = rand((20, 4, 64), 3), rand((20, 2, 64), 4)
    a, b = rotary.rotary(q, k, pos, freqs)
    torch.autograd.backward([a, b], [dq, dk])
    wq, wk = rotary.rotate_bwd(dq, dk, pos, freqs)
    assert torch.equal(q.grad, wq) and torch.equal(k.grad, wk)
    for keep in (0, 1):
        x = [t.detach().clone().requires_grad_() for t in (q, k)]
        rotary.rotary(*x, pos, freqs)[keep].backward((dq, dk)[keep])
        assert torch.equal(x[keep].grad, (wq, wk)[keep]) and x[1 - keep].grad is None
    # and against the formula: <dq, R x> changes by <R^T dq, dx>, R being linear
    y = rand((20, 4, 64), 9)
    z, _ = rotary.rotate(y, None, pos, freqs)
    lhs, rhs = (f64(z) * f64(dq)).sum(), (f64(y) * f64(wq)).sum()
    # 5120 products of roundings to bf16, independent
    assert abs(lhs - rhs) <= 8 * 2.0 ** -8 * 5120 ** 0.5


def test_refusals():
    need_gpu()
    q, pos, f = rand((4, 2, 64), 1), torch.arange(4, device="cuda"), rotary.frequencies(64)
    with pytest.raises(ValueError, match="tokens, heads"):
        rotary.rotate(q[0], None, pos, f)
    with pytest.raises(TypeError, match="bf16 or fp16"):
        rotary.rotate(q.float(), None, pos, f)
    with pytest.raises(ValueError, match="positions must be"):
        rotary.rotate(q, None, pos[:3], f)
    with pytest.raises(TypeError, match="positions must be"):
        rotary.rotate(q, None, pos.float(), f)
    with pytest.raises(ValueError, match="to turn in heads of"):
        rotary.rotate(q[..., :32], None, pos, f)
    with pytest.raises(TypeError, match="K must be"):
        rotary.rotate(q, q.half(), pos, f)
    with pytest.raises(ValueError, match="last dimension"):
        rotary.rotate(q.transpose(1, 2), None, pos, rotary.frequencies(2))
    with pytest.raises(RuntimeError, match="overlap"):
        rotary.rotate(q, None, pos, f, Q_out=q[:1].expand(4, 2, 64))
