"""The differentiable forms of norm, SwiGLU and the int8 product on the GPU:
gradients that go missing, and the smallest widths."""

import numpy as np
import pytest
import torch

from bit_nf4_quantized_double_amd import int8, qlora, rows
from rows_util import close16, f64, need_gpu, rand

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def test_bias_gradient_with_rows_in_8_bits():
    """Int8Linear on rows that are in 8 bits already: its bias is a parameter
    there too."""
    need_gpu()
    lin = int8.Int8Linear(rand((48, 200), 1, F32, 0.02), rand((48,), 2))
    x, d = rand((6, 200), 3), rand((6, 48), 4)
    q = rows.quantize_rows(x)
    y = lin(q)
    assert torch.equal(y, int8.linear_fwd(lin.w, q, lin.bias.detach()))
    y.backward(d)
    close16(lin.bias.grad, f64(d).sum(0), np.abs(f64(d)).sum(0))
    with torch.no_grad():
        assert not lin(q).requires_grad
    lin.bias.requires_grad_(False)
    assert not lin(q).requires_grad
    assert not int8.Int8Linear(rand((48, 200), 1, F32, 0.02))(q).requires_grad


def _twice(first, leaves):
    """Gradients of gradients, beside a term that has them."""
    leaf = leaves[0]
    for loss in (first, (first.float().square()).sum(), first.float().sum() + leaf.float().square().sum()):
        loss = loss.float().sum()
        g = torch.autograd.grad(loss, leaf, create_graph=True, retain_graph=True)[0]
        with pytest.raises(RuntimeError, match="second derivative"):
            (g.float().square().sum() + leaf.float().square().sum()).backward()
    # a first-order step with the graph kept is as it was
    want = torch.autograd.grad(first.float().sum(), leaf, retain_graph=True)[0]
    got = torch.autograd.grad(first.float().sum(), leaf, retain_graph=True, create_graph=True)[0]
    assert torch.equal(want, got)


def test_no_second_derivatives():
    """They have no formula here: asked for, they are refused, not left out."""
    need_gpu()
    x, r = rand((6, 64), 1).requires_grad_(), rand((6, 64), 2).requires_grad_()
    _twice(rows.swiglu(x, r), (x, r))
    _twice(rows.RMSNorm(64, EPS)(x), (x,))
    y, h = rows.RMSNorm(64, EPS)(x, r)
    _twice(y + h, (r,))
    _twice(int8.Int8Linear(rand((32, 64), 3, F32, 0.02), rand((32,), 4), transposed=True)(x), (x,))


def test_no_second_derivatives_of_the_nf4_linear():
    need_gpu()
    lin = qlora.QLoRALinear(rand((64, 128), 1, F32, 0.02), r=8, alpha=16.0)
    with torch.no_grad():
        lin.B.copy_(rand((64, 8), 2, scale=0.1))
    x = rand((6, 128), 3).requires_grad_()
    _twice(lin(x), (x,))
    _twice(lin(x), (lin.A,))


@pytest.mark.parametrize("m", [1, 5])
def test_rows_of_one_value(m):
    """Also where a gradient or an input is one value seen m times."""
    need_gpu()
    g, u = rand((m, 1), 1).requires_grad_(), rand((m, 1), 2).requires_grad_()
    rows.swiglu(g, u).sum().backward()
    dg, du = rows.swiglu_bwd(torch.ones((m, 1), dtype=BF16, device="cuda"), g.detach(), u.detach())
    assert torch.equal(g.grad, dg) and torch.equal(u.grad, du)
    one = rand((1, 1), 3).expand(m, 1)
    assert torch.equal(rows.swiglu(one, u.detach()), rows.swiglu(one.contiguous(), u.detach()))
    x = rand((m, 1), 4).requires_grad_()
    norm = rows.RMSNorm(1, EPS)
    norm(x).sum().backward()
    _, h, rstd = rows.rms_norm_fwd(x.detach(), norm.weight.detach(), EPS)
    dx, dgamma = rows.rms_norm_bwd(torch.ones((m, 1), dtype=BF16, device="cuda"), h, rstd, norm.weight.detach())
    assert torch.equal(x.grad, dx) and torch.equal(norm.weight.grad, dgamma.to(BF16))


def test_no_rows_and_rows_of_no_values():
    need_gpu()
    for shape in ((0, 64), (2, 0, 64), (3, 0), (2, 3, 0)):
        x, r = (torch.empty(shape, dtype=BF16, device="cuda", requires_grad=True) for _ in range(2))
        norm = rows.RMSNorm(shape[-1], EPS)
        y, h = norm(x, r)
        s = rows.swiglu(y, h)
        assert y.shape == h.shape == s.shape == shape
        s.sum().backward()
        assert x.grad.shape == r.grad.shape == shape and (norm.weight.grad == 0).all()
        lin = int8.Int8Linear(rand((40, shape[-1]), 1, F32, 0.02), rand((40,), 2), transposed=True)
        x.grad = None
        out = lin(x)
        out.sum().backward()
        rows_in = out.numel() // 40
        assert out.shape == (*shape[:-1], 40) and x.grad.shape == shape
        assert torch.equal(out, lin.bias.detach().expand(out.shape)) and (lin.bias.grad == rows_in).all()


@pytest.mark.parametrize("shape", [(6, 64), (2, 3, 64)])
def test_outputs_modified_in_place(shape):
    """What a form returns is a tensor of its own: it can be changed in place
    where no gradient needs it, and where one does (h) the backward says so."""
    need_gpu()
    x, r = rand(shape, 1).requires_grad_(), rand(shape, 2).requires_grad_()
    norm = rows.RMSNorm(64, EPS)
    lin = int8.Int8Linear(rand((64, 64), 3, F32, 0.02), rand((64,), 4), transposed=True)
    d = rand(shape, 5)
    for call in (lambda: norm(x), lambda: norm(x, r)[0], lambda: rows.swiglu(x, r), lambda: lin(x)):
        want = torch.autograd.grad(call(), x, 2 * d)[0]
        y = call()
        y.mul_(2)
        assert torch.equal(torch.autograd.grad(y, x, d)[0], want)
    y, h = norm(x, r)
    h.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward(d)
