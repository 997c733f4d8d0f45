"""The differentiable forms without a GPU: what they refuse before any kernel
is called, and which gradients they ask the kernels for (the kernels' calls
replaced by torch)."""

import pytest
import torch

from bit_nf4_quantized_double_amd import int8, rows

BF16 = torch.bfloat16


def zeros(*shape):
    return torch.zeros(shape, dtype=BF16)


# as many elements, or as many rows of the other's width: nothing that a
# reshape to matrices would stumble over
SHAPES = [((8, 64), (4, 128)), ((2, 3, 64), (3, 2, 64)), ((2, 3, 64), (6, 64)), ((6, 64), (64,)), ((4, 64), (1, 64))]


@pytest.mark.parametrize("a,b", SHAPES)
def test_operands_of_other_shapes_are_refused(a, b):
    with pytest.raises(ValueError, match="up must have shape"):
        rows.swiglu(zeros(*a), zeros(*b))
    with pytest.raises(ValueError, match="up must have shape"):
        rows.swiglu(zeros(*b), zeros(*a))
    with pytest.raises(ValueError, match="residual must have shape"):
        rows.RMSNorm(a[-1], device="cpu")(zeros(*a), zeros(*b))
    with pytest.raises(TypeError, match="residual must be a torch.Tensor"):
        rows.RMSNorm(64, device="cpu")(zeros(4, 64), 0)


@pytest.mark.parametrize("shape", [(8, 64), (128, 1), (2, 1, 64), (128, 128, 2)])
def test_product_refuses_rows_of_another_width(shape):
    w = int8.Int8Weight(torch.empty(int8.weight_bytes(32, 128), dtype=torch.uint8), torch.ones(32), 32, 128)
    with pytest.raises(ValueError, match="columns, the weight 128"):
        int8.Int8LinearFunction.apply(zeros(*shape), None, w)


@pytest.fixture
def norm_calls(monkeypatch):
    """The norm's kernels replaced by torch; the backward's arguments recorded."""
    calls = []

    def fwd(X, gamma, eps, residual=None, *, H=None, Y=None):
        h = X if residual is None else torch.add(X, residual, out=H)
        rstd = (h.float().square().mean(1) + eps).rsqrt()
        return Y.copy_((h.float() * rstd[:, None] * gamma.float()).to(X.dtype)), h, rstd

    def bwd(dY, H, rstd, gamma, dH=None):
        calls.append(dH)
        h32, dy = H.float(), dY.float()
        hat, g = h32 * rstd[:, None], dy * gamma.float()
        dx = rstd[:, None] * (g - hat * (g * hat).mean(1, keepdim=True))
        return (dx if dH is None else dx + dH.float()).to(H.dtype), (dy * hat).sum(0)

    monkeypatch.setattr(rows, "rms_norm_fwd", fwd)
    monkeypatch.setattr(rows, "rms_norm_bwd", bwd)
    return calls


def _norm_inputs():
    g = torch.Generator().manual_seed(1)
    x, r = (torch.randn(5, 32, generator=g).to(BF16).requires_grad_() for _ in range(2))
    return rows.RMSNorm(32, device="cpu"), x, r, torch.randn(5, 32, generator=g).to(BF16)


def test_norm_without_a_gradient_of_the_residual_stream(norm_calls):
    """The last norm of a model: nothing reads h, so no gradient of it is made."""
    norm, x, r, d = _norm_inputs()
    y, h = norm(x, r)
    y.backward(d)
    assert norm_calls == [None]
    assert torch.equal(x.grad, r.grad) and norm.weight.grad is not None


def test_norm_with_a_gradient_of_the_residual_stream_alone(norm_calls):
    """Nothing reads y: the gradient passes through, and gamma's is zero."""
    norm, x, r, d = _norm_inputs()
    y, h = norm(x, r)
    h.backward(d)
    assert norm_calls == []
    assert torch.equal(x.grad, d) and torch.equal(r.grad, d) and (norm.weight.grad == 0).all()


def test_norm_with_both_gradients(norm_calls):
    norm, x, r, d = _norm_inputs()
    y, h = norm(x, r)
    torch.autograd.backward([y, h], [d, d])
    assert len(norm_calls) == 1 and torch.equal(norm_calls[0], d)


def test_norm_with_a_frozen_weight(norm_calls):
    norm, x, r, d = _norm_inputs()
    norm.weight.requires_grad_(False)
    norm(x, r)[0].backward(d)
    assert norm.weight.grad is None and x.grad is not None
    norm, x, r, d = _norm_inputs()
    norm(x.detach(), r.detach())[0].backward(d)
    assert norm.weight.grad is not None and x.grad is None and r.grad is None
