"""The differentiable forms without a GPU: what they refuse before any kernel
is called."""

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
