"""What the served MLP block keeps of the block it was made from."""

import pytest
import torch

from bit_nf4_quantized_double_amd import block
from rows_util import need_gpu, rand

pytestmark = pytest.mark.gpu


def _block(width, hidden, seed=0):
    return block.MLPBlock(rand((hidden, width), seed, torch.float32, 0.02), rand((hidden, width), seed + 1, torch.float32, 0.02),
                          rand((width, hidden), seed + 2, torch.float32, 0.02), r=8, alpha=16.0)


def test_served_block_keeps_what_it_was_made_from():
    """Training that goes on after the conversion does not reach it."""
    need_gpu()
    b = _block(256, 384)
    s = block.Int8MLPBlock(b)
    x, r = rand((7, 256), 1), rand((7, 256), 2)
    y, _ = s(x, r)
    with torch.no_grad():
        for p in b.parameters():
            p.mul_(1.5).add_(0.25)
    assert torch.equal(s(x, r)[0], y)
