"""A caller's workspace tensor: what a call may write into, and what it
refuses (no GPU: the check is made before anything is enqueued)."""

import pytest
import torch

from bit_nf4_quantized_double_amd import qlora

CPU = torch.device("cpu")


def test_workspace_is_taken_when_it_holds_the_bytes():
    for ws in (torch.empty(100, dtype=torch.uint8), torch.empty(30), torch.empty(5, 20, dtype=torch.uint8)):
        got, n = qlora._ws(100, CPU, ws)
        assert got is ws and 100 <= n <= ws.numel() * ws.element_size()
    assert qlora._ws(0, CPU, torch.empty(3)) == (None, 0)


def test_workspace_that_is_too_small_is_replaced():
    for ws in (None, torch.empty(99, dtype=torch.uint8), torch.empty(24)):
        got, n = qlora._ws(100, CPU, ws)
        assert got is not ws and n == 100 == got.numel() and got.dtype == torch.uint8


@pytest.mark.parametrize("ws", [
    torch.empty(1, dtype=torch.uint8).expand(1000),    # one byte seen a thousand times
    torch.empty(4000, dtype=torch.uint8)[::4],         # bytes apart
    torch.empty(40, 30, dtype=torch.uint8).t(),
], ids=["expanded", "strided", "transposed"])
def test_workspace_that_is_not_contiguous_is_refused(ws):
    with pytest.raises(ValueError, match="contiguous"):
        qlora._ws(100, CPU, ws)


def test_workspace_elsewhere_is_refused():
    """On another device, or on the host, the kernels would write to an
    address that is not theirs."""
    with pytest.raises(ValueError, match="must be on meta"):
        qlora._ws(100, torch.device("meta"), torch.empty(1000, dtype=torch.uint8))
    with pytest.raises(ValueError, match="must be on cpu"):
        qlora._ws(100, CPU, torch.empty(1000, dtype=torch.uint8, device="meta"))


def test_workspace_that_is_no_tensor_is_refused():
    with pytest.raises(TypeError, match="ws must be a torch.Tensor"):
        qlora._ws(100, CPU, bytearray(1000))
