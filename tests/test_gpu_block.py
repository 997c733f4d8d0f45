"""The MLP block of a decoder layer: trained with NF4 linears, adapters, norm
and SwiGLU, served in 8 bits."""

import numpy as np
import pytest
import torch

import oracle.rows as ref
from bit_nf4_quantized_double_amd import block, int8, qlora, rows
from rows_util import codes_of, f64, need_gpu, rand

pytestmark = pytest.mark.gpu


def _block(width, hidden, seed=0):
    return block.MLPBlock(rand((hidden, width), seed, torch.float32, 0.02), rand((hidden, width), seed + 1, torch.float32, 0.02),
                          rand((width, hidden), seed + 2, torch.float32, 0.02), r=8, alpha=16.0)


def test_training_block_gradients_against_differences():
    """The loss' change along the gradient of each kind of parameter (norm,
    adapters) and of both inputs, against the step it predicts."""
    need_gpu()
    b = _block(128, 192)
    with torch.no_grad():
        for lin in (b.gate, b.up, b.down):
            lin.B.copy_(rand(tuple(lin.B.shape), 5, scale=0.05))
    x, r, d = rand((40, 128), 6).requires_grad_(), rand((40, 128), 7).requires_grad_(), rand((40, 128), 8)
    dh = rand((40, 128), 9)

    def loss():
        y, h = b(x, r)
        return float((y.double() * d.double()).sum() + (h.double() * dh.double()).sum())

    y, h = b(x, r)
    torch.autograd.backward([y, h], [d, dh])
    for name, p in (("norm", b.norm.weight), ("gate.A", b.gate.A), ("down.B", b.down.B), ("x", x), ("residual", r)):
        g = p.grad.double()
        v = (g / g.norm() * p.detach().double().norm() * 0.05)
        with torch.no_grad():
            keep = p.detach().clone()
            p.copy_((keep.double() + v).to(p.dtype))
            up, hi = loss(), p.detach().double().clone()
            p.copy_((keep.double() - v).to(p.dtype))
            down, lo = loss(), p.detach().double().clone()
            p.copy_(keep)
        want = float((g * (hi - lo)).sum())  # along the step as it was rounded
        # bf16 activations and gradients (2^-8 each, as independent errors over
        # the entries) and the curvature over a twentieth of the norm
        assert abs((up - down) - want) <= 0.05 * abs(want), (name, up - down, want)


def test_served_block_is_its_operators():
    """Bit for bit what the operators give one by one."""
    need_gpu()
    b = _block(256, 384)
    s = block.Int8MLPBlock(b)
    for m in (1, 3, 40, 300):
        x, r = rand((m, 256), m), rand((m, 256), m + 1)
        y, h = s(x, r)
        q, h2 = rows.rms_norm_int8(x, b.norm.weight.detach(), b.norm.eps, r)
        gate = int8.linear_fwd(int8.quantize_weight(qlora.merge(b.gate.w, b.gate.A.detach(), b.gate.B.detach(), 8, 16.0)), q)
        up = int8.linear_fwd(int8.quantize_weight(qlora.merge(b.up.w, b.up.A.detach(), b.up.B.detach(), 8, 16.0)), q)
        want = int8.linear_fwd(s.down, rows.swiglu_int8(gate, up))
        assert torch.equal(h, h2) and torch.equal(y, want)


def test_served_block_against_64_bits():
    """The served block's own numbers, from its codes and scales."""
    need_gpu()
    b = _block(256, 384, seed=3)
    s = block.Int8MLPBlock(b)
    x, r = rand((33, 256), 1), rand((33, 256), 2)
    y, h = s(x, r)
    gu, dn = codes_of(s.gate_up) * f64(s.gate_up.scale)[:, None], codes_of(s.down) * f64(s.down.scale)[:, None]
    n, _ = ref.rms_norm_fwd(f64(h), f64(b.norm.weight), b.norm.eps)
    q, sc = ref.quantize_rows(n)
    t = (q * sc[:, None]) @ gu.T
    q, sc = ref.quantize_rows(ref.swiglu_fwd(t[:, :384], t[:, 384:]))
    want = (q * sc[:, None]) @ dn.T
    # bf16 roundings of gate and up move some codes by one step of 127 to the amax
    assert np.linalg.norm(f64(y) - want) <= 0.01 * np.linalg.norm(want)


def test_command():
    need_gpu()
    out = block.main(["--width", "256", "--hidden", "512", "--tokens", "200", "--steps", "4"])
    assert out["losses"][-1] < out["losses"][0] and out["same_residual"] and out["difference"] < 0.03


def test_refusals():
    need_gpu()
    with pytest.raises(ValueError, match="w_down"):
        block.MLPBlock(rand((64, 128), 1, torch.float32), rand((64, 128), 1, torch.float32), rand((64, 128), 1, torch.float32))


# At these sizes all three numbers of tokens take the few tokens' kernel, on rows
# that the norm and SwiGLU wrote; tiles in a graph: test_gpu_int8_plans.py.
def test_served_block_in_a_graph():
    """Captured once, replayed on new inputs: every replay is the eager result,
    with eager work in between (1 token: quantized inside the product; 40: its
    own launch; 300: tiles)."""
    need_gpu()
    s = block.Int8MLPBlock(_block(256, 384))
    for m in (1, 40, 300):
        x, r = rand((m, 256), 1), rand((m, 256), 2)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s(x, r)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y, h = s(x, r)
        for seed in (3, 4, 5):
            x.copy_(rand((m, 256), seed))
            r.copy_(rand((m, 256), seed + 10))
            want, hw = s(x, r)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want) and torch.equal(h, hw)
