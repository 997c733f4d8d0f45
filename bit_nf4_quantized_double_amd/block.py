"""The MLP half of a decoder layer, trained and served with this package's
operators.

:class:`MLPBlock` trains: RMS norm with the residual, gate and up projections,
SwiGLU and the down projection, the three linears with a frozen NF4 weight and
an adapter each.  :class:`Int8MLPBlock` serves what was trained: the adapters
are merged, the merged weights quantized to 8 bits, and the norm and SwiGLU
write the 8-bit operands of the products themselves.

    python -m bit_nf4_quantized_double_amd.block [--width 4096 --hidden 11008 --tokens 2048]

trains a small number of steps on synthetic data, converts, and prints the
loss, how far the two forms differ and the time of a call of each.
"""

from __future__ import annotations

import argparse

import torch

from . import int8, qlora, rows


class MLPBlock(torch.nn.Module):
    """(x, residual) -> (down(silu(gate(n)) * up(n)), h) with h = x + residual
    and n the RMS norm of h; the weights are fp32 [n_out, k_in] and frozen as
    NF4, the adapters and the norm's weight are trained, in bf16."""

    def __init__(self, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, r: int = 16,
                 alpha: float = 32.0, eps: float = 1e-5):
        super().__init__()
        hidden, width = w_gate.shape
        if w_up.shape != (hidden, width) or w_down.shape != (width, hidden):
            raise ValueError("w_gate and w_up must be [hidden, width], w_down [width, hidden]")
        self.norm = rows.RMSNorm(width, eps, device=w_gate.device)
        self.gate = qlora.QLoRALinear(w_gate, r, alpha)
        self.up = qlora.QLoRALinear(w_up, r, alpha)
        self.down = qlora.QLoRALinear(w_down, r, alpha)

    def forward(self, x, residual):
        y, h = self.norm(x, residual)
        return self.down(rows.swiglu(self.gate(y), self.up(y))), h


def _merged(lin: qlora.QLoRALinear) -> torch.Tensor:
    return qlora.merge(lin.w, lin.A.detach(), lin.B.detach(), lin.r, lin.alpha)


class Int8MLPBlock:
    """An :class:`MLPBlock` with its adapters merged, in 8 bits: norm,
    product, SwiGLU, product, and no quantizer between them.  Gate and up are
    one product, whose output's halves SwiGLU reads."""

    def __init__(self, block: MLPBlock):
        # a copy, as the merged weights are: training that goes on does not reach it
        self.gamma, self.eps = block.norm.weight.detach().clone(), block.norm.eps
        self.hidden = block.gate.w.n_out
        self.gate_up = int8.quantize_weight(torch.cat([_merged(block.gate), _merged(block.up)]))
        self.down = int8.quantize_weight(_merged(block.down))

    @torch.no_grad()
    def __call__(self, x: torch.Tensor, residual: torch.Tensor):
        """bf16 [tokens, width] each; returns (output, new residual stream)."""
        q, h = rows.rms_norm_int8(x, self.gamma, self.eps, residual)
        gu = int8.linear_fwd(self.gate_up, q)
        act = rows.swiglu_int8(gu[:, :self.hidden], gu[:, self.hidden:])
        return int8.linear_fwd(self.down, act), h


def _time(fn, n: int = 20) -> float:
    for _ in range(3):
        fn()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        fn()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / n


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--width", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=11008)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args(argv)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)

    def randn(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * scale

    block = MLPBlock(randn(a.hidden, a.width, scale=0.02), randn(a.hidden, a.width, scale=0.02),
                     randn(a.width, a.hidden, scale=0.02))
    x, r, target = (randn(a.tokens, a.width).bfloat16() for _ in range(3))
    opt = torch.optim.SGD(block.parameters(), lr=1e-1)
    losses = []
    for _ in range(a.steps):
        opt.zero_grad()
        y, _ = block(x, r)
        loss = (y.float() - target.float()).square().mean()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    served = Int8MLPBlock(block)
    with torch.no_grad():
        y4, h4 = block(x, r)
        y8, h8 = served(x, r)
        out = {"losses": losses, "difference": float((y8.float() - y4.float()).norm() / y4.float().norm()),
               "same_residual": bool(torch.equal(h4, h8)),
               "nf4_ms": _time(lambda: block(x, r)), "int8_ms": _time(lambda: served(x, r)),
               "nf4_token_ms": _time(lambda: block(x[:1], r[:1])), "int8_token_ms": _time(lambda: served(x[:1], r[:1]))}
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")
    print(f"8-bit against 4-bit with adapters: {100 * out['difference']:.2f} % of the output's norm")
    print(f"{a.tokens} tokens: {out['nf4_ms']:.3f} ms with NF4 and adapters, {out['int8_ms']:.3f} ms in 8 bits")
    print(f"1 token: {out['nf4_token_ms']:.3f} ms with NF4 and adapters, {out['int8_token_ms']:.3f} ms in 8 bits")
    return out


if __name__ == "__main__":
    main()
