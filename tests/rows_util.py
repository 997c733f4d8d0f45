"""Inputs and error bounds shared by the tests of the row-wise operators and
the int8 product.

Bounds.  A 16-bit output is one rounding to nearest (relative error at most
half a spacing, U = 2^-8 for bf16 and 2^-11 for fp16; half the spacing of
subnormals below the normal range) of a value computed in fp32 from exact
inputs.  Each fp32 operation adds at most 2^-24 of the magnitude of what it
produces; a sum of n terms in any order adds at most n 2^-24 of the sum of the
terms' magnitudes, and in the kernels' order (16 or 32 terms in a row, then
halves) at most 64 of them.  So

    |got - ref| <= U |ref| + TINY + OPS 2^-24 mag,

with mag the sum of the magnitudes of the terms that make up the value and
OPS = 128 (more than twice the operations on any path).
"""

import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
E32 = 128 * 2.0 ** -24


def need_gpu():
    import pytest
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rand(shape, seed, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def f64(t) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def close16(got: torch.Tensor, ref: np.ndarray, mag, what=""):
    """A 16-bit output against its reference, by the bound above."""
    g, u, tiny = f64(got), U[got.dtype], TINY[got.dtype]
    bound = u * np.abs(ref) * (1 + 2.0 ** -10) + tiny + E32 * mag * (1 + u)
    bad = ~(np.abs(g - ref) <= bound)
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside the bound, first at {at}: got {g[at]}, "
                             f"want {ref[at]} within {bound[at]}")


def codes_of(q) -> np.ndarray:
    """The integer codes of Int8Rows or Int8Weight, [rows, k]: the values at scale 1."""
    from bit_nf4_quantized_double_amd import int8, rows
    ones = torch.ones_like(q.scale)
    if isinstance(q, rows.Int8Rows):
        return f64(rows.dequant_rows(rows.Int8Rows(q.codes, ones, q.m, q.k, torch.bfloat16)))
    return f64(int8.dequant_weight(int8.Int8Weight(q.codes, ones, q.n_out, q.k_in)))


def strided(t: torch.Tensor, pad: int, offset: int = 0) -> torch.Tensor:
    """The same matrix as a slice of a wider one: rows `pad` elements further
    apart, starting `offset` elements in; what is around it is NaN."""
    m, k = t.shape
    wide = torch.full((m, k + pad), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, offset:offset + k] = t
    return wide[:, offset:offset + k]
