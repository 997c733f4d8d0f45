"""Rotary positions, attention and the head's loss through the bounds-checked
library: the same bits as the normal one, and no access out of range, also where
what lies behind the buffers is another's."""

import pytest
import torch

from bit_nf4_quantized_double_amd import attention, cross_entropy, qlora, rotary
from decoder_util import cu
from rows_util import need_gpu, rand, strided

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def both(run):
    """run() through both libraries: equal bits, nothing out of range."""
    a = run()
    torch.cuda.synchronize()
    with qlora.library(qlora.LIB_CHECKED_PATH):
        qlora.debug_oob_count(reset=True)
        b = run()
        torch.cuda.synchronize()
        assert qlora.debug_oob_count(reset=True) == 0
    for i, (x, y) in enumerate(zip(a, b)):
        ints = torch.int16 if x.dtype in (BF16, F16) else torch.int32
        assert torch.equal(x.view(ints), y.view(ints)), i


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("t,h,hk,d,rot,apart", [(1, 1, 1, 2, 2, 0), (37, 6, 2, 64, 64, 0), (37, 6, 2, 64, 32, 8),
                                                (5, 3, 1, 33, 10, 1), (700, 10, 2, 80, 32, 0)])
def test_rotary(t, h, hk, d, rot, apart, dtype):
    need_gpu()
    wide = rand((t, (h + hk) * d + apart), 1, dtype)[:, apart:]
    q, k = wide[:, :h * d].unflatten(1, (h, d)), wide[:, h * d:].unflatten(1, (hk, d))
    pos, f = torch.arange(t, device="cuda") * 7, rotary.frequencies(rot)
    for interleaved in (False, True):
        both(lambda: (*rotary.rotate(q, k, pos, f, interleaved=interleaved), *rotary.rotate_bwd(q, k, pos, f)))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lq,lk,h,hk,d,causal", [
    ([1], [1], 1, 1, 8, True), ([129], [129], 7, 1, 72, True), ([100, 0, 31, 300], [100, 0, 31, 300], 4, 2, 128, True),
    ([40, 70], [10, 0], 2, 1, 64, True), ([70, 20], [10, 3], 5, 5, 128, False), ([1, 1, 1], [700, 30, 2000], 8, 2, 128, True),
    ([200], [2100], 2, 2, 128, True), ([33, 64], [500, 64], 48, 3, 40, True)])
def test_attention(lq, lk, h, hk, d, causal, dtype):
    need_gpu()
    q, do = rand((sum(lq), h, d), 1, dtype), rand((sum(lq), h, d), 2, dtype)
    k, v = rand((sum(lk), hk, d), 3, dtype), rand((sum(lk), hk, d), 4, dtype)

    def run():
        o, lse = attention.attention_fwd(q, k, v, cu(lq), cu(lk), causal=causal)
        return (o, lse, *attention.attention_bwd(do, q, k, v, o, lse, cu(lq), cu(lk), causal=causal))

    both(run)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("h,hk,d", [(8, 1, 128), (4, 2, 72), (16, 1, 64), (3, 3, 128)])
def test_attention_heads_first(h, hk, d, dtype):
    """[heads, tokens, d] tensors, the last head at the end of its buffer: whole tiles of
    dK and dV read rows of heads that are far apart."""
    need_gpu()
    t = 517
    q, do = (rand((h, t, d), i, dtype).transpose(0, 1) for i in (1, 2))
    k, v = (rand((hk, t, d), i, dtype).transpose(0, 1) for i in (3, 4))

    def run():
        o, lse = attention.attention_fwd(q, k, v, cu([t]))
        return (o, lse, *attention.attention_bwd(do, q, k, v, o, lse, cu([t])))

    both(run)


@pytest.mark.parametrize("ends", [[0, 500], [-7, 40, 30, 90], [90, 10, 2 ** 31 - 1], [-(2 ** 31), 5, 5]])
def test_ends_outside_the_tensors(ends):
    """cu that does not ascend or lies outside, and lengths that do: whatever comes
    out, nothing outside the tensors is read or written."""
    need_gpu()
    t, h, hk, d = 77, 4, 2, 64
    q, do = rand((t, h, d), 1), rand((t, h, d), 2)
    k, v = rand((t, hk, d), 3), rand((t, hk, d), 4)
    c = torch.tensor(ends, dtype=torch.int32, device="cuda")
    n = torch.tensor([10 ** 6, -5, 3][:len(ends) - 1], dtype=torch.int32, device="cuda")
    with qlora.library(qlora.LIB_CHECKED_PATH):
        qlora.debug_oob_count(reset=True)
        for lengths in (None, n):
            o, lse = attention.attention_fwd(q, k, v, c, lengths_q=lengths)
            attention.attention_bwd(do, q, k, v, o, lse, c, lengths_q=lengths)
            attention.attention_fwd(q[:2], k, v, c, c.flip(0), lengths_k=lengths)
        torch.cuda.synchronize()
        assert qlora.debug_oob_count(reset=True) == 0


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,k,v,apart", [(1, 8, 1, 0), (17, 72, 129, 0), (200, 136, 1000, 5), (300, 64, 5003, 0), (64, 4096, 300, 8)])
def test_cross_entropy(m, k, v, apart, dtype):
    need_gpu()
    x, w = rand((m, k), 1, dtype), rand((v, k), 2, dtype, 0.1)
    if apart:
        x, w = strided(x, apart, 3), strided(w, 8, 8)
    y = torch.randint(0, v, (m,), device="cuda")
    y[::3] = -100
    y[1::5] = 2 ** 50
    both(lambda: (*cross_entropy.linear_cross_entropy_fwd(x, w, y),
                  *cross_entropy.linear_cross_entropy_grad(x, w, y, torch.ones(m, device="cuda"))))
    g = rand((m, k), 3, dtype)
    both(lambda: (cross_entropy.scale_rows(g, torch.arange(m, dtype=torch.float32, device="cuda")),))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,k,v", [(1, 8, 1), (17, 72, 129), (8200, 64, 300)])
def test_cross_entropy_in_units(m, k, v, dtype):
    need_gpu()
    x, w = rand((m, k), 1, dtype), rand((v, k), 2, dtype, 0.1)
    y = torch.randint(0, v, (m,), device="cuda")
    y[1::3] = -100
    y[2::5] = 2 ** 50
    both(lambda: cross_entropy.linear_cross_entropy_units(x, w, y))
