"""Rotary positions, attention and the head's loss run together, with the NF4
linears, norm and SwiGLU: a decoder trained on packed sequences and scored over a
cache."""

import numpy as np
import pytest
import torch

from bit_nf4_quantized_double_amd import block, decoder, qlora, rotary
from rows_util import f64, need_gpu, rand

pytestmark = pytest.mark.gpu


def _model(layers=2, seed=0):
    m = decoder.synthetic(128, 192, 4, 2, 300, layers, r=8, alpha=16.0, seed=seed)
    with torch.no_grad():
        for i, p in enumerate(m.parameters()):
            if p.dim() == 2 and not bool(p.any()):  # adapters' B start at zero
                p.copy_(rand(tuple(p.shape), seed + i, scale=0.05))
    return m


def _inputs(lengths, seed=0):
    n = sum(lengths)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    tokens, targets = (torch.randint(0, 300, (n,), device="cuda", generator=gen) for _ in range(2))
    targets[::7] = -100
    return (tokens, targets, *decoder.packed(lengths))


def _losses64(m, tokens, targets, lengths, other=None):
    """The model in 64 bits, sequence by sequence.  ``other``: {parameter: its value}."""
    value = lambda p: (other or {}).get(p, p.detach().double())

    def _linear64(lin, x):
        return x @ qlora.dequant(lin.w).double().t() + (lin.alpha / lin.r) * (x @ value(lin.A).t()) @ value(lin.B).t()

    def _norm64(norm, h):
        return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + norm.eps) * value(norm.weight)

    out, at = [], 0
    for n in lengths:
        x, h = m.token_rows[tokens[at:at + n]].double(), 0.0
        for a, mlp in m.layers:
            h = x + h
            y = _norm64(a.norm, h)
            q, k, v = (_linear64(lin, y).unflatten(-1, (-1, a.head_dim)) for lin in (a.q, a.k, a.v))
            f = 10000.0 ** (-2.0 * torch.arange(a.head_dim // 2, device="cuda").double() / a.head_dim)
            angle = torch.arange(n, device="cuda").double()[:, None, None] * f
            c, s, half = angle.cos(), angle.sin(), a.head_dim // 2
            q, k = (torch.cat([t[..., :half] * c - t[..., half:] * s, t[..., half:] * c + t[..., :half] * s], -1) for t in (q, k))
            o = torch.empty_like(q)
            hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
            for i in range(a.heads):
                j = i // (a.heads // a.kv_heads)
                z = (q[:, i].contiguous() @ k[:, j].t().contiguous()) * a.head_dim ** -0.5
                o[:, i] = torch.softmax(z.masked_fill(hidden, -float("inf")), -1) @ v[:, j].contiguous()
            x = _linear64(a.o, o.flatten(-2))
            h = x + h
            y = _norm64(mlp.norm, h)
            g = _linear64(mlp.gate, y)
            x = _linear64(mlp.down, g * torch.sigmoid(g) * _linear64(mlp.up, y))
        z = _norm64(m.norm, x + h) @ m.head.double().t()
        y = targets[at:at + n]
        loss = torch.logsumexp(z, -1) - z.gather(1, y.clamp(min=0)[:, None])[:, 0]
        out.append(torch.where(y >= 0, loss, 0.0))
        at += n
    return torch.cat(out)


def test_losses_against_64_bits():
    """Some twenty roundings to bf16 a token on the way (2^-8 each at most, half of
    that or less on average, independent), which reach logits of about 1 as their
    root mean square: 2^-8 sqrt(20) = 0.02; 5 times that for the worst of some
    hundred tokens."""
    need_gpu()
    m, lengths = _model(), [70, 1, 33]
    tokens, targets, cu, positions = _inputs(lengths)
    got = m.score(tokens, targets, cu, positions)
    want = _losses64(m, tokens, targets, lengths)
    assert float((got.double() - want).abs().max()) <= 0.1
    assert float((got.double() - want).square().mean().sqrt()) <= 0.02
    n = int((targets >= 0).sum())
    assert abs(m.loss(tokens, targets, cu, positions).item() - float(want.sum()) / n) <= 0.02


def test_gradients_against_differences():
    """Along the gradient of a parameter of each kind: its own slope against that of
    the model in 64 bits, by central differences (over a millionth of the step that
    would change the loss by a twentieth: the third derivative and 2^-53 of the loss
    are far below).  The gradient has gone through some forty roundings to bf16, each
    2^-8 at most and independent: 2^-8 sqrt(40) = 0.025 of it, and twice that here."""
    need_gpu()
    m, lengths = _model(), [70, 1, 33]
    args = _inputs(lengths, 3)
    m.loss(*args).backward()
    n = int((args[1] >= 0).sum())
    a, mlp = m.layers[0]
    for name, p in (("q.A", a.q.A), ("k.B", a.k.B), ("v.A", a.v.A), ("o.B", a.o.B), ("norm", a.norm.weight),
                    ("gate.A", mlp.gate.A), ("final norm", m.norm.weight), ("second q.A", m.layers[1][0].q.A)):
        g = p.grad.double()
        v = g / g.norm().square() * 0.05e-6
        hi, lo = (float(_losses64(m, *args[:2], lengths, {p: p.detach().double() + s * v}).sum()) / n for s in (1, -1))
        assert abs((hi - lo) / 1e-7 - 1.0) <= 0.05, (name, (hi - lo) / 1e-7)


def test_packing_does_not_mix_sequences():
    """A sequence's losses packed among others and by itself."""
    need_gpu()
    m, lengths = _model(), [40, 5, 90]
    tokens, targets, cu, positions = _inputs(lengths, 5)
    got = m.score(tokens, targets, cu, positions)
    at = 0
    for n in lengths:
        alone = m.score(tokens[at:at + n], targets[at:at + n], *decoder.packed([n]))
        # other kernels for other numbers of tokens: roundings as above
        assert float((got[at:at + n] - alone).abs().max()) <= 0.1
        at += n
    # and another sequence's tokens change nothing at all
    other = tokens.clone()
    other[:40] = (other[:40] + 1) % 300
    assert torch.equal(m.score(other, targets, cu, positions)[40:], got[40:])


def test_cache_token_by_token():
    """Prompts of different lengths, then single tokens of both sequences."""
    need_gpu()
    m, lengths, prompt = _model(), [60, 23], [50, 13]
    tokens, targets, cu, positions = _inputs(lengths, 7)
    whole = m.score(tokens, targets, cu, positions)
    cache = m.cache(2, 64)
    got = torch.empty_like(whole)
    first = [0, 60]

    def feed(new):
        at = torch.cat([torch.arange(f + u, f + u + n) for f, u, n in zip(first, cache.used, new)]).cuda()
        got[at] = m.score(tokens[at], targets[at], *cache.extend(new), cache)

    feed(prompt)
    for _ in range(10):
        feed([1, 1])
    assert cache.used == lengths
    assert float((got - whole).abs().max()) <= 0.1  # roundings as above
    with pytest.raises(ValueError, match="longer than"):
        cache.extend([5, 0])
    with pytest.raises(ValueError, match="sequences"):
        cache.extend([1])


def test_cache_without_new_tokens_and_with_gradients():
    need_gpu()
    m = _model()
    tokens, targets, _, _ = _inputs([5, 0], 3)
    cache, other = m.cache(2, 8), m.cache(2, 8)
    m.score(tokens, targets, *cache.extend([5, 0]), cache)
    none = m.score(tokens[:0], targets[:0], *cache.extend([0, 0]), cache)
    assert none.shape == (0,) and cache.used == [5, 0]
    with pytest.raises(RuntimeError, match="no gradients"):
        m(tokens, *other.extend([5, 0]), other)


def test_command():
    need_gpu()
    out = decoder.main(["--width", "128", "--hidden", "256", "--heads", "4", "--vocabulary", "500", "--tokens", "200",
                        "--steps", "2"])
    assert np.isfinite(out["losses"]).all() and out["difference"] <= 0.1


def test_refusals():
    need_gpu()
    w = lambda *s: rand(s, 1, torch.float32)
    f = rotary.frequencies(32)
    with pytest.raises(ValueError, match="whole heads"):
        decoder.AttentionBlock(w(128, 128), w(64, 128), w(64, 128), w(128, 128), 4, 3, f)
    with pytest.raises(ValueError, match="w_q must be"):
        decoder.AttentionBlock(w(128, 128), w(128, 128), w(64, 128), w(128, 128), 4, 2, f)
    with pytest.raises(ValueError, match="to turn in heads"):
        decoder.AttentionBlock(w(128, 128), w(64, 128), w(64, 128), w(128, 128), 4, 2, rotary.frequencies(64))
    with pytest.raises(ValueError, match="same width"):
        decoder.Decoder(w(10, 64), [], w(10, 128))
