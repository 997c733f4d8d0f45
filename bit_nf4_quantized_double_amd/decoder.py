"""A decoder trained and evaluated with this package's operators: token rows,
layers of an attention and an MLP block, a norm, and a frozen output head.

:class:`AttentionBlock` is the attention half of a layer (RMS norm with the
residual, query, key and value projections, rotary positions, attention of packed
sequences, output projection), :class:`Decoder` the whole: the linears with frozen
NF4 weights and an adapter each, token rows and head frozen in bf16.
:meth:`Decoder.loss` trains it on packed sequences without the head's logits;
:meth:`Decoder.score` gives the loss of each token, of whole sequences or of new
tokens over a :class:`Cache`.

    python -m bit_nf4_quantized_double_amd.decoder [--width 1024 --layers 2 --tokens 2048]

trains a small number of steps on synthetic sequences, scores one of them at once
and token by token over a cache, and prints the losses, how far the two scores
differ and the time of a step of each kind.
"""

from __future__ import annotations

import argparse

import torch

from . import attention, cross_entropy, qlora, rotary, rows
from .block import MLPBlock, _time


def packed(lengths, start=None, device="cuda"):
    """(cu, positions) of sequences one after another: where each begins and ends,
    and each token's place in its own (on from ``start``, a number for each)."""
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    start = [0] * len(lengths) if start is None else start
    places = [torch.arange(a, a + n, dtype=torch.int32) for a, n in zip(start, lengths)]
    positions = torch.cat(places) if places else torch.empty(0, dtype=torch.int32)
    return torch.tensor(cu, dtype=torch.int32, device=device), positions.to(device)


class Cache:
    """Keys and values of ``sequences`` sequences with room for ``room`` tokens
    each, for every layer."""

    def __init__(self, layers: int, sequences: int, room: int, kv_heads: int, head_dim: int, dtype=torch.bfloat16,
                 device="cuda"):
        shape = (layers, sequences * room, kv_heads, head_dim)
        self.k, self.v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
        self.room, self.used = room, [0] * sequences
        self.cu = torch.arange(sequences + 1, dtype=torch.int32, device=device) * room
        self.lengths = torch.zeros(sequences, dtype=torch.int32, device=device)

    def extend(self, new):
        """Room for new[i] tokens of sequence i: returns (cu, positions) of the new
        tokens; the layers then put their keys and values there."""
        if len(new) != len(self.used):
            raise ValueError(f"{len(self.used)} sequences in the cache, {len(new)} given")
        if any(n < 0 or u + n > self.room for n, u in zip(new, self.used)):
            raise ValueError(f"a sequence is longer than the cache's room of {self.room}")
        cu, positions = packed(new, self.used, self.k.device)
        first = torch.arange(len(new), device=self.k.device) * self.room
        sizes = torch.tensor(new, device=self.k.device)
        self.rows = torch.repeat_interleave(first, sizes, output_size=sum(new)) + positions
        self.used = [u + n for n, u in zip(new, self.used)]
        self.lengths.copy_(torch.tensor(self.used, dtype=torch.int32))
        return cu, positions

    def put(self, layer: int, k: torch.Tensor, v: torch.Tensor):
        """A layer's new keys and values; returns all of them.  Not for training:
        the cache would hold one call's graph into the next."""
        if torch.is_grad_enabled() and (k.requires_grad or v.requires_grad):
            raise RuntimeError("a cache keeps no gradients: call under torch.no_grad()")
        self.k[layer].index_copy_(0, self.rows, k)
        self.v[layer].index_copy_(0, self.rows, v)
        return self.k[layer], self.v[layer]


class AttentionBlock(torch.nn.Module):
    """(x, residual) -> (o(attention(q(n), k(n), v(n))), h) with h = x + residual
    and n the RMS norm of h; queries and keys are turned to their positions.  The
    weights are fp32 [n_out, width] and frozen as NF4, the adapters and the norm's
    weight are trained, in bf16."""

    def __init__(self, w_q: torch.Tensor, w_k: torch.Tensor, w_v: torch.Tensor, w_o: torch.Tensor, heads: int, kv_heads: int,
                 freqs: rotary.Frequencies, r: int = 16, alpha: float = 32.0, eps: float = 1e-5):
        super().__init__()
        width, inner = w_o.shape
        if heads < 1 or kv_heads < 1 or heads % kv_heads or inner % heads:
            raise ValueError("w_o's columns must be whole heads, heads a multiple of kv_heads")
        d = inner // heads
        if w_q.shape != (inner, width) or w_k.shape != (kv_heads * d, width) or w_v.shape != w_k.shape:
            raise ValueError("w_q must be [heads * head_dim, width], w_k and w_v [kv_heads * head_dim, width]")
        if freqs.rot > d:
            raise ValueError(f"{freqs.rot} values to turn in heads of {d}")
        self.heads, self.kv_heads, self.head_dim, self.freqs = heads, kv_heads, d, freqs
        self.norm = rows.RMSNorm(width, eps, device=w_q.device)
        self.q, self.k, self.v, self.o = (qlora.QLoRALinear(w, r, alpha) for w in (w_q, w_k, w_v, w_o))

    def forward(self, x, residual, cu, positions, cache: Cache | None = None, layer: int = 0):
        """Sequences packed one after another (:func:`packed`), or, with a cache,
        the new tokens of its sequences (:meth:`Cache.extend`)."""
        y, h = self.norm(x, residual)
        q, k, v = (lin(y).unflatten(-1, (-1, self.head_dim)) for lin in (self.q, self.k, self.v))
        q, k = rotary.rotary(q, k, positions, self.freqs)
        if cache is None:
            o = attention.attention(q, k, v, cu)
        else:
            keys, values = cache.put(layer, k, v)
            o = attention.attention(q, keys, values, cu, cache.cu, lengths_k=cache.lengths)
        return self.o(o.flatten(-2)), h


class Decoder(torch.nn.Module):
    """``layers``: pairs of an :class:`AttentionBlock` and an MLPBlock; ``token_rows`` and
    ``head`` are [vocabulary, width], frozen."""

    def __init__(self, token_rows: torch.Tensor, layers, head: torch.Tensor, eps: float = 1e-5):
        super().__init__()
        if token_rows.shape[1] != head.shape[1]:
            raise ValueError("token rows and head must have the same width")
        self.register_buffer("token_rows", token_rows)
        self.register_buffer("head", head)
        self.layers = torch.nn.ModuleList(torch.nn.ModuleList(pair) for pair in layers)
        self.norm = rows.RMSNorm(head.shape[1], eps, device=head.device)

    def cache(self, sequences: int, room: int) -> Cache:
        a = self.layers[0][0]
        return Cache(len(self.layers), sequences, room, a.kv_heads, a.head_dim, self.head.dtype, self.head.device)

    def forward(self, tokens, cu, positions, cache: Cache | None = None):
        """Hidden states [tokens, width] as the head reads them."""
        x = self.token_rows[tokens]
        h = torch.zeros_like(x)
        for i, (attend, mlp) in enumerate(self.layers):
            x, h = attend(x, h, cu, positions, cache, i)
            x, h = mlp(x, h)
        return self.norm(x, h)[0]

    def loss(self, tokens, targets, cu, positions, ignore_index: int = -100):
        """The mean loss of packed sequences."""
        return cross_entropy.linear_cross_entropy(self(tokens, cu, positions), self.head, targets, ignore_index=ignore_index)

    @torch.no_grad()
    def score(self, tokens, targets, cu, positions, cache: Cache | None = None, ignore_index: int = -100):
        """The loss of each token, fp32."""
        return cross_entropy.linear_cross_entropy_fwd(self(tokens, cu, positions, cache), self.head, targets,
                                                      ignore_index=ignore_index)[0]


def synthetic(width: int, hidden: int, heads: int, kv_heads: int, vocabulary: int, layers: int, r: int = 16,
              alpha: float = 32.0, seed: int = 0) -> Decoder:
    """A decoder of random weights."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape, scale=0.02):
        return torch.randn(shape, generator=gen, device="cuda") * scale

    d = width // heads
    freqs = rotary.frequencies(d)
    pairs = []
    for _ in range(layers):
        a = AttentionBlock(randn(width, width), randn(kv_heads * d, width), randn(kv_heads * d, width), randn(width, width),
                           heads, kv_heads, freqs, r, alpha)
        m = MLPBlock(randn(hidden, width), randn(hidden, width), randn(width, hidden), r, alpha)
        pairs.append((a, m))
    return Decoder(randn(vocabulary, width, scale=1.0).bfloat16(), pairs, randn(vocabulary, width, scale=width ** -0.5).bfloat16())


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2816)
    ap.add_argument("--heads", type=int, default=8)
    ap.add_argument("--kv-heads", type=int, default=2)
    ap.add_argument("--vocabulary", type=int, default=32000)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args(argv)
    model = synthetic(a.width, a.hidden, a.heads, a.kv_heads, a.vocabulary, a.layers)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    lengths = [a.tokens // 2, a.tokens // 3]
    lengths.append(a.tokens - sum(lengths))
    cu, positions = packed(lengths)
    tokens = torch.randint(0, a.vocabulary, (a.tokens,), generator=gen, device="cuda")
    targets = tokens.roll(-1)
    targets[(cu[1:] - 1).long()] = -100  # the last token of a sequence has none
    opt = torch.optim.SGD(model.parameters(), lr=1.0)

    def step():
        opt.zero_grad()
        loss = model.loss(tokens, targets, cu, positions)
        loss.backward()
        opt.step()
        return loss

    losses = [step().item() for _ in range(a.steps)]
    # the last sequence at once, and token by token behind a prompt of all but 8 tokens
    n = lengths[-1]
    last, goal = tokens[-n:], targets[-n:]
    whole = model.score(last, goal, *packed([n]))
    cache = model.cache(1, n)
    parts, at = [], 0
    for m in [max(1, n - 8)] + [1] * min(8, n - 1):
        parts.append(model.score(last[at:at + m], goal[at:at + m], *cache.extend([m]), cache))
        at += m
    by_token = torch.cat(parts)
    one, new = model.cache(1, n + 64), last[:1]
    model.score(last, goal, *one.extend([n]), one)
    ends = one.extend([1])
    out = {"losses": losses, "difference": float((by_token - whole).abs().max()),
           "step_ms": _time(step), "token_ms": _time(lambda: model.score(new, new, *ends, one))}
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps of {a.tokens} tokens")
    print(f"scored at once and token by token over a cache: the losses differ by {out['difference']:.4f} at most")
    print(f"{out['step_ms']:.3f} ms a training step, {out['token_ms']:.3f} ms for a token behind {n}")
    return out


if __name__ == "__main__":
    main()
