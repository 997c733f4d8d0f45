"""Attention of packed sequences against 64 bits, forward and backward, and its
masks, lengths, strides and edges.  Bounds: decoder_util.py."""

import numpy as np
import pytest
import torch

from bit_nf4_quantized_double_amd import attention, rotary
from decoder_util import attention_reference, close, cu, starts
from rows_util import U, f64, need_gpu, rand

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16

# (queries, keys of each sequence, heads, key heads, head_dim, causal)
SHAPES = [
    ([1], [1], 1, 1, 128, True),
    ([1], [1], 2, 1, 8, True),
    ([5], [5], 1, 1, 64, True),
    ([33], [33], 3, 3, 72, True),
    ([64], [64], 2, 2, 128, False),
    ([128], [128], 4, 1, 128, True),
    ([129], [129], 2, 2, 96, True),
    ([300], [300], 2, 1, 128, True),
    ([257], [257], 7, 1, 80, True),
    ([100, 1, 0, 31, 200], [100, 1, 0, 31, 200], 4, 2, 128, True),
    ([0, 0, 3], [0, 7, 3], 2, 2, 64, True),
    ([40, 70], [10, 0], 2, 1, 64, True),        # rows that see nothing, a sequence without keys
    ([70, 20], [10, 3], 5, 5, 128, False),
    ([3, 1, 17], [190, 65, 400], 8, 2, 128, True),   # new tokens behind prefixes
    ([130], [500], 2, 2, 56, True),
    ([260, 5], [131, 260], 6, 3, 40, True),
    ([200], [2100], 2, 2, 128, True),           # keys split over workgroups of 128 rows
]


def _inputs(lq, lk, h, hk, d, dtype, seed=0):
    tq, tk = sum(lq), sum(lk)
    return (rand((tq, h, d), seed, dtype), rand((tk, hk, d), seed + 1, dtype), rand((tk, hk, d), seed + 2, dtype),
            rand((tq, h, d), seed + 3, dtype))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lq,lk,h,hk,d,causal", SHAPES)
def test_forward_and_backward(lq, lk, h, hk, d, causal, dtype):
    need_gpu()
    q, k, v, do = _inputs(lq, lk, h, hk, d, dtype)
    want = attention_reference(q, k, v, lq, lk, causal, do=do)
    o, lse = attention.attention_fwd(q, k, v, cu(lq), cu(lk), causal=causal)
    close(lse, want["lse"], "lse")
    close(o, want["o"], "o")
    dq, dk, dv = attention.attention_bwd(do, q, k, v, o, lse, cu(lq), cu(lk), causal=causal)
    close(dv, want["dv"], "dv")
    close(dk, want["dk"], "dk")
    close(dq, want["dq"], "dq")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lq,lk,causal", [([300], [0], True), ([300], [0], False), ([1000], [10], True),
                                          ([260, 400, 70], [0, 20, 70], True)])
def test_whole_tiles_that_see_nothing(lq, lk, causal, d, dtype):
    """Row tiles none of whose rows see a key: their dQ is zero, whatever a workgroup
    that ran before has left in LDS."""
    need_gpu()
    h, hk = 4, 2
    q, k, v, do = _inputs(lq, lk, h, hk, d, dtype)
    want = attention_reference(q, k, v, lq, lk, causal, do=do)
    fill = [-abs(x) for x in _inputs([4096], [4096], h, hk, d, dtype, 9)]  # negative numbers all over LDS
    o, lse = attention.attention_fwd(q, k, v, cu(lq), cu(lk), causal=causal)
    fo, fl = attention.attention_fwd(*fill[:3], cu([4096]))
    attention.attention_bwd(fill[3], *fill[:3], fo, fl, cu([4096]))
    dq, dk, dv = attention.attention_bwd(do, q, k, v, o, lse, cu(lq), cu(lk), causal=causal)
    for at, n, m in zip(starts(lq), lq, lk):
        blind = n if m == 0 else max(n - m, 0) if causal else 0
        assert bool((dq[at:at + blind] == 0).all())
    for got, name in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        close(got, want[name], name)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("new,room,lk,h,hk,d", [
    (1, 40, [40, 1, 17], 4, 4, 128), (1, 700, [700, 513, 512, 33, 1, 0], 16, 2, 128), (4, 300, [300, 4, 257], 8, 1, 64),
    (1, 5000, [5000, 4097], 8, 8, 128), (2, 3000, [2999], 7, 1, 72)])
def test_few_tokens_over_a_cache(new, room, lk, h, hk, d, dtype):
    """Few queries, sequences with room behind them, keys split over workgroups;
    what is behind a sequence is NaN."""
    need_gpu()
    n = len(lk)
    q = rand((n * new, h, d), 1, dtype)
    k, v = rand((n * room, hk, d), 2, dtype), rand((n * room, hk, d), 3, dtype)
    for i, m in enumerate(lk):
        k[i * room + m:(i + 1) * room] = float("nan")
        v[i * room + m:(i + 1) * room] = float("nan")
    ends = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    o, lse = attention.attention_fwd(q, k, v, ends * new, ends * room, lengths_k=torch.tensor(lk, dtype=torch.int32, device="cuda"))
    want = attention_reference(q, k, v, [new] * n, lk, True, at_q=np.arange(n) * new, at_k=np.arange(n) * room)
    close(lse, want["lse"], "lse")
    close(o, want["o"], "o")


def test_plans_cover_split_keys():
    """The cases above take both kernels, split and unsplit."""
    need_gpu()
    ends = lambda n, m: torch.arange(n + 1, dtype=torch.int32, device="cuda") * m
    q = lambda t, h: torch.empty(t, h, 128, dtype=BF16, device="cuda")
    assert attention.plan(q(6, 16), q(4200, 2), ends(6, 1))["rows"] == 32
    assert attention.plan(q(6, 16), q(4200, 2), ends(6, 1))["splits"] > 1
    assert attention.plan(q(200, 2), q(2100, 2), ends(1, 200)) == {"rows": 128, "splits": 5}
    assert attention.plan(q(300, 2), q(300, 1), ends(1, 300)) == {"rows": 128, "splits": 1}
    assert attention.plan(q(8192, 32), q(8192, 8), ends(1, 8192)) == {"rows": 128, "splits": 1}


def test_without_room_for_the_split():
    """A workspace is optional in the forward: unsplit, the same within rounding."""
    need_gpu()
    q, k, v = rand((1, 8, 128), 1), rand((3000, 2, 128), 2), rand((3000, 2, 128), 3)
    want = attention_reference(q, k, v, [1], [3000], True)
    import ctypes
    from bit_nf4_quantized_double_amd import qlora
    c, *h = attention._describe(q, k, v, cu([1]), cu([3000]), None, None, True, None, False)
    o, lse = torch.empty_like(q), torch.empty(1, 8, device="cuda")
    r = ctypes.byref
    oh = attention.check_heads(o, "O")
    qlora._check(qlora.lib().qlora_attention_fwd(r(c), *map(r, h), r(oh), lse.data_ptr(), None, 0,
                                                 torch.cuda.current_stream().cuda_stream), "fwd")
    close(o, want["o"], "o")
    close(lse, want["lse"], "lse")


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_padded_batch(dtype):
    """[n, room, heads, d] with lengths: padding is NaN, has no effect, and gets zeros."""
    need_gpu()
    n, room, h, hk, d, lens = 4, 96, 4, 2, 64, [96, 0, 41, 1]
    q, do = rand((n * room, h, d), 1, dtype), rand((n * room, h, d), 2, dtype)
    k, v = rand((n * room, hk, d), 3, dtype), rand((n * room, hk, d), 4, dtype)
    for t in (q, do, k, v):
        for i, m in enumerate(lens):
            t[i * room + m:(i + 1) * room] = float("nan")
    ends = torch.arange(n + 1, dtype=torch.int32, device="cuda") * room
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = attention.attention_fwd(q, k, v, ends, lengths_q=ln)
    grads = attention.attention_bwd(do, q, k, v, o, lse, ends, lengths_q=ln)
    want = attention_reference(q, k, v, lens, lens, True, do=do, at_q=np.arange(n) * room, at_k=np.arange(n) * room)
    for name, got in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
        close(got, want[name], name)


def test_tokens_of_no_sequence():
    """Before the first sequence and behind the last: zeros in new outputs, left as
    they are in given ones, forward and backward."""
    need_gpu()
    t, h, hk, d = 400, 4, 2, 128
    q, k, v, do = _inputs([t], [t], h, hk, d, BF16)
    ends = torch.tensor([3, 150, 150, 377], dtype=torch.int32, device="cuda")
    inside = torch.zeros(t, dtype=torch.bool)
    inside[3:377] = True
    o, lse = attention.attention_fwd(q, k, v, ends)
    new = (o, *attention.attention_bwd(do, q, k, v, o, lse, ends))
    assert all(bool((x[~inside] == 0).all()) and bool(torch.isfinite(x).all()) for x in new)
    assert bool((lse[~inside] == float("-inf")).all()) and bool(torch.isfinite(lse[inside]).all())
    marked = [torch.full_like(x, 7.0) for x in new]
    l2 = torch.full_like(lse, 7.0)
    attention.attention_fwd(q, k, v, ends, O=marked[0], lse=l2)
    attention.attention_bwd(do, q, k, v, o, lse, ends, dQ=marked[1], dK=marked[2], dV=marked[3])
    for x, y in zip(marked, new):
        assert bool((x[~inside] == 7.0).all()) and torch.equal(x[inside], y[inside])
    assert bool((l2[~inside] == 7.0).all()) and torch.equal(l2[inside], lse[inside])


def test_strided_views():
    """Slices of one projection's output, heads-first tensors, one broadcast key head."""
    need_gpu()
    t, h, hk, d = 200, 4, 2, 64
    qkv = rand((t, (h + 2 * hk) * d), 1)
    q, k, v = qkv[:, :h * d].view(t, h, d), qkv[:, h * d:(h + hk) * d].view(t, hk, d), qkv[:, (h + hk) * d:].view(t, hk, d)
    do = rand((h, t, d), 2).transpose(0, 1)
    o = torch.empty(h, t, d, dtype=BF16, device="cuda").transpose(0, 1)
    _, lse = attention.attention_fwd(q, k, v, cu([t]), O=o)
    want = attention_reference(q, k, v, [t], [t], True, do=do)
    close(o, want["o"], "o")
    for got, name in zip(attention.attention_bwd(do, q, k, v, o, lse, cu([t])), ("dq", "dk", "dv")):
        close(got, want[name], name)
    kb = k[:, :1].expand(t, hk, d)
    o2, _ = attention.attention_fwd(q, kb, v, cu([t]))
    close(o2, attention_reference(q, kb, v, [t], [t], True)["o"], "broadcast key head")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("t,h,hk,d", [(200, 2, 1, 128), (70, 1, 1, 64)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_what_is_masked_has_no_effect(t, h, hk, d, dtype, value):
    """An infinity or a NaN in token i's key, value, query or gradient reaches only
    what sees it: outputs of tokens before i (forward, dQ), and keys after i (dK,
    dV), are bit for bit as without it."""
    need_gpu()
    q, k, v, do = _inputs([t], [t], h, hk, d, dtype)
    ends = cu([t])

    def run(q, k, v, do):
        o, lse = attention.attention_fwd(q, k, v, ends)
        return (o, lse, *attention.attention_bwd(do, q, k, v, o, lse, ends))

    clean = run(q, k, v, do)
    for i in (1, 31, 66):
        for which in range(4):
            x = [y.clone() for y in (q, k, v, do)]
            x[which][i, 0, 5] = value
            got = run(*x)
            if which in (1, 2):  # key or value of token i
                for j in (0, 1, 2):
                    assert torch.equal(got[j][:i], clean[j][:i]), (i, which, j)
                # and everything that sees it is reached
                assert not torch.isfinite(got[0][i:, 0]).all(-1).any() or which == 1
            else:  # query or gradient of token i: keys after it do not see it
                for j in (3, 4):
                    assert torch.equal(got[j][i + 1:], clean[j][i + 1:]), (i, which, j)
                assert torch.equal(got[2][:i], clean[2][:i]) and torch.equal(got[2][i + 1:], clean[2][i + 1:])
                if which == 3:
                    assert not torch.isfinite(got[4][:i + 1, 0, 5]).any()


def test_large_scores():
    """Scores up to thousands: the running reference moves, nothing overflows."""
    need_gpu()
    lq, lk = [150], [400]
    q, k, v, do = _inputs(lq, lk, 2, 2, 64, BF16)
    q, k = q * 30, k * 30 * torch.linspace(0, 1, 400, device="cuda")[:, None, None].to(BF16)
    want = attention_reference(q, k, v, lq, lk, True, do=do)
    o, lse = attention.attention_fwd(q, k, v, cu(lq), cu(lk))
    close(o, want["o"], "o")
    close(lse, want["lse"], "lse")
    for got, name in zip(attention.attention_bwd(do, q, k, v, o, lse, cu(lq), cu(lk)), ("dq", "dk", "dv")):
        close(got, want[name], name)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("tq,h,hk", [(1, 2, 2), (2, 64, 64), (200, 2, 1), (300, 128, 2)])
@pytest.mark.parametrize("sink", [0, 1777, 4096])
@pytest.mark.parametrize("gap", [8.0, 17.5, 22.0])
def test_many_small_weights(gap, sink, tq, h, hk, dtype):
    """One key far above 4096 others, its value zero: what the others add up to is
    all there is of O.  Scores are exact.  A weight is off by U of itself, and in fp16
    by at most half the smallest step times 2^-12: 2^-37 of the largest."""
    need_gpu()
    tk, d = 4097, 64
    q, k, v = rand((tq, h, d), 1, dtype), torch.zeros((tk, hk, d), dtype=dtype, device="cuda"), rand((tk, hk, d), 3, dtype)
    q[..., 0], k[sink, :, 0] = 4.0, gap / 4
    v = v.abs() + 0.5
    v[sink] = 0
    o, lse = attention.attention_fwd(q, k, v, cu([tq]), cu([tk]), causal=False, scale=1.0)
    p, V = np.exp(-gap), f64(v)
    total = 1 + 4096 * p
    want = np.broadcast_to(np.repeat(p * V.sum(0) / total, h // hk, 0), (tq, h, d))
    assert np.abs(f64(lse) - (gap + np.log(total))).max() <= 2.0 ** -20 * (1 + gap)
    bound = (U[dtype] * 2 + 2.0 ** -19) * want
    if dtype == F16:
        bound = bound + 2.0 ** -37 * np.repeat(V.sum(0), h // hk, 0) / total
    close(o, (want, bound), "o")


@pytest.mark.parametrize("loss_scale", [1.0, 2.0 ** 14, 2.0 ** -14])
def test_f16_gradients_in_range(loss_scale):
    """fp16 with gradients near either end of its range."""
    need_gpu()
    t = 500
    q, k, v, do = _inputs([t], [t], 2, 1, 64, F16)
    do = (do * 0.25 * loss_scale).to(F16)
    o, lse = attention.attention_fwd(q, k, v, cu([t]))
    want = attention_reference(q, k, v, [t], [t], True, do=do)
    for got, name in zip(attention.attention_bwd(do, q, k, v, o, lse, cu([t])), ("dq", "dk", "dv")):
        assert bool(torch.isfinite(got).all())
        close(got, want[name], name)


def test_same_bits_every_time():
    need_gpu()
    lq = [300, 70, 5]
    q, k, v, do = _inputs(lq, lq, 8, 2, 128, BF16)

    def run():
        o, lse = attention.attention_fwd(q, k, v, cu(lq))
        return (o, lse, *attention.attention_bwd(do, q, k, v, o, lse, cu(lq)))

    a = run()
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(a, run()))


def test_autograd_against_differences():
    """The loss' change along the gradient of each input against the step it predicts."""
    need_gpu()
    lq, lk = [60, 9], [80, 9]
    q, k, v, do = _inputs(lq, lk, 4, 2, 64, BF16)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    attention.attention(*leaves, cu(lq), cu(lk)).backward(do)

    def loss(*x):
        return float((f64(attention.attention(*x, cu(lq), cu(lk))) * f64(do)).sum())

    for i, x in enumerate(leaves):
        g = x.grad.double()
        v_ = g / g.norm() * x.detach().double().norm() * 0.05
        hi, lo = ([y.detach() for y in leaves] for _ in range(2))
        hi[i], lo[i] = (x.detach().double() + v_).to(BF16), (x.detach().double() - v_).to(BF16)
        want = float((g * (hi[i].double() - lo[i].double())).sum())
        # outputs and gradients rounded to bf16 (2^-8 each, independent over the entries), and the step's curvature
        assert abs(loss(*hi) - loss(*lo) - want) <= 0.05 * abs(want)


def test_autograd_copies_what_is_not_aligned():
    need_gpu()
    t, h, d = 50, 2, 64
    wide = rand((t, h, d + 3), 1)
    x = wide[..., 1:d + 1]
    k, v = rand((t, h, d), 2), rand((t, h, d), 3)
    a = x.detach().requires_grad_()
    b = x.detach().contiguous().requires_grad_()
    attention.attention(a, k, v, cu([t])).sum().backward()
    attention.attention(b, k, v, cu([t])).sum().backward()
    assert torch.equal(a.grad, b.grad)


def test_in_a_graph():
    """Captured once, replayed on new inputs and lengths; eager work between."""
    need_gpu()
    h, hk, d, t = 4, 2, 128, 260
    q, k, v, do = _inputs([t], [t], h, hk, d, BF16)
    ends = cu([200, 60])

    def run():
        o, lse = attention.attention_fwd(q, k, v, ends)
        return (o, lse, *attention.attention_bwd(do, q, k, v, o, lse, ends))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for seed, lens in ((10, [200, 60]), (20, [1, 259]), (30, [100, 100])):
        for x, y in zip((q, k, v, do), _inputs([t], [t], h, hk, d, BF16, seed)):
            x.copy_(y)
        ends.copy_(cu(lens))
        want = run()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))


def test_autograd_in_a_graph():
    """Rotary positions and attention, forward and backward, captured and replayed."""
    need_gpu()
    t, h, hk, d = 200, 6, 2, 64
    q, k, v, do = _inputs([t], [t], h, hk, d, BF16)
    leaves = [x.requires_grad_() for x in (q, k, v)]
    ends, positions, f = cu([150, 50]), torch.arange(t, device="cuda"), rotary.frequencies(d)

    def run():
        a, b = rotary.rotary(q, k, positions, f)
        o = attention.attention(a, b, v, ends)
        return (o.detach(), *torch.autograd.grad(o, leaves, do))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for seed, lens in ((10, [150, 50]), (20, [1, 199]), (30, [0, 200])):
        with torch.no_grad():
            for x, y in zip((q, k, v, do), _inputs([t], [t], h, hk, d, BF16, seed)):
                x.copy_(y)
            ends.copy_(cu(lens))
        want = run()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))


def test_graphs_that_share_a_workspace():
    """Single tokens over a cache (split keys) and a backward, replayed in turn while
    the cache's lengths grow."""
    need_gpu()
    h, hk, d, room = 8, 2, 64, 4096
    q, k, v, _ = _inputs([1, 1], [room, room], h, hk, d, BF16)
    lens = torch.tensor([3, 4000], dtype=torch.int32, device="cuda")
    one = dict(lengths_k=lens)
    tq, tk, tv, do = _inputs([70], [70], h, hk, d, BF16, 5)
    o, lse = attention.attention_fwd(tq, tk, tv, cu([70]))
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    runs = [lambda ws=None: attention.attention_fwd(q, k, v, cu_q, cu_k, ws=ws, **one),
            lambda ws=None: attention.attention_bwd(do, tq, tk, tv, o, lse, cu_t, ws=ws)]
    cu_q, cu_k, cu_t = cu([1, 1]), cu([room, room]), cu([70])
    assert attention.plan(q, k, cu_q)["splits"] > 1
    graphs, outs = [], []
    for run in runs:
        run(ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(ws))
        graphs.append(g)
    for i in (0, 1, 0, 0, 1, 0):
        lens += 17
        for t in outs[i]:
            t.zero_()
        graphs[i].replay()
        want = runs[i]()
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want))


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_many_sequences(dtype):
    """More sequences than a wave's lanes, none of whose ends is a tile's."""
    need_gpu()
    lq = [(i * 5) % 12 for i in range(330)]
    lk = [n + i % 4 for i, n in enumerate(lq)]
    for h, hk in ((7, 1), (4, 4)):
        test_forward_and_backward(lq, lk, h, hk, 64, True, dtype)


def test_offsets_past_32_bits():
    """Tokens so far apart that their offsets need more than 32 bits, forward and
    backward, few queries and many: the same bits as close together."""
    need_gpu()
    far, t, hk, d = 1 << 20, 4200, 2, 64
    room = [torch.empty((t - 1) * far + hk * d, dtype=BF16, device="cuda") for _ in range(2)]

    def apart(x, into):
        y = into.as_strided(x.shape, (far, d, 1))
        y.copy_(x)
        return y

    for lq in ([2, 1], [4200]):
        lk = [4000, 200] if len(lq) > 1 else [4200]
        q, k, v, do = _inputs(lq, lk, 4, hk, d, BF16)
        o, lse = attention.attention_fwd(q, k, v, cu(lq), cu(lk))
        want = (o, lse, *attention.attention_bwd(do, q, k, v, o, lse, cu(lq), cu(lk)))
        k, v = apart(k, room[0]), apart(v, room[1])
        got = attention.attention_fwd(q, k, v, cu(lq), cu(lk))
        got += attention.attention_bwd(do, q, k, v, o, lse, cu(lq), cu(lk))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        dk, dv = torch.empty_like(want[3]), room[1].as_strided(k.shape, (far, d, 1))
        v = want[4].new_empty(want[4].shape).copy_(v)
        attention.attention_bwd(do, q, k, v, o, lse, cu(lq), cu(lk), dQ=torch.empty_like(q), dK=dk, dV=dv)
        assert torch.equal(dv, want[4]) and torch.equal(dk, want[3])


def test_a_cache_of_many_rows():
    """More rows of a cache, times heads, than a backward takes: the forward does."""
    need_gpu()
    h, hk, d, room, lk = 128, 1, 8, 1 << 26, [700, 30]
    q, k, v, _ = _inputs([1, 1], lk, h, hk, d, BF16)
    wide = [torch.empty(2 * room, hk, d, dtype=BF16, device="cuda") for _ in range(2)]
    for x, y in zip((k, v), wide):
        y[:lk[0]], y[room:room + lk[1]] = x[:lk[0]], x[lk[0]:]
    ends = torch.arange(3, dtype=torch.int32, device="cuda")
    o, lse = attention.attention_fwd(q, *wide, ends, ends * room, lengths_k=torch.tensor(lk, dtype=torch.int32, device="cuda"))
    want = attention_reference(q, k, v, [1, 1], lk, True)
    close(o, want["o"], "o")
    close(lse, want["lse"], "lse")
    with pytest.raises(RuntimeError, match="backward"):
        attention.attention_bwd(q, q, *wide, o, lse, ends, ends * room)


def test_no_sequences():
    need_gpu()
    q, k, v, do = _inputs([5], [5], 2, 2, 64, BF16)
    ends = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = attention.attention_fwd(q, k, v, ends)
    assert bool((o == 0).all()) and bool((lse == -float("inf")).all())
    for g in attention.attention_bwd(do, q, k, v, o, lse, ends):
        assert bool((g == 0).all())


def test_another_stream():
    need_gpu()
    lq = [130]
    q, k, v, _ = _inputs(lq, lq, 2, 2, 64, BF16)
    want, _ = attention.attention_fwd(q, k, v, cu(lq))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, _ = attention.attention_fwd(q, k, v, cu(lq))
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
