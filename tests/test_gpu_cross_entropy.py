"""The head's cross entropy against 64 bits: loss, log-sum, gradient, ignored and
invalid targets, pieces of the vocabulary, strides, edges.

Bounds.  A logit is a sum of k products in fp32, off by dz <= (k + 8) 2^-24 sum
|x w| at most; the loss and the log-sum by 2 dz and 2^-20 of their size (the
exponentials and sums of at most 16 in a row, 16, and a tile for each 128
entries; logarithms), the loss of a token that is known well relative to itself
down to fp32's range (a loss below 2^-126, its smallest normal number, may be zero).
The gradient's weights p are off by a relative 2 dz + 2^-20, rounded to 16 bits
(U) as operands, and may be zero below 2^-126 (fp16: those 2^-29 below the largest, or half the smallest step
of what is kept times 2^15, are lost: 2^-29), and the result is rounded once:

    |error| <= g ((U + rel) sum_v p_v |w_v| + 2^-28 sum_v |w_v| (fp16)) + U |dx|
"""

import numpy as np
import pytest
import torch

import oracle.decoder as ref
from bit_nf4_quantized_double_amd import cross_entropy
from rows_util import TINY, U, f64, need_gpu, rand, strided

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
IGNORE = -100


def _inputs(m, k, v, dtype, seed=0, scale=1.0):
    w = rand((v, k), seed, dtype, k ** -0.5)
    y = torch.randint(0, v, (m,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))
    known = torch.linspace(0, 20, m, device="cuda")[:, None]
    x = (rand((m, k), seed + 1, torch.float32, scale) + known * w[y].float()).to(dtype)
    return x, w, y


def check(loss, lse, dx, x, w, y, dloss=None, ignore=IGNORE):
    X, W, Y = f64(x), f64(w), y.cpu().numpy()
    g = None if dloss is None else f64(dloss)
    rl, rs, rd = ref.cross_entropy(X, W, Y, ignore, g)
    z = X @ W.T
    dz = (X.shape[1] + 8) * 2.0 ** -24 * (np.abs(X) @ np.abs(W).T).max(1)
    rel = 2 * dz + 2.0 ** -20
    assert (np.abs(f64(lse) - rs) <= 2 * dz + 2.0 ** -20 * (1 + np.abs(rs))).all()
    live = Y != ignore
    bound = np.where(rl < 0.5, rl * (2 * rel) + 2.0 ** -125, 2 * dz + 2.0 ** -20 * (1 + np.abs(rs) + np.abs(rl)))
    assert (np.abs(f64(loss) - rl)[live] <= bound[live]).all(), np.abs(f64(loss) - rl)[live].max()
    assert (f64(loss)[~live] == 0).all()
    if dx is None:
        return
    p = np.exp(z - rs[:, None])
    p[np.arange(len(Y))[live], Y[live]] = 0
    u = U[x.dtype]
    mag = (u + rel)[:, None] * (p @ np.abs(W)) + (p.sum(1) * rel)[:, None] * np.abs(W[np.where(live, Y, 0)])
    mag += 2.0 ** -125 * np.abs(W).sum(0)
    if x.dtype == F16:
        mag += 2.0 ** -28 * np.abs(W).sum(0)
    mag = np.where(live, 1.0 if g is None else np.abs(g), 0.0)[:, None] * mag + u * np.abs(rd) * (1 + 2.0 ** -6) + TINY[x.dtype]
    bad = ~(np.abs(f64(dx) - rd) <= mag)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[0], f64(dx)[bad][0], rd[bad][0], mag[bad][0])
    assert (f64(dx)[~live] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,k,v", [(1, 8, 1), (1, 64, 2), (3, 72, 100), (16, 128, 127), (17, 128, 128), (64, 256, 129),
                                   (65, 200, 1000), (200, 64, 5003), (257, 136, 384), (300, 1000, 777), (5, 4096, 3001)])
def test_loss_and_gradient(m, k, v, dtype):
    need_gpu()
    x, w, y = _inputs(m, k, v, dtype)
    if m > 2:
        y[1::3] = IGNORE
    loss, lse = cross_entropy.linear_cross_entropy_fwd(x, w, y)
    check(loss, lse, None, x, w, y)
    dloss = torch.rand(m, device="cuda") + 0.1
    for g in (None, dloss):
        loss, lse, dx = cross_entropy.linear_cross_entropy_grad(x, w, y, g)
        check(loss, lse, dx, x, w, y, g)


def test_pieces_of_the_vocabulary():
    """More tokens than a round of launches, and a vocabulary in several pieces."""
    need_gpu()
    m, k, v = 8192 + 70, 64, 70001  # 2 rounds; 3 pieces in the first
    x, w, y = _inputs(m, k, v, BF16)
    y[::5] = IGNORE
    loss, lse, dx = cross_entropy.linear_cross_entropy_grad(x, w, y)
    at = torch.cat([torch.arange(0, 200), torch.arange(8150, m)]).cuda()
    check(loss[at], lse[at], dx[at], x[at], w, y[at])
    l2, s2 = cross_entropy.linear_cross_entropy_fwd(x, w, y)
    check(l2[at], s2[at], None, x[at], w, y[at])


def test_logits_that_grow():
    """The running maximum moves from piece to piece and tile to tile, by more than 16 bits' range."""
    need_gpu()
    for dtype in (BF16, F16):
        x, w, y = _inputs(40, 64, 3000, dtype)
        w *= torch.linspace(0, 30, 3000, device="cuda")[:, None].to(dtype)
        loss, lse, dx = cross_entropy.linear_cross_entropy_grad(x, w, y)
        check(loss, lse, dx, x, w, y)
        loss, lse, dx = cross_entropy.linear_cross_entropy_grad(x, w.flip(0).contiguous(), y)
        check(loss, lse, dx, x, w.flip(0), y)


def test_known_tokens_keep_their_digits():
    """1 - p of e^-20: the loss and the gradient are right relative to themselves."""
    need_gpu()
    x, w, y = _inputs(64, 256, 1000, BF16)
    x = (25 * w[y].float() / w[y].float().square().sum(1, keepdim=True)).to(BF16)
    loss, lse, dx = cross_entropy.linear_cross_entropy_grad(x, w, y)
    check(loss, lse, dx, x, w, y)
    assert float(loss.max()) < 1e-5 and float(loss.min()) > 0
    want = ref.cross_entropy(f64(x), f64(w), y.cpu().numpy())[2]
    assert np.linalg.norm(f64(dx) - want) <= 2.0 ** -7 * np.linalg.norm(want)


def test_strides_alignment_and_in_place():
    need_gpu()
    m, k, v = 70, 200, 600
    x, w, y = _inputs(m, k, v, BF16)
    want = cross_entropy.linear_cross_entropy_grad(x, w, y)
    got = cross_entropy.linear_cross_entropy_grad(strided(x, 7, 3), strided(w, 8, 8), y)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    x2 = x.clone()
    got = cross_entropy.linear_cross_entropy_grad(x2, w, y, dX=x2)
    assert got[2] is x2 and all(torch.equal(a, b) for a, b in zip(want, got))


def test_offsets_past_32_bits():
    """Rows so far apart that their offsets need more than 32 bits: the same bits."""
    need_gpu()
    m, k, v, far = 2200, 72, 3000, 1 << 20
    x, w, y = _inputs(m, k, v, BF16)
    want = cross_entropy.linear_cross_entropy_grad(x, w, y)
    room = torch.empty((v - 1) * far + k, dtype=BF16, device="cuda")
    for wide in (0, 1):
        t = room.as_strided((v, k) if wide else (m, k), (far, 1))
        t.copy_(w if wide else x)
        got = cross_entropy.linear_cross_entropy_grad(x if wide else t, t if wide else w, y)
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_ignored_and_invalid_targets():
    """An ignored token's row has no effect and no gradient, whatever it holds; a
    target outside the vocabulary shows as NaN; neither reaches other tokens."""
    need_gpu()
    m, k, v = 40, 64, 300
    x, w, y = _inputs(m, k, v, BF16)
    clean = cross_entropy.linear_cross_entropy_grad(x, w, y)
    y2, x2 = y.clone(), x.clone()
    y2[3], y2[5], y2[7], y2[9] = IGNORE, v, -1, 2 ** 40
    x2[3] = float("nan")
    x2[11, 4] = float("inf")
    loss, lse, dx = cross_entropy.linear_cross_entropy_grad(x2, w, y2)
    assert float(loss[3]) == 0 and bool((dx[3] == 0).all())
    for i in (5, 7, 9):
        assert bool(loss[i].isnan()) and bool(dx[i].isnan().all())
        assert abs(float(lse[i]) - float(clean[1][i])) <= 2.0 ** -18 * (1 + abs(float(clean[1][i])))
    assert not bool(torch.isfinite(loss[11])) and not bool(torch.isfinite(dx[11]).any())
    keep = [i for i in range(m) if i not in (3, 5, 7, 9, 11)]
    assert torch.equal(loss[keep], clean[0][keep]) and torch.equal(dx[keep], clean[2][keep])
    all_ignored = cross_entropy.linear_cross_entropy_grad(x, w, torch.full_like(y, IGNORE))
    assert bool((all_ignored[0] == 0).all()) and bool((all_ignored[2] == 0).all())
    # another ignore_index, one that is an entry
    a = cross_entropy.linear_cross_entropy_grad(x, w, torch.full_like(y, 4), ignore_index=4)
    assert bool((a[0] == 0).all()) and bool((a[2] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("v", [1, 50, 300])
def test_a_target_whose_logit_is_infinite(v, dtype):
    """It alone, every other one -inf: the loss is inf - inf, no zero, and the gradient
    no number either; other tokens do not notice."""
    need_gpu()
    x, w, y = _inputs(20, 64, v, dtype)
    w[:, 4] = -1
    w[y[7], 4] = 1
    clean = cross_entropy.linear_cross_entropy_grad(x, w, y)
    x[7, 4] = float("inf")
    loss, lse, dx = cross_entropy.linear_cross_entropy_grad(x, w, y)
    alone, _ = cross_entropy.linear_cross_entropy_fwd(x, w, y)
    assert bool(loss[7].isnan()) and bool(alone[7].isnan()) and float(lse[7]) == float("inf") and bool(dx[7].isnan().all())
    keep = [i for i in range(20) if i != 7]
    assert torch.equal(loss[keep], clean[0][keep]) and torch.equal(dx[keep], clean[2][keep])


def test_no_tokens():
    need_gpu()
    x, w, y = rand((0, 64), 1), rand((10, 64), 2), torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse, dx = cross_entropy.linear_cross_entropy_grad(x, w, y)
    assert loss.shape == lse.shape == (0,) and dx.shape == (0, 64)


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_autograd(reduction):
    """Each reduction's value and gradient, leading dimensions, against the formula
    in 64 bits and against differences."""
    need_gpu()
    x, w, y = _inputs(60, 64, 500, BF16)
    y[::4] = IGNORE
    x, y = x.view(3, 20, 64), y.view(3, 20)
    leaf = x.clone().requires_grad_()
    out = cross_entropy.linear_cross_entropy(leaf, w, y, reduction=reduction)
    up = torch.rand(out.shape, device="cuda") + 0.5
    out.backward(up)
    n = int((y != IGNORE).sum())
    g = up.reshape(-1).expand(60) / (n if reduction == "mean" else 1)
    loss, _, dx = ref.cross_entropy(f64(x).reshape(60, 64), f64(w), y.cpu().numpy().reshape(-1), IGNORE, f64(g))
    want = {"none": loss.reshape(3, 20), "sum": loss.sum(), "mean": loss.sum() / n}[reduction]
    assert np.allclose(f64(out), want, rtol=1e-4, atol=1e-5)
    # weights, the unit gradient and its multiple: three roundings to bf16
    assert np.linalg.norm(f64(leaf.grad).reshape(60, 64) - dx) <= 3 * 2.0 ** -8 * np.linalg.norm(dx)
    step = (f64(leaf.grad) / np.linalg.norm(f64(leaf.grad)) * np.linalg.norm(f64(x)) * 0.02)
    hi, lo = ((x.double().cpu() + s * torch.from_numpy(step)).to(BF16).cuda() for s in (1, -1))
    f = lambda t: float((cross_entropy.linear_cross_entropy(t, w, y, reduction=reduction).double() * up.double()).sum())
    pred = float((f64(leaf.grad) * (f64(hi) - f64(lo))).sum())
    # bf16 roundings of the gradient, and the curvature over a fiftieth of the norm
    assert abs(f(hi) - f(lo) - pred) <= 0.05 * abs(pred)


def test_same_bits_and_graph():
    """Captured once, replayed on new inputs; eager work between."""
    need_gpu()
    for m, k, v in ((40, 256, 3000), (300, 136, 1000)):
        x, w, y = _inputs(m, k, v, BF16)
        run = lambda: cross_entropy.linear_cross_entropy_grad(x, w, y)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            first = run()
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(first, run()))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        for seed in (5, 6, 7):
            for a, b in zip((x, w, y), _inputs(m, k, v, BF16, seed)):
                a.copy_(b)
            want = run()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_sums_of_losses():
    """Against 64 bits (one rounding), whatever ignored tokens hold; none that counts."""
    need_gpu()
    for m in (0, 1, 63, 1025, 70001):
        loss = rand((m,), m + 1, torch.float32).square() if m else torch.empty(0, device="cuda")
        y = torch.arange(m, device="cuda") % 7
        loss[y == 3] = float("nan")
        live = (y != 3).cpu()
        for mean in (False, True):
            got = cross_entropy.reduce_losses(loss, y, mean, ignore_index=3)
            n = int(live.sum())
            want = loss.cpu().double()[live].sum() / (n if mean else 1)
            assert torch.allclose(got[0].cpu().double(), want, rtol=2.0 ** -23, atol=0, equal_nan=True)
            assert float(got[1]) == (float(np.float32(1) / np.float32(n)) if mean and n else float("inf") if mean else 1.0)
    y.fill_(3)
    assert bool(torch.isnan(cross_entropy.reduce_losses(loss, y, True, ignore_index=3)[0]))
    assert float(cross_entropy.reduce_losses(loss, y, False, ignore_index=3)[0]) == 0.0


def test_training_step_in_a_graph():
    """Loss and gradient of more tokens than a block of any reduction, captured and
    replayed on new inputs with eager work between."""
    need_gpu()
    m, k, v = 70001, 8, 16
    x, w, y = _inputs(m, k, v, BF16)
    x.requires_grad_()

    def run(reduction):
        loss = cross_entropy.linear_cross_entropy(x, w, y, reduction=reduction)
        return loss.detach(), torch.autograd.grad(loss, x)[0]

    for reduction in ("sum", "mean"):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run(reduction)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(reduction)
        for seed in range(5, 9):
            with torch.no_grad():
                for a, b in zip((x, w, y), _inputs(m, k, v, BF16, seed)):
                    a.copy_(b)
                y[::seed] = IGNORE
            want = run(reduction)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_graphs_that_share_a_workspace():
    need_gpu()
    ins = [_inputs(m, 136, v, BF16, m) for m, v in ((300, 1000), (20, 4000))]
    ws = torch.empty(max(cross_entropy.workspace_bytes(len(y), 136, len(w), True) for _, w, y in ins), dtype=torch.uint8,
                     device="cuda")
    graphs, outs = [], []
    for x, w, y in ins:
        run = lambda: cross_entropy.linear_cross_entropy_grad(x, w, y, ws=ws)
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0):
        for t in outs[i]:
            t.zero_()
        graphs[i].replay()
        want = cross_entropy.linear_cross_entropy_grad(*ins[i])
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want))


def test_ignored_tokens_take_no_gradient():
    """Whatever comes from above for them; and no gradient is made without grad mode."""
    need_gpu()
    x, w, y = _inputs(20, 64, 50, BF16)
    y[::2] = IGNORE
    x.requires_grad_()
    up = torch.where(y == IGNORE, float("nan"), 1.0)
    g, = torch.autograd.grad(cross_entropy.linear_cross_entropy(x, w, y, reduction="none"), x, up)
    assert bool((g[::2] == 0).all()) and bool(torch.isfinite(g).all())
    with torch.no_grad():
        assert not cross_entropy.linear_cross_entropy(x, w, y).requires_grad


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("reduction", ["sum", "mean"])
def test_reduced_losses_give_ignored_tokens_no_gradient(reduction, dtype):
    """All tokens ignored (the mean is a NaN then), and an infinite gradient from
    above with some of them."""
    need_gpu()
    x, w, y = _inputs(20, 64, 50, dtype)
    x.requires_grad_()
    some = y.clone()
    some[::2] = IGNORE
    for targets, up in ((torch.full_like(y, IGNORE), 1.0), (torch.full_like(y, IGNORE), float("inf")), (some, float("inf"))):
        loss = cross_entropy.linear_cross_entropy(x, w, targets, reduction=reduction)
        g, = torch.autograd.grad(loss, x, torch.tensor(up, device="cuda"))
        live = targets != IGNORE
        assert bool((g[~live] == 0).all())
        assert not bool(torch.isfinite(g[live]).all(1).any())


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_f16_keeps_small_gradients(reduction):
    """Tokens known to 1 - p of 1e-3 to 1e-9 under a loss scale, in fp16: as far from
    64 bits as three roundings leave them.

    The row is stored times unit with (1 - p) unit at least 1/8, off by U of itself and
    half of fp16's smallest step, 2^-25 / unit <= 2^-22 (1 - p); then multiplied and
    rounded once more.  What comes before is check()'s bound, where the weights that
    are lost are 2^-28 of the largest of the target's rivals (the target's own is not
    among them)."""
    need_gpu()
    m, k, v, scale = 100, 256, 1000, 65536.0
    _, w, y = _inputs(m, k, v, F16)
    y[::9] = IGNORE
    gain = torch.linspace(14, 28, m, device="cuda")[:, None]
    own = w[y.clamp(min=0)].float()
    x = (gain * own / own.square().sum(1, keepdim=True)).to(F16).requires_grad_()
    out = cross_entropy.linear_cross_entropy(x, w, y, reduction=reduction)
    n = int((y != IGNORE).sum())
    # as large as no product leaves fp16's range: (1 - p) |w| is below 2^-9
    up = torch.full(out.shape, scale * (n if reduction == "mean" else 1), device="cuda")
    out.backward(up)
    got, X, W, Y = f64(x.grad), f64(x), f64(w), y.cpu().numpy()
    want = ref.cross_entropy(X, W, Y, IGNORE, np.full(m, scale))[2]
    live = Y != IGNORE
    assert (got[~live] == 0).all()
    z = X @ W.T
    rel = 2 * (k + 8) * 2.0 ** -24 * (np.abs(X) @ np.abs(W).T).max(1) + 2.0 ** -20
    lse = z.max(1) + np.log(np.exp(z - z.max(1)[:, None]).sum(1))
    p = np.exp(z - lse[:, None])
    p[np.arange(m), np.where(live, Y, 0)] = 0
    u, rest = U[F16], p.sum(1)
    assert rest[live].max() > 1e-4 and rest[live].min() < 1e-8
    mag = (u + rel)[:, None] * (p @ np.abs(W)) + (rest * rel)[:, None] * np.abs(W[np.where(live, Y, 0)])
    mag += 2.0 ** -28 * p.max(1)[:, None] * np.abs(W).sum(0) + 2.0 ** -22 * rest[:, None]
    bound = scale * mag + 2 * u * np.abs(want) * (1 + 2.0 ** -6) + TINY[F16]
    bad = ~(np.abs(got - want) <= bound) & live[:, None]
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[0], got[bad][0], want[bad][0], bound[bad][0])


def test_units():
    """dX in units: the same values as without where nothing is lost, powers of two;
    1 for targets that are no entry, whose rows are as ever."""
    need_gpu()
    for dtype in (BF16, F16):
        x, w, y = _inputs(300, 72, 500, dtype)
        y[::7], y[3] = IGNORE, 500
        loss, lse, dx = cross_entropy.linear_cross_entropy_grad(x, w, y)
        l2, s2, du, unit = cross_entropy.linear_cross_entropy_units(x, w, y)
        assert torch.equal(lse, s2) and torch.equal(loss[y < 500], l2[y < 500]) and bool(l2[3].isnan())
        assert bool((torch.frexp(unit)[0] == 0.5).all()) and bool((unit[::7] == 1).all()) and float(unit[3]) == 1
        assert bool((du[::7] == 0).all()) and bool(du[3].isnan().all())
        rest = -torch.expm1(-loss.double())
        at = ((y >= 0) & (y < 500) & (rest > 2.0 ** -60)).nonzero()[:, 0]
        # [1/8, 1/4), up to the rounding of the loss where it is next to a power of two
        assert bool(((rest * unit)[at] > 0.12499).all()) and bool(((rest * unit)[at] < 0.25001).all())
        back = cross_entropy.scale_rows(du, 1 / unit)
        # bf16: the exponent only; fp16: what the direct form rounds below its normal range
        if dtype == BF16:
            assert torch.equal(back[at], dx[at])
        else:
            far = (dx.float().abs() >= 2.0 ** -14) & ((du.float().abs() >= 2.0 ** -14)) & (y >= 0)[:, None] & (y < 500)[:, None]
            assert torch.equal(back[far], dx[far]) and int(far.sum()) > 1000


def test_f16_training_step_in_a_graph():
    need_gpu()
    x, w, y = _inputs(300, 72, 500, F16)
    x.requires_grad_()

    def run():
        loss = cross_entropy.linear_cross_entropy(x, w, y)
        return loss.detach(), torch.autograd.grad(loss * 4096.0, x)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for seed in range(5, 9):
        with torch.no_grad():
            for a, b in zip((x, w, y), _inputs(300, 72, 500, F16, seed)):
                a.copy_(b)
            y[::seed] = IGNORE
        want = run()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals():
    need_gpu()
    x, w, y = _inputs(4, 64, 50, BF16)
    ce = cross_entropy.linear_cross_entropy_fwd
    with pytest.raises(TypeError, match="W must be"):
        ce(x, w.half(), y)
    with pytest.raises(ValueError, match="columns"):
        ce(x, w[:, :32], y)
    with pytest.raises(TypeError, match="targets must be"):
        ce(x, w, y.int())
    with pytest.raises(ValueError, match="targets must be"):
        ce(x, w, y[:3])
    with pytest.raises(RuntimeError, match="multiple of 8"):
        ce(x[:, :60].contiguous(), w[:, :60].contiguous(), y)
    with pytest.raises(RuntimeError, match="W must be 16-byte"):
        ce(x[:, :56], w.flatten()[1:49 * 64 + 1].view(49, 64)[:, :56], y)
    with pytest.raises(ValueError, match="frozen"):
        cross_entropy.linear_cross_entropy(x, w.clone().requires_grad_(), y)
    with pytest.raises(ValueError, match="targets must have shape"):
        cross_entropy.linear_cross_entropy(x, w, y[:, None])
    with pytest.raises(RuntimeError, match="second derivative"):
        leaf = x.clone().requires_grad_()
        g, = torch.autograd.grad(cross_entropy.linear_cross_entropy(leaf, w, y), leaf, create_graph=True)
        g.sum().backward()
