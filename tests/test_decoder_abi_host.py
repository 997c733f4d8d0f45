"""Host side of rotary positions, attention and the head's loss (CPU only; device
pointers are fake and never reached): argument checks, workspaces, plans, and what
the Python forms refuse before any kernel is called."""

import ctypes
import os

import pytest
import torch

from bit_nf4_quantized_double_amd import attention, cross_entropy, qlora, rotary

INVALID, SHAPE, ALIGN, WORKSPACE = -1, -2, -3, -4
P, P2, BF16, F16 = 0x10000, 0x10002, 0, 1
FWD, BWD = qlora.QLORA_OP_FWD, qlora.QLORA_OP_BWD


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(qlora.LIB_PATH):
        from bit_nf4_quantized_double_amd import build
        build.build(verbose=False)
    return qlora.lib()


def heads(p=P, token=256, head=64):
    return ctypes.byref(rotary.CHeads(p, token, head))


def rope(L, q=None, h=4, k=None, hk=0, t=8, d=64, rot=64, pos=P, turns=P, factor=1.0, qo=None, ko=None, dtype=BF16, pos64=0):
    return L.qlora_rope(q or heads(), h, k or heads(0), hk, t, d, rot, 0, pos, pos64, turns, factor, 0, qo or heads(),
                        ko or heads(0), dtype, None)


@pytest.mark.parametrize("args,want", [
    (dict(t=-1), INVALID), (dict(h=-1), INVALID), (dict(hk=-1), INVALID), (dict(d=-8), INVALID), (dict(h=70000), SHAPE),
    (dict(rot=63), SHAPE), (dict(rot=66), SHAPE), (dict(rot=-2), SHAPE), (dict(dtype=2), INVALID), (dict(dtype=7), INVALID),
    (dict(factor=float("nan")), INVALID), (dict(factor=float("inf")), INVALID), (dict(pos=None), INVALID),
    (dict(turns=None), INVALID), (dict(pos=P + 2), ALIGN), (dict(pos=P + 4, pos64=1), ALIGN), (dict(turns=P + 4), ALIGN),
    (dict(q=heads(0)), INVALID), (dict(qo=heads(0)), INVALID), (dict(q=heads(P + 1)), ALIGN), (dict(hk=2), INVALID),
    (dict(q=heads(token=-256)), INVALID), (dict(qo=heads(token=128)), INVALID), (dict(qo=heads(head=32)), INVALID),
    (dict(q=heads(token=1 << 41)), SHAPE)])
def test_rope_refuses(L, args, want):
    assert rope(L, **args) == want and L.qlora_last_error()


def test_rope_refuses_other_strides_in_place(L):
    assert rope(L, qo=heads(token=512)) == INVALID and b"strides" in L.qlora_last_error()
    assert rope(L, k=heads(), hk=4, ko=heads(head=72, token=288)) == INVALID and b"strides" in L.qlora_last_error()


def test_rope_refuses_outputs_that_are_the_other_input(L):
    at = [heads(P + 0x10000 * i) for i in range(4)]
    for q, k, qo, ko in ((0, 1, 2, 2), (0, 1, 1, 2), (0, 1, 2, 0), (0, 1, 1, 0), (0, 0, 0, 0), (0, 0, 0, 1)):
        assert rope(L, q=at[q], k=at[k], hk=4, qo=at[qo], ko=at[ko]) == INVALID
        assert b"apart" in L.qlora_last_error()


def test_rope_has_nothing_to_do(L):
    assert rope(L, t=0, q=heads(0), qo=heads(0), pos=None, turns=None) == 0
    assert rope(L, h=0, q=heads(0), qo=heads(0)) == 0
    assert rope(L, d=0, rot=0) == 0


def describe(**change):
    c = attention._CAttention(64, 64, 2, 8, 2, 64, P, P, None, None, 0.125, 1, 0, BF16)
    for name, value in change.items():
        setattr(c, name, value)
    return c


WIDE = dict(token=8 * 64, head=64)


def fwd(L, c, q=None, k=None, v=None, o=None, lse=P, ws=P, n=1 << 30):
    return L.qlora_attention_fwd(ctypes.byref(c), q or heads(**WIDE), k or heads(**WIDE), v or heads(**WIDE),
                                 o or heads(**WIDE), lse, ws, n, None)


def bwd(L, c, lse=P, ws=P, n=1 << 30, **change):
    t = {name: change.get(name) or heads(**WIDE) for name in ("do", "q", "k", "v", "o", "dq", "dk", "dv")}
    return L.qlora_attention_bwd(ctypes.byref(c), t["do"], t["q"], t["k"], t["v"], t["o"], lse, t["dq"], t["dk"], t["dv"], ws,
                                 n, None)


@pytest.mark.parametrize("change,want", [
    (dict(tokens_q=-1), INVALID), (dict(tokens_k=-1), INVALID), (dict(batch=-1), INVALID), (dict(heads=-8), INVALID),
    (dict(tokens_k=2 ** 31 - 200), SHAPE), (dict(tokens_q=2 ** 30, heads=8, kv_heads=2), SHAPE),
    (dict(heads=9), SHAPE), (dict(kv_heads=0), SHAPE), (dict(kv_heads=3), SHAPE), (dict(head_dim=0), SHAPE),
    (dict(head_dim=60), SHAPE), (dict(head_dim=136), SHAPE), (dict(head_dim=256), SHAPE), (dict(dtype=2), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(cu_q=None), INVALID), (dict(cu_k=None), INVALID), (dict(cu_q=P2), ALIGN),
    (dict(len_k=P2), ALIGN), (dict(batch=2 ** 25), SHAPE), (dict(tokens_k=2 ** 30, kv_heads=8), SHAPE)])
def test_attention_refuses_sizes(L, change, want):
    c = describe(**change)
    assert fwd(L, c) == want and bwd(L, c) == want and L.qlora_last_error()
    assert L.qlora_attention_workspace_bytes(BWD, ctypes.byref(c)) == 0
    assert L.qlora_attention_plan(ctypes.byref(c), 256, (ctypes.c_int64 * 2)()) == want


@pytest.mark.parametrize("most,over", [
    (dict(tokens_q=32 * ((1 << 21) - 67), tokens_k=1, batch=64, heads=8, kv_heads=8), dict(tokens_q=32 * ((1 << 21) - 67) + 1)),
    (dict(tokens_q=1, tokens_k=(1 << 30) - 1, batch=16, heads=128, kv_heads=8), dict(tokens_k=1 << 30)),
    (dict(tokens_q=1 << 24, tokens_k=(1 << 30) - 1, batch=1 << 20, heads=8, kv_heads=8), dict(batch=3 << 19))])
def test_attention_forward_limits(L, most, over):
    """Either side of each; keys have no part in the forward's launches."""
    out = (ctypes.c_int64 * 2)()
    assert L.qlora_attention_plan(ctypes.byref(describe(**most)), 256, out) == 0
    c = describe(**{**most, **over})
    assert L.qlora_attention_plan(ctypes.byref(c), 256, out) == SHAPE and fwd(L, c) == bwd(L, c) == SHAPE


@pytest.mark.parametrize("most,over", [
    (dict(tokens_q=1, tokens_k=128 * ((1 << 17) - 67), batch=64, heads=128, kv_heads=8), dict(tokens_k=128 * ((1 << 17) - 67) + 1)),
    (dict(tokens_q=1, tokens_k=4 * ((1 << 24) - 2 - 64) - 1, batch=64, heads=8, kv_heads=8), dict(tokens_k=4 * ((1 << 24) - 2 - 64))),
    (dict(tokens_q=1, tokens_k=1, batch=(1 << 21) - 4, heads=8, kv_heads=1), dict(batch=(1 << 21) - 3))])
def test_attention_backward_limits(L, most, over):
    """The forward takes both sides of each."""
    out, need = (ctypes.c_int64 * 2)(), lambda c: L.qlora_attention_workspace_bytes(BWD, ctypes.byref(c))
    c = describe(**{**most, **over})
    assert need(c) == 0 and bwd(L, c) == SHAPE and b"backward" in L.qlora_last_error()
    assert L.qlora_attention_plan(ctypes.byref(c), 256, out) == 0
    assert need(describe(**most)) > 0


@pytest.mark.parametrize("name", ["q", "k", "v", "o"])
def test_attention_refuses_tensors(L, name):
    call = lambda **t: (fwd(L, describe(), **t), bwd(L, describe(), **t))
    assert call(**{name: heads(0, **WIDE)}) == (INVALID, INVALID)
    assert call(**{name: heads(P2, **WIDE)}) == (ALIGN, ALIGN)
    assert call(**{name: heads(P, 8 * 64, 68)}) == (ALIGN, ALIGN)
    assert call(**{name: heads(P, 8 * 64 + 4, 64)}) == (ALIGN, ALIGN)
    assert call(**{name: heads(P, -512, 64)}) == (INVALID, INVALID)
    assert call(**{name: heads(P, 1 << 24, 64)}) == (SHAPE, SHAPE)


def test_attention_refuses_outputs(L):
    assert fwd(L, describe(), o=heads(P, 64, 64)) == INVALID  # overlapping tokens
    for name in ("dq", "dk", "dv"):
        assert bwd(L, describe(), **{name: heads(P, 64, 0)}) == INVALID
        assert bwd(L, describe(), **{name: heads(0, **WIDE)}) == INVALID
    assert fwd(L, describe(), lse=None) == INVALID and fwd(L, describe(), lse=P2) == ALIGN
    assert bwd(L, describe(), lse=None) == INVALID and bwd(L, describe(), lse=P2) == ALIGN
    assert fwd(L, describe(), ws=P2) == ALIGN and bwd(L, describe(), ws=P2) == ALIGN
    c = describe()
    need = L.qlora_attention_workspace_bytes(BWD, ctypes.byref(c))
    assert need > 0 and bwd(L, c, n=need - 1) == WORKSPACE and bwd(L, c, ws=None) == WORKSPACE
    assert L.qlora_attention_fwd(None, *[heads(**WIDE)] * 4, P, P, 1 << 30, None) == INVALID
    assert L.qlora_attention_workspace_bytes(7, ctypes.byref(c)) == 0


def test_attention_refuses_outputs_that_are_inputs(L):
    """With all else right (these have the same pointer throughout)."""
    at = lambda p: heads(p, **WIDE)
    apart = [at(P + 0x1000 * i) for i in range(9)]
    c = describe()
    assert L.qlora_attention_fwd(ctypes.byref(c), *apart[:3], apart[1], P, None, 0, None) == INVALID
    assert b"output is an input" in L.qlora_last_error()
    n = L.qlora_attention_workspace_bytes(BWD, ctypes.byref(c))
    for i in (5, 6, 7):  # dQ, dK, dV
        for other in (0, 1, 2, 3, 4):
            t = list(apart[:8])
            t[i] = t[other]
            assert L.qlora_attention_bwd(ctypes.byref(c), *t[:5], P, *t[5:], P, n, None) == INVALID
            assert b"output is an input" in L.qlora_last_error()
    assert L.qlora_attention_bwd(ctypes.byref(c), *apart[:5], P, apart[5], apart[6], apart[6], P, n, None) == INVALID
    assert b"same tensor" in L.qlora_last_error()


def test_attention_has_nothing_to_do(L):
    none = heads(0)
    c = describe(tokens_q=0)
    assert fwd(L, c, q=none, o=none, lse=None) == 0
    c = describe(tokens_q=0, tokens_k=0)
    assert bwd(L, c, do=none, q=none, k=none, v=none, o=none, dq=none, dk=none, dv=none, lse=None, ws=None, n=0) == 0
    c = describe(heads=0)
    assert fwd(L, c, q=none, o=none, lse=None) == 0


def test_attention_plan(L):
    out = (ctypes.c_int64 * 2)()

    def plan(**change):
        assert L.qlora_attention_plan(ctypes.byref(describe(**change)), 256, out) == 0
        return out[0], out[1]

    # a training step, a serving step of 16 sequences, one sequence, short ones
    assert plan(tokens_q=8192, tokens_k=8192, batch=1, heads=32, kv_heads=8, head_dim=128) == (128, 1)
    assert plan(tokens_q=16, tokens_k=16 * 16384, batch=16, heads=64, kv_heads=8) == (32, 8)
    assert plan(tokens_q=1, tokens_k=32768, batch=1, heads=8, kv_heads=8) == (32, 64)
    assert plan(tokens_q=16, tokens_k=16 * 500, batch=16, heads=64, kv_heads=8) == (32, 1)
    c = describe(tokens_q=1, tokens_k=32768, batch=1, heads=8, kv_heads=8)
    assert L.qlora_attention_workspace_bytes(FWD, ctypes.byref(c)) == 64 * 8 * (64 + 1) * 4
    assert L.qlora_attention_plan(ctypes.byref(c), 256, None) == INVALID


def loss(L, x=P, ldx=64, w=P, ldw=64, t=P, m=4, k=64, v=100, g=None, loss=P, lse=P, dx=P, dtype=BF16, ws=P, n=1 << 30):
    return L.qlora_cross_entropy(x, ldx, w, ldw, t, m, k, v, -100, g, loss, lse, dx, dtype, ws, n, None)


@pytest.mark.parametrize("args,want", [
    (dict(m=-1), INVALID), (dict(k=-8), INVALID), (dict(v=-1), INVALID), (dict(v=0), SHAPE), (dict(k=0), SHAPE),
    (dict(k=60), SHAPE), (dict(k=2 ** 21), SHAPE), (dict(v=2 ** 25), SHAPE), (dict(m=2 ** 31), SHAPE), (dict(dtype=2), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(t=None), INVALID), (dict(loss=None), INVALID),
    (dict(lse=None), INVALID), (dict(x=P + 1), ALIGN), (dict(w=P2), ALIGN), (dict(t=P + 4), ALIGN), (dict(loss=P2), ALIGN),
    (dict(g=P2), ALIGN), (dict(dx=P2), ALIGN), (dict(ldx=63), INVALID), (dict(ldw=56), INVALID), (dict(ldw=68), ALIGN),
    (dict(ldw=2 ** 22 + 8), SHAPE), (dict(ldx=2 ** 41), SHAPE), (dict(ldx=72, x=P, dx=P), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws=P2), ALIGN), (dict(n=1000), WORKSPACE)])
def test_cross_entropy_refuses(L, args, want):
    assert loss(L, **{**dict(dx=0x90000), **args}) == want and L.qlora_last_error()


def test_cross_entropy_units_refuses(L):
    def call(x=P, ldx=64, w=P, m=4, k=64, v=100, loss=P, dx=0x90000, unit=P, dtype=BF16, ws=P, n=1 << 30):
        return L.qlora_cross_entropy_units(x, ldx, w, 64, P, m, k, v, -100, loss, P, dx, unit, dtype, ws, n, None)

    for args, want in ((dict(dx=None), INVALID), (dict(unit=None), INVALID), (dict(unit=P2), ALIGN), (dict(dx=P2), ALIGN),
                       (dict(x=None), INVALID), (dict(loss=None), INVALID), (dict(w=P2), ALIGN), (dict(m=-1), INVALID),
                       (dict(k=60), SHAPE), (dict(v=0), SHAPE), (dict(dtype=2), INVALID), (dict(ldx=72, dx=P), INVALID),
                       (dict(n=1000), WORKSPACE), (dict(ws=P2), ALIGN)):
        assert call(**args) == want and L.qlora_last_error(), args
    assert call(m=0, x=None, loss=None, dx=None, unit=None, ws=None, n=0) == 0


def test_cross_entropy_workspace(L):
    ws = L.qlora_cross_entropy_workspace_bytes
    assert loss(L, m=0, x=None, t=None, loss=None, lse=None, dx=None, ws=None, n=0) == 0
    assert ws(0, 64, 100, 1) == 0 and ws(4, 60, 100, 1) == 0 and ws(4, 64, 0, 1) == 0
    assert 0 < ws(100, 4096, 32000, 0) < ws(100, 4096, 32000, 1)
    # it stops growing with the tokens
    most = ws(8192, 4096, 128256, 1)
    assert ws(10 ** 6, 4096, 128256, 1) <= 2 * most and ws(8192 * 100, 4096, 128256, 1) == most
    # a smaller last round may need more for its splits: the whole is never less than either
    assert ws(8192 + 70, 64, 70001, 1) >= max(ws(8192, 64, 70001, 1), ws(70, 64, 70001, 1))


def test_loss_sum_refuses(L):
    call = lambda loss=P, targets=P, m=4, out=P: L.qlora_loss_sum(loss, targets, m, -100, 1, out, None)
    assert call(m=-1) == call(loss=None) == call(targets=None) == call(out=None) == INVALID
    assert call(loss=P2) == call(targets=P + 4) == call(out=P2) == ALIGN
    assert call(m=1 << 31) == SHAPE
    with pytest.raises(ValueError, match="on the GPU"):
        cross_entropy.reduce_losses(torch.zeros(3), torch.zeros(3, dtype=torch.int64), True)


def test_scale_rows_refuses(L):
    f = lambda x=P, g=P, m=4, k=64, y=P, dtype=BF16: L.qlora_scale_rows(x, g, m, k, y, dtype, None)
    assert f(k=60) == SHAPE and f(m=-1) == INVALID and f(x=None) == INVALID and f(g=P2) == ALIGN and f(y=P2) == ALIGN
    assert f(dtype=2) == INVALID and f(m=0, x=None) == 0


def test_frequencies():
    """Fractions of a turn to 2^-64, every scaling's defining property."""
    for rot in (2, 34, 128):
        f = rotary.frequencies(rot, device="cpu")
        assert f.rot == rot and f.factor == 1.0 and f.turns.dtype == torch.int64
        got = [(int(t) % 2 ** 64) / 2 ** 64 * 6.283185307179586 for t in f.turns]
        assert all(abs(g - 10000.0 ** (-2 * i / rot)) <= 1e-15 * 7 for i, g in enumerate(got))
    radians = lambda f: torch.tensor([(int(t) % 2 ** 64) / 2 ** 64 * 6.283185307179586 for t in f.turns], dtype=torch.float64)
    plain = radians(rotary.frequencies(64, device="cpu"))
    assert torch.allclose(radians(rotary.frequencies(64, scaling="linear", by=4.0, device="cpu")), plain / 4, rtol=1e-12)
    base = radians(rotary.frequencies(64, scaling="base", by=4.0, device="cpu"))
    assert base[0] == plain[0] and abs(base[-1] / plain[-1] * 4 - 1) < 1e-12
    blend = rotary.frequencies(64, scaling="blended", by=4.0, device="cpu")
    b = radians(blend)
    turns = 4096 * plain / 6.283185307179586
    assert torch.allclose(b[turns >= 32], plain[turns >= 32], rtol=1e-12)
    assert torch.allclose(b[turns <= 1], plain[turns <= 1] / 4, rtol=1e-12)
    assert abs(blend.factor - (0.1 * 1.3862943611198906 + 1)) < 1e-12
    # a negative frequency and one above a turn are taken modulo one
    assert int(rotary.Frequencies([-1.0], device="cpu").turns[0]) == -int(rotary.Frequencies([1.0], device="cpu").turns[0])
    for bad in (dict(rot=3), dict(rot=64, scaling="x"), dict(rot=64, by=0.5), dict(rot=64, base=0.0),
                dict(rot=64, scaling="blended", low=2.0, high=1.0)):
        with pytest.raises(ValueError):
            rotary.frequencies(**bad, device="cpu")
    with pytest.raises(ValueError, match="finite"):
        rotary.Frequencies([float("nan")], device="cpu")


def test_forms_refuse_tensors_off_the_gpu():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="no CPU path"):
        rotary.rotate(x, None, torch.arange(4), rotary.frequencies(64, device="cpu"))
    with pytest.raises(ValueError, match="no CPU path"):
        attention.attention_fwd(x, x, x, cu)
    with pytest.raises(ValueError, match="must be a \\[tokens"):
        attention.attention(x[0], x, x, cu)
    with pytest.raises(ValueError, match="no CPU path"):
        cross_entropy.linear_cross_entropy_fwd(x[:, 0], x[:, 0], torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="targets must have shape"):
        cross_entropy.linear_cross_entropy(x[:, 0], x[:, 0], torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="unknown reduction"):
        cross_entropy.linear_cross_entropy(x[:, 0], x[:, 0], torch.zeros(4, dtype=torch.int64), reduction="max")
    with pytest.raises(ValueError, match="frozen"):
        cross_entropy.linear_cross_entropy(x[:, 0], x[:, 0].clone().requires_grad_(), torch.zeros(4, dtype=torch.int64))
