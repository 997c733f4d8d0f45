"""Cases of the 8-bit serving and block operators: what is measured, in plain torch and through the package.

Six kinds of call, the ones a decoder block makes around and instead of its 4-bit linears:

  norm          residual addition and RMS norm, forward and backward (training)
  norm8         the same forward with the norm's output in 8 bits, a scale for each token (serving)
  swiglu        silu(gate) * up, forward and backward (training)
  swiglu8       silu(gate) * up in 8 bits, a scale for each token (serving)
  linear8       Y = X W^T + bias with W in 8 bits (a scale for each output channel) and X quantized on the way in
                (a scale for each token)
  linear8_train that product and dX = dY W, dY quantized on the way in

Quantization of a row x: amax = max(max |x|, 1e-30), scale = amax / 127, code = 127 x / amax rounded to the nearest
integer, ties to even.  8-bit outputs are returned as the values they stand for, in the 16-bit type of the inputs.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5
FLOOR = 1e-30


def listed():
    return [
        # a training step's norms at the 7B layer's width, one sequence of 2048 tokens
        {"name": "norm_train_2048x4096", "op": "norm", "m": 2048, "k": 4096, "dtype": "bf16", "residual": True},
        # the last, partly filled batch of a run, an uneven width, fp16, the block's first norm (no residual)
        {"name": "norm_train_777x2500_f16", "op": "norm", "m": 777, "k": 2500, "dtype": "f16", "residual": False},
        # one generated token at the 70B width: nothing but latency
        {"name": "norm8_1x8192", "op": "norm8", "m": 1, "k": 8192, "dtype": "bf16", "residual": True},
        # a batch of prompts, 4 x 2048 tokens at the 8B width
        {"name": "norm8_8192x4096", "op": "norm8", "m": 8192, "k": 4096, "dtype": "bf16", "residual": True},
        # training step of the 7B layer's MLP
        {"name": "swiglu_train_2048x11008", "op": "swiglu", "m": 2048, "k": 11008, "dtype": "bf16", "fused": False},
        # sixteen sequences decoding together; gate and up are the halves of one product's output
        {"name": "swiglu8_16x14336", "op": "swiglu8", "m": 16, "k": 14336, "dtype": "bf16", "fused": True},
        # a batch of prompts at the 8B layer's MLP width
        {"name": "swiglu8_8192x14336", "op": "swiglu8", "m": 8192, "k": 14336, "dtype": "bf16", "fused": False},
        # one generated token through the 70B gate weight: reading the weight is all there is
        {"name": "linear8_1x28672x8192", "op": "linear8", "m": 1, "n": 28672, "k": 8192, "dtype": "bf16", "bias": False},
        # sixteen sequences decoding together through the 70B down weight
        {"name": "linear8_16x8192x28672", "op": "linear8", "m": 16, "n": 8192, "k": 28672, "dtype": "bf16", "bias": False},
        # a short, uneven chunk of tokens through an uneven weight with a bias, fp16
        {"name": "linear8_150x1000x2500_f16", "op": "linear8", "m": 150, "n": 1000, "k": 2500, "dtype": "f16", "bias": True},
        # a batch of prompts through the 8B gate weight
        {"name": "linear8_8192x14336x4096", "op": "linear8", "m": 8192, "n": 14336, "k": 4096, "dtype": "bf16", "bias": False},
        # adapters trained over a frozen 8-bit layer: the 7B down weight, forward and the gradient that passes through
        {"name": "linear8_train_2048x4096x11008", "op": "linear8_train", "m": 2048, "n": 4096, "k": 11008, "dtype": "bf16", "bias": False},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm8", "swiglu", "swiglu8", "linear8", "linear8_train"])
    case = {"op": op, "m": _spread(rng, 1, 8192), "dtype": rng.choice(["bf16", "bf16", "f16"])}
    if op in ("norm", "norm8"):
        case.update(k=_spread(rng, 64, 16384), residual=rng.random() < 0.7)
    elif op in ("swiglu", "swiglu8"):
        case.update(k=_spread(rng, 64, 28672), fused=rng.random() < 0.5)
    else:
        case.update(n=_spread(rng, 64, 28672), k=_spread(rng, 64, 28672), bias=rng.random() < 0.5)
    # half of the widths are those of real layers (multiples of 128), the others as they come
    if rng.random() < 0.5:
        for d in ("n", "k"):
            if d in case:
                case[d] = max(128, case[d] // 128 * 128)
    # no more than the largest listed ones
    if "n" in case:
        times = 2 if op == "linear8_train" else 1
        case["m"] = max(1, min(case["m"], 8192 * 14336 * 4096 // (times * case["n"] * case["k"])))
    else:
        case["m"] = max(1, min(case["m"], 8192 * 14336 // (2 * case["k"])))
    return case


def _normal(gen, shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _activations(gen, m, k, dtype):
    """Hidden states: normal, with a few channels that are larger than the others throughout."""
    channel = 1.0 + 5.0 * (torch.rand(k, generator=gen, device="cuda") < 0.005)
    return (torch.randn(m, k, generator=gen, device="cuda") * channel).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype, m, k = DTYPES[case["dtype"]], case["m"], case["k"]
    state = {"op": case["op"], "dtype": dtype}
    if case["op"] in ("norm", "norm8"):
        state["x"] = _activations(gen, m, k, dtype)
        state["residual"] = _activations(gen, m, k, dtype) if case["residual"] else None
        state["gamma"] = (1.0 + 0.1 * torch.randn(k, generator=gen, device="cuda")).to(dtype)
        if case["op"] == "norm":
            state["dy"], state["dh"] = _normal(gen, (m, k), 1.0, dtype), _normal(gen, (m, k), 1.0, dtype)
    elif case["op"] in ("swiglu", "swiglu8"):
        if case["fused"]:
            both = _activations(gen, m, 2 * k, dtype)
            state["gate"], state["up"] = both[:, :k], both[:, k:]
        else:
            state["gate"], state["up"] = _activations(gen, m, k, dtype), _activations(gen, m, k, dtype)
        if case["op"] == "swiglu":
            state["dy"] = _normal(gen, (m, k), 1.0, dtype)
    else:
        n = case["n"]
        state["x"] = _activations(gen, m, k, dtype)
        state["bias"] = _normal(gen, (n,), 0.1, dtype) if case["bias"] else None
        # an 8-bit weight as a checkpoint holds it: codes [n, k] and a scale for each output channel
        weight = _normal(gen, (n, k), 0.02)
        scale = weight.abs().amax(1) / 127.0
        codes = torch.round(weight / scale[:, None]).clamp_(-127, 127).to(torch.int8)
        train = case["op"] == "linear8_train"
        if train:
            state["dy"] = _normal(gen, (m, n), 1.0, dtype)
        if own:
            from bit_nf4_quantized_double_amd import int8
            state["weight"] = int8.weight_from_codes(codes, scale, transposed=train)
        else:
            state["codes"], state["scale"] = codes, scale
    return state


def _quantize(x):
    """Codes (whole numbers in fp32) and scales of the rows of an fp32 matrix."""
    amax = x.abs().amax(1, keepdim=True).clamp(min=FLOOR)
    return torch.round(x * 127.0 / amax), amax / 127.0


def _plain_norm(s):
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["dtype"])
    # the norm is of the hidden state as it is stored
    h32, gamma = h.float(), s["gamma"].float()
    rstd = torch.rsqrt((h32 * h32).mean(1, keepdim=True) + EPS)
    return h, h32, gamma, rstd, h32 * rstd * gamma


def _run_plain(s):
    op, dtype = s["op"], s["dtype"]
    if op == "norm":
        h, h32, gamma, rstd, y = _plain_norm(s)
        dy = s["dy"].float()
        hat, g = h32 * rstd, dy * gamma
        dx = s["dh"].float() + rstd * (g - hat * (g * hat).mean(1, keepdim=True))
        return {"y": y.to(dtype), "h": h, "dx": dx.to(dtype), "dgamma": (dy * hat).sum(0)}
    if op == "norm8":
        h, _, _, _, y = _plain_norm(s)
        q, scale = _quantize(y)
        return {"h": h, "scale": scale[:, 0], "values": (q * scale).to(dtype)}
    if op in ("swiglu", "swiglu8"):
        gate, up = s["gate"].float(), s["up"].float()
        sig = 1.0 / (1.0 + torch.exp(-gate))
        y = gate * sig * up
        if op == "swiglu8":
            q, scale = _quantize(y)
            return {"scale": scale[:, 0], "values": (q * scale).to(dtype)}
        dy = s["dy"].float()
        dgate = dy * up * sig * (1.0 + gate * (1.0 - sig))
        return {"y": y.to(dtype), "dgate": dgate.to(dtype), "dup": (dy * gate * sig).to(dtype)}
    codes = s["codes"].float()
    q, scale = _quantize(s["x"].float())
    y = (q @ codes.t()) * scale * s["scale"]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if op == "linear8":
        return y.to(dtype)
    q, scale = _quantize(s["dy"].float() * s["scale"])
    return {"y": y.to(dtype), "dx": ((q @ codes) * scale).to(dtype)}


def _run_own(s):
    from bit_nf4_quantized_double_amd import int8, rows
    op = s["op"]
    if op == "norm":
        y, h, rstd = rows.rms_norm_fwd(s["x"], s["gamma"], EPS, residual=s["residual"])
        dx, dgamma = rows.rms_norm_bwd(s["dy"], h, rstd, s["gamma"], dH=s["dh"])
        return {"y": y, "h": h, "dx": dx, "dgamma": dgamma}
    if op == "norm8":
        q, h = rows.rms_norm_int8(s["x"], s["gamma"], EPS, residual=s["residual"])
        return {"h": h, "scale": q.scale, "values": rows.dequant_rows(q)}
    if op == "swiglu":
        y = rows.swiglu_fwd(s["gate"], s["up"])
        dgate, dup = rows.swiglu_bwd(s["dy"], s["gate"], s["up"])
        return {"y": y, "dgate": dgate, "dup": dup}
    if op == "swiglu8":
        q = rows.swiglu_int8(s["gate"], s["up"])
        return {"scale": q.scale, "values": rows.dequant_rows(q)}
    y = int8.linear_fwd(s["weight"], s["x"], bias=s["bias"])
    if op == "linear8":
        return y
    return {"y": y, "dx": int8.linear_bwd(s["weight"], s["dy"])}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    mk = m * k
    if op == "norm":
        # x, (residual), gamma, dy, dh read; y, (h), dx written in 16 bits, dgamma in 32
        return {"bytes": 2 * mk * (5 + 2 * case["residual"]) + 6 * k, "flops": 14 * mk}
    if op == "norm8":
        return {"bytes": 2 * mk * (2 + 2 * case["residual"]) + 2 * k + 4 * m, "flops": 8 * mk}
    if op == "swiglu":
        return {"bytes": 2 * mk * 6, "flops": 18 * mk}
    if op == "swiglu8":
        return {"bytes": 2 * mk * 3 + 4 * m, "flops": 10 * mk}
    n = case["n"]
    once = {"bytes": n * k + 4 * n + 2 * m * (n + k) + 2 * n * case["bias"], "flops": 2 * m * n * k}
    if op == "linear8":
        return once
    return {"bytes": once["bytes"] + 2 * m * (n + k), "flops": 2 * once["flops"]}


def _exact_rows(v):
    """(codes, scales) of the rows of an fp64 matrix."""
    top = torch.clamp(torch.amax(torch.abs(v), dim=-1), min=FLOOR)
    return torch.round(torch.div(torch.mul(v, 127), top[:, None])), torch.div(top, 127)


def exact(case, seed):
    s = _exact_state(case, seed)
    op, x64 = case["op"], lambda t: t.to(torch.float64)
    if op in ("norm", "norm8"):
        h = x64(s["x"])
        if s["residual"] is not None:
            h = h + x64(s["residual"])
        # what is stored, and so normalised, has the 16-bit type
        v = x64(h.to(s["dtype"]))
        norm = torch.sqrt(torch.mean(torch.square(v), dim=-1) + EPS)[:, None]
        unit = torch.div(v, norm)
        y = unit * x64(s["gamma"])
        if op == "norm8":
            q, scale = _exact_rows(y)
            return {"h": h, "scale": scale, "values": q * scale[:, None]}
        dunit = x64(s["dy"]) * x64(s["gamma"])
        along = torch.sum(dunit * unit, dim=-1, keepdim=True) / case["k"]
        dx = x64(s["dh"]) + torch.div(dunit - along * unit, norm)
        return {"y": y, "h": h, "dx": dx, "dgamma": torch.sum(x64(s["dy"]) * unit, dim=0)}
    if op in ("swiglu", "swiglu8"):
        g, u = x64(s["gate"]), x64(s["up"])
        silu = torch.div(g, 1 + torch.exp(-g))
        if op == "swiglu8":
            q, scale = _exact_rows(silu * u)
            return {"scale": scale, "values": q * scale[:, None]}
        dy, e = x64(s["dy"]), torch.exp(-g)
        # d(g / (1 + e^-g)) / dg = (1 + e^-g + g e^-g) / (1 + e^-g)^2
        slope = torch.div(1 + e + g * e, torch.square(1 + e))
        return {"y": silu * u, "dgate": dy * u * slope, "dup": dy * silu}
    w = torch.mul(x64(s["codes"]), x64(s["scale"])[:, None])
    q, scale = _exact_rows(x64(s["x"]))
    y = torch.mm(q * scale[:, None], w.t())
    if s["bias"] is not None:
        y = y + x64(s["bias"])[None, :]
    if op == "linear8":
        return y
    q, scale = _exact_rows(x64(s["dy"]) * x64(s["scale"]))
    return {"y": y, "dx": torch.mm(q * scale[:, None], x64(s["codes"]))}


def _exact_state(case, seed):
    """The inputs with the weight as codes and scales, whatever the package would keep."""
    global own
    kept, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = kept
