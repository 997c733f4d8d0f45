"""Cases of the operators between a decoder's linears and at its end: what is measured, in plain torch and through
the package.

Seven kinds of call:

  rotate        rotary positions of queries and keys (serving)
  rotate_train  the same and its backward, the inverse rotation of the gradients
  prompt        attention of packed sequences, each query to its own sequence's keys up to its own place (serving)
  decode        the same for a few new tokens of each sequence, over a cache with room behind each sequence
  attend_train  packed attention, forward and backward
  score         the loss of each token under a frozen output head, without its logits (evaluation)
  loss_train    that loss and the gradient of the hidden states

Rotary positions: token t turns pair i of a head by the angle p_t f_i, and lengthens it by a factor (1, or that of
the scaling for long contexts).  Pairs are (i, i + r/2) of the r rotated values, or (2i, 2i + 1) ("interleaved").

Attention: query i of a sequence with n queries and m keys sees keys 0 .. i + m - n ("causal"; the last query sees
all keys) or all of them.  A query that sees none gets zeros and a log-sum of -inf.  Query head h reads key head
h // (heads / kv_heads).

Loss: z = X W^T in 32 bits, loss_t = log sum_v exp z_tv - z_t,target, 0 for a token whose target is IGNORE.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
IGNORE = -100
BASE = 10000.0


def listed():
    return [
        # one new token in each of 16 sequences, far into their contexts, at the 8B layer's heads: nothing but latency
        {"name": "rotate_16x32_8", "op": "rotate", "t": 16, "heads": 32, "kv_heads": 8, "d": 128, "rot": 128,
         "interleaved": False, "scaling": "none", "far": 131072, "dtype": "bf16"},
        # a training step's queries and keys, slices of one projection's output, four sequences of 2048
        {"name": "rotate_train_8192x32_8", "op": "rotate_train", "t": 8192, "heads": 32, "kv_heads": 8, "d": 128,
         "rot": 128, "interleaved": False, "scaling": "none", "far": 2048, "dtype": "bf16"},
        # part of an uneven head, pairs side by side, frequencies blended for 4 times the trained context, fp16
        {"name": "rotate_train_777x10_2x80_f16", "op": "rotate_train", "t": 777, "heads": 10, "kv_heads": 2, "d": 80,
         "rot": 32, "interleaved": True, "scaling": "blended", "far": 16384, "dtype": "f16"},
        # one question of some words: the smallest prompt
        {"name": "prompt_100x32", "op": "prompt", "lq": "100", "lk": "100", "heads": 32, "kv_heads": 32, "d": 128,
         "causal": True, "dtype": "bf16"},
        # new turns of four conversations: prompts behind prefixes that are in the cache already
        {"name": "prompt_4_turns_64_8", "op": "prompt", "lq": "512, 1000, 37, 2048", "lk": "8704, 5096, 16421, 2048",
         "heads": 64, "kv_heads": 8, "d": 128, "causal": True, "dtype": "bf16"},
        # a serving step of 16 sequences of mixed lengths, one new token each
        {"name": "decode_16x64_8", "op": "decode", "new": 1,
         "lk": "16384, 12000, 9001, 8192, 7777, 5000, 4096, 4095, 3001, 2049, 2048, 1025, 600, 129, 64, 1",
         "room": 16384, "heads": 64, "kv_heads": 8, "d": 128, "dtype": "bf16"},
        # a training step of the 7B layer: short and long samples packed into 2048 tokens
        {"name": "attend_train_packed_2048x32", "op": "attend_train", "lq": "700, 41, 333, 1, 462, 511",
         "lk": "700, 41, 333, 1, 462, 511", "heads": 32, "kv_heads": 32, "d": 128, "causal": True, "dtype": "bf16"},
        # the 8B layer on one sequence of 8192 tokens
        {"name": "attend_train_8192x32_8", "op": "attend_train", "lq": "8192", "lk": "8192", "heads": 32, "kv_heads": 8,
         "d": 128, "causal": True, "dtype": "bf16"},
        # uneven heads and lengths, a sequence with fewer keys than queries (rows that see nothing), an empty one, fp16
        {"name": "attend_train_odd_10_2x80_f16", "op": "attend_train", "lq": "130, 0, 65, 777, 1", "lk": "130, 0, 40, 777, 9",
         "heads": 10, "kv_heads": 2, "d": 80, "causal": True, "dtype": "f16"},
        # the likelihood of the 16 tokens of an answer at the 70B width
        {"name": "score_16x8192x128256", "op": "score", "t": 16, "k": 8192, "v": 128256, "ignored": 0.0, "dtype": "bf16"},
        # a training step's loss on the answers of short samples: the 7B layer's width, a vocabulary of 32000, fp16
        {"name": "loss_train_1001x4096x32000_f16", "op": "loss_train", "t": 1001, "k": 4096, "v": 32000, "ignored": 0.4,
         "dtype": "f16"},
        # the 8B layer's step of 8192 tokens with a vocabulary of 128256, whose logits would take 4 GB
        {"name": "loss_train_8192x4096x128256", "op": "loss_train", "t": 8192, "k": 4096, "v": 128256, "ignored": 0.1,
         "dtype": "bf16"},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rotate", "rotate_train", "prompt", "decode", "attend_train", "attend_train", "score",
                     "loss_train", "loss_train"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16"])}
    if op in ("score", "loss_train"):
        k = _spread(rng, 64, 8192) // 8 * 8
        v = _spread(rng, 100, 131072)
        t = _spread(rng, 1, 8192)
        if op == "score":
            t = min(t, 2 * 8192 * 4096 * 128256 // (k * v))
        else:
            t = min(t, 8192 * 4096 * 128256 // (k * v))
        case.update(t=max(1, t), k=k, v=v, ignored=rng.choice([0.0, 0.1, 0.5]))
        return case
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    case.update(heads=kv_heads * rng.choice([1, 1, 2, 4, 7, 8]), kv_heads=kv_heads,
                d=rng.choice([128, 128, 128, 64, 64, 80, 96, 8 * rng.randint(1, 16)]))
    if op in ("rotate", "rotate_train"):
        t = min(_spread(rng, 1, 8192), 8192 * 40 * 128 // ((case["heads"] + kv_heads) * case["d"]))
        case.update(t=max(1, t), rot=rng.choice([case["d"], case["d"], 2 * rng.randint(1, case["d"] // 2)]),
                    interleaved=rng.random() < 0.4, scaling=rng.choice(["none", "none", "linear", "base", "blended"]),
                    far=_spread(rng, 16, 1048576))
        return case
    if op == "decode":
        n = _spread(rng, 1, 32)
        room = _spread(rng, 16, 32768)
        room = max(16, min(room, 16 * 16384 * 8 * 128 // (n * kv_heads * case["d"])))
        new = min(room, rng.choice([1, 1, 1, 2, 5]))
        case.update(new=new, room=room,
                    lk=_text(min(room, max(new, _spread(rng, 1, room))) for _ in range(n)))
        return case
    case["causal"] = rng.random() < 0.85
    lq, lk = [], []
    longest = _spread(rng, 1, 8192)
    for _ in range(_spread(rng, 1, 16)):
        q = rng.choice([0, 1, longest, _spread(rng, 1, longest), _spread(rng, 1, longest)])
        k = q
        if op == "prompt" and rng.random() < 0.5:
            k = q + _spread(rng, 1, 4096)
        elif rng.random() < 0.1:
            k = rng.randint(0, q)  # queries that see nothing
        # products of all queries and keys, no more than the largest listed one
        if sum(a * b for a, b in zip(lq + [q], lk + [k])) * case["heads"] * case["d"] > 8192 * 8192 * 32 * 128:
            break
        if sum(lk) + k > 40000:
            break
        lq.append(q)
        lk.append(k)
    if sum(lq) == 0:
        lq, lk = [17], [17]
    case.update(lq=_text(lq), lk=_text(lk))
    return case


def _lengths(text):
    return [int(n) for n in text.split(",")]


def _text(lengths):
    return ", ".join(str(n) for n in lengths)


def _starts(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return at


def _cu(lengths):
    return torch.tensor(_starts(lengths), dtype=torch.int32, device="cuda")


def _frequencies(rot, scaling, dtype=torch.float64):
    """f_i and the factor, by the published rules: one frequency a pair; positions divided ("linear"); a larger base
    ("base"); blended by how many turns a pair makes over the trained context, with a factor ("blended")."""
    i = torch.arange(rot // 2, dtype=dtype)
    base, s = BASE, 4.0
    if scaling == "base":
        base = base * s ** (rot / (rot - 2)) if rot > 2 else base
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / s
    if scaling != "blended":
        return f, 1.0
    turns = 4096 * f / (2 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    return f / s * (1 - keep) + f * keep, 0.1 * math.log(s) + 1.0


def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    s = {"op": op, "dtype": dtype}
    if op in ("score", "loss_train"):
        t, k, v = case["t"], case["k"], case["v"]
        s["w"] = _normal(gen, (v, k), dtype, 0.02)
        s["targets"] = torch.randint(0, v, (t,), generator=gen, device="cuda")
        # hidden states that know some targets well, some a little and some not at all, as a trained model's do:
        # a target's logit is up to 25 above the others, which are normal
        known = 25.0 * torch.rand(t, 1, generator=gen, device="cuda") ** 2
        s["x"] = (torch.randn(t, k, generator=gen, device="cuda") * (2500.0 / k) ** 0.5
                  + known * s["w"][s["targets"]].float() / (0.0004 * k)).to(dtype)
        s["targets"][torch.rand(t, generator=gen, device="cuda") < case["ignored"]] = IGNORE
        if op == "loss_train":
            # the mean over the tokens that count; fp16 with the loss scaled, as it is trained
            count = (s["targets"] != IGNORE).sum().clamp(min=1)
            s["dloss"] = (torch.ones(t, device="cuda") / count) * (65536.0 if case["dtype"] == "f16" else 1.0)
        return s
    h, hk, d = case["heads"], case["kv_heads"], case["d"]
    if op in ("rotate", "rotate_train"):
        t, rot = case["t"], case["rot"]
        s["interleaved"] = case["interleaved"]
        qkv = _normal(gen, (t, (h + 2 * hk) * d), dtype)
        s["q"], s["k"] = qkv[:, :h * d].view(t, h, d), qkv[:, h * d:(h + hk) * d].view(t, hk, d)
        far = case["far"]
        # sequences of 2048 (or the whole range, where it is smaller), ending far out
        s["positions"] = (far - 1 - torch.arange(t, device="cuda") % min(far, 2048)).flip(0).to(torch.int32)
        if op == "rotate_train":
            s["dq"], s["dk"] = _normal(gen, (t, h, d), dtype), _normal(gen, (t, hk, d), dtype)
        f, factor = _frequencies(rot, case["scaling"])
        if own:
            from bit_nf4_quantized_double_amd import rotary
            s["freqs"] = rotary.Frequencies(f, factor, device="cuda")
        else:
            s["f"], s["factor"], s["rot"] = f.cuda(), factor, rot
        return s
    if op == "decode":
        lk, new, room = _lengths(case["lk"]), case["new"], case["room"]
        n = len(lk)
        s["lq"], s["lk"], s["room"], s["causal"] = [new] * n, lk, room, True
        s["q"] = _normal(gen, (n * new, h, d), dtype)
        s["k"], s["v"] = _normal(gen, (n * room, hk, d), dtype), _normal(gen, (n * room, hk, d), dtype)
        s["cu_q"] = torch.arange(n + 1, dtype=torch.int32, device="cuda") * new
        s["cu_k"] = torch.arange(n + 1, dtype=torch.int32, device="cuda") * room
        s["lengths_k"] = torch.tensor(lk, dtype=torch.int32, device="cuda")
        return s
    s["lq"], s["lk"], s["causal"] = _lengths(case["lq"]), _lengths(case["lk"]), case["causal"]
    tq, tk = sum(s["lq"]), sum(s["lk"])
    s["q"] = _normal(gen, (tq, h, d), dtype)
    s["k"], s["v"] = _normal(gen, (tk, hk, d), dtype), _normal(gen, (tk, hk, d), dtype)
    s["cu_q"], s["cu_k"] = _cu(s["lq"]), _cu(s["lk"])
    if op == "attend_train":
        s["do"] = _normal(gen, (tq, h, d), dtype)
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------

def _turned(x, positions, f, factor, rot, interleaved, back):
    angle = positions.double()[:, None] * f
    cos = (torch.cos(angle) * factor).float()[:, None, :]
    sin = (torch.sin(angle) * (-factor if back else factor)).float()[:, None, :]
    x32 = x.float()
    out = x32.clone()
    if interleaved:
        a, b = x32[..., 0:rot:2], x32[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x32[..., :rot // 2], x32[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return out.to(x.dtype)


def _plain_rotate(s):
    args = (s["positions"], s["f"], s["factor"], s["rot"], s["interleaved"])
    out = {"q": _turned(s["q"], *args, False), "k": _turned(s["k"], *args, False)}
    if s["op"] == "rotate_train":
        out.update(dq=_turned(s["dq"], *args, True), dk=_turned(s["dk"], *args, True))
    return out


def _by_heads(x, group):
    """[tokens, heads, d] -> fp32 [heads * group, tokens, d], each head `group` times."""
    return x.float().transpose(0, 1).repeat_interleave(group, 0).contiguous()


def _plain_attention(s):
    q, dtype = s["q"], s["dtype"]
    tq, h, d = q.shape
    group = h // s["k"].shape[1]
    scale = d ** -0.5
    train = s["op"] == "attend_train"
    o = torch.zeros(tq, h, d, dtype=dtype, device="cuda")
    lse = torch.full((tq, h), -math.inf, device="cuda")
    grads = [torch.zeros_like(x) for x in (q, s["k"], s["v"])] if train else []
    room = [s["room"]] * len(s["lk"]) if s["op"] == "decode" else s["lk"]
    # the heads of a few key heads at a time: scores in 32 bits fit beside one another
    for n, m, q0, k0 in zip(s["lq"], s["lk"], _starts(s["lq"]), _starts(room)):
        if n == 0 or m == 0:
            continue
        hidden = None
        if s["causal"]:
            hidden = torch.arange(m, device="cuda")[None, :] > torch.arange(n, device="cuda")[:, None] + (m - n)
        step = max(1, min(s["k"].shape[1], 2 ** 31 // (n * m * group)))
        for g in range(0, s["k"].shape[1], step):
            kh, qh = slice(g, g + step), slice(g * group, (g + step) * group)
            qs = _by_heads(q[q0:q0 + n, qh], 1)
            ks, vs = (_by_heads(x[k0:k0 + m, kh], group) for x in (s["k"], s["v"]))
            z = torch.bmm(qs, ks.transpose(1, 2).contiguous()) * scale
            if hidden is not None:
                z.masked_fill_(hidden, -math.inf)
            top = z.amax(-1, keepdim=True)
            top = torch.where(top == -math.inf, torch.zeros_like(top), top)
            p = torch.exp(z - top)
            total = p.sum(-1, keepdim=True)
            lse[q0:q0 + n, qh] = (top + torch.log(total))[..., 0].transpose(0, 1)
            p = p / torch.where(total == 0, torch.ones_like(total), total)
            y = torch.bmm(p, vs)
            o[q0:q0 + n, qh] = y.transpose(0, 1).to(dtype)
            if train:
                dy = _by_heads(s["do"][q0:q0 + n, qh], 1)
                dv = torch.bmm(p.transpose(1, 2).contiguous(), dy)
                dz = p * (torch.bmm(dy, vs.transpose(1, 2).contiguous()) - (dy * y).sum(-1, keepdim=True)) * scale
                grads[0][q0:q0 + n, qh] = torch.bmm(dz, ks).transpose(0, 1).to(dtype)
                dk = torch.bmm(dz.transpose(1, 2).contiguous(), qs)
                for out, x in ((grads[1], dk), (grads[2], dv)):
                    out[k0:k0 + m, kh] = x.view(-1, group, m, d).sum(1).transpose(0, 1).to(dtype)
    out = {"o": o, "lse": lse}
    if train:
        out.update(dq=grads[0], dk=grads[1], dv=grads[2])
    return out


def _plain_loss(s):
    x, w, targets = s["x"].float(), s["w"].float(), s["targets"]
    counts = targets != IGNORE
    at = torch.where(counts, targets, torch.zeros_like(targets))[:, None]
    z = x @ w.t()
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    # the target's own term apart from the others': 1 - p of a token that is known well would lose all its digits
    mine = e.gather(1, at)
    others = e.scatter(1, at, 0.0)
    rest = others.sum(1, keepdim=True)
    loss = torch.where(counts, torch.where(rest[:, 0] < mine[:, 0], torch.log1p(rest / mine)[:, 0],
                                           (top + torch.log(total) - z.gather(1, at))[:, 0]), 0.0)
    lse = (top + torch.log(total))[:, 0]
    if s["op"] == "score":
        return {"loss": loss, "lse": lse}
    g = torch.where(counts, s["dloss"], 0.0)[:, None]
    dx = g * ((others @ w) / total - (rest / total) * w[at[:, 0]])
    return {"loss": loss, "lse": lse, "dx": dx.to(s["dtype"])}


# ---- through the package ---------------------------------------------------------------------------------------

def _run_own(s):
    op = s["op"]
    if op in ("rotate", "rotate_train"):
        from bit_nf4_quantized_double_amd import rotary
        q, k = rotary.rotate(s["q"], s["k"], s["positions"], s["freqs"], interleaved=s["interleaved"])
        if op == "rotate":
            return {"q": q, "k": k}
        dq, dk = rotary.rotate_bwd(s["dq"], s["dk"], s["positions"], s["freqs"], interleaved=s["interleaved"])
        return {"q": q, "k": k, "dq": dq, "dk": dk}
    if op in ("score", "loss_train"):
        from bit_nf4_quantized_double_amd import cross_entropy
        if op == "score":
            loss, lse = cross_entropy.linear_cross_entropy_fwd(s["x"], s["w"], s["targets"], ignore_index=IGNORE)
            return {"loss": loss, "lse": lse}
        loss, lse, dx = cross_entropy.linear_cross_entropy_grad(s["x"], s["w"], s["targets"], s["dloss"],
                                                                ignore_index=IGNORE)
        return {"loss": loss, "lse": lse, "dx": dx}
    from bit_nf4_quantized_double_amd import attention
    o, lse = attention.attention_fwd(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], lengths_k=s.get("lengths_k"),
                                     causal=s["causal"])
    if op != "attend_train":
        return {"o": o, "lse": lse}
    dq, dk, dv = attention.attention_bwd(s["do"], s["q"], s["k"], s["v"], o, lse, s["cu_q"], s["cu_k"],
                                         causal=s["causal"])
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def run(state):
    if own:
        return _run_own(state)
    if state["op"] in ("rotate", "rotate_train"):
        return _plain_rotate(state)
    return _plain_loss(state) if state["op"] in ("score", "loss_train") else _plain_attention(state)


def _case_lengths(case):
    lk = _lengths(case["lk"])
    return ([case["new"]] * len(lk) if case["op"] == "decode" else _lengths(case["lq"])), lk


def _pairs(case):
    """Query-key pairs that are seen."""
    lq, lk = _case_lengths(case)
    if not case.get("causal", True):
        return sum(n * m for n, m in zip(lq, lk))
    total = 0
    for n, m in zip(lq, lk):
        # the last query sees m keys, the one before m - 1, ..., down to 1 or to the first query
        seen = min(n, m)
        total += seen * m - seen * (seen - 1) // 2
    return total


def work(case):
    op = case["op"]
    if op in ("score", "loss_train"):
        t, k, v = case["t"], case["k"], case["v"]
        train = op == "loss_train"
        return {"bytes": 2 * v * k + 2 * t * k * (1 + train) + 16 * t + 4 * t * train, "flops": 2 * t * k * v * (1 + train)}
    h, hk, d = case["heads"], case["kv_heads"], case["d"]
    if op in ("rotate", "rotate_train"):
        n = case["t"] * (h + hk)
        times = 1 + (op == "rotate_train")
        return {"bytes": times * (4 * n * d + 4 * case["t"]) + 8 * (case["rot"] // 2), "flops": times * 3 * n * case["rot"]}
    tq, tk = (sum(n) for n in _case_lengths(case))
    bytes_, flops = 2 * d * (2 * tq * h + 2 * tk * hk) + 4 * tq * h, 4 * _pairs(case) * h * d
    if op == "attend_train":
        # dO read, dQ, dK, dV written beside q, k, v, o and the log-sums, read again
        bytes_ += 2 * d * (4 * tq * h + 4 * tk * hk) + 4 * tq * h
        flops += 10 * _pairs(case) * h * d
    return {"bytes": bytes_, "flops": flops}


# ---- in 64 bits ------------------------------------------------------------------------------------------------

def _exact_state(case, seed):
    """The inputs with plain frequencies, whatever the package would keep."""
    global own
    kept, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = kept


def _exact_rotation(x, s, sign):
    """Pairs as complex numbers times factor e^(i angle)."""
    v = x.to(torch.float64)
    r = s["rot"]
    head, tail = v[..., :r], v[..., r:]
    pairs = head.unflatten(-1, (r // 2, 2)) if s["interleaved"] else torch.stack((head[..., :r // 2], head[..., r // 2:]), -1)
    turn = torch.polar(torch.full((1,), s["factor"], dtype=torch.float64, device=x.device),
                       torch.outer(s["positions"].to(torch.float64), s["f"]) * sign)
    done = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn.unsqueeze(1))
    head = done.flatten(-2) if s["interleaved"] else torch.cat((done[..., 0], done[..., 1]), -1)
    return torch.cat((head, tail), -1)


def _exact_head(q, k, v, do, first):
    """One head of one sequence, rows of queries in turn; `first` is how many keys the first row sees, less one
    (None: all)."""
    n, m, c = q.shape[0], k.shape[0], 1.0 / math.sqrt(q.shape[1])
    out, sums, dq = torch.empty_like(q), q.new_empty(n), torch.empty_like(q)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    for a in range(0, n, 4096):
        b = min(n, a + 4096)
        score = torch.mm(q[a:b] * c, k.t())
        if first is not None:
            rows, cols = torch.arange(a, b, device=q.device), torch.arange(m, device=q.device)
            score = torch.where(torch.le(cols, rows[:, None] + first), score, -math.inf)
        sums[a:b] = torch.logsumexp(score, 1)
        p = torch.nan_to_num(torch.exp(score - sums[a:b, None]), nan=0.0)
        out[a:b] = torch.mm(p, v)
        if do is not None:
            dp = torch.mm(do[a:b], v.t())
            # the softmax' derivative from P alone
            ds = c * (p * dp - p * torch.sum(p * dp, 1, keepdim=True))
            dq[a:b] = torch.mm(ds, k)
            dk += torch.mm(ds.t(), q[a:b])
            dv += torch.mm(p.t(), do[a:b])
    return out, sums, dq, dk, dv


def exact(case, seed):
    s, op = _exact_state(case, seed), case["op"]
    if op in ("rotate", "rotate_train"):
        out = {"q": _exact_rotation(s["q"], s, 1.0), "k": _exact_rotation(s["k"], s, 1.0)}
        if op == "rotate_train":
            out.update(dq=_exact_rotation(s["dq"], s, -1.0), dk=_exact_rotation(s["dk"], s, -1.0))
        return out
    if op in ("score", "loss_train"):
        w = s["w"].to(torch.float64)
        loss, lse, dx = [], [], []
        for a in range(0, case["t"], 1024):
            x, y = s["x"][a:a + 1024].to(torch.float64), s["targets"][a:a + 1024]
            z = torch.mm(x, w.t())
            sums = torch.logsumexp(z, 1)
            live = torch.ne(y, IGNORE)
            rows = torch.arange(len(y), device=y.device)[live]
            l = torch.zeros_like(sums)
            l[rows] = sums[rows] - z[rows, y[rows]]
            loss.append(l)
            lse.append(sums)
            if op == "loss_train":
                p = torch.softmax(z, 1)
                p[rows, y[rows]] -= 1.0
                p *= torch.where(live, s["dloss"][a:a + 1024].to(torch.float64), 0.0)[:, None]
                dx.append(torch.mm(p, w))
        out = {"loss": torch.cat(loss), "lse": torch.cat(lse)}
        if op == "loss_train":
            out["dx"] = torch.cat(dx)
        return out
    tq, h, d = s["q"].shape
    hk = s["k"].shape[1]
    train = op == "attend_train"
    new = lambda like: torch.zeros(like.shape, dtype=torch.float64, device=like.device)
    out = {"o": new(s["q"]), "lse": torch.full((tq, h), -math.inf, dtype=torch.float64, device="cuda")}
    if train:
        out.update(dq=new(s["q"]), dk=new(s["k"]), dv=new(s["v"]))
    starts_k = _starts([s["room"]] * len(s["lk"]) if op == "decode" else s["lk"])
    for n, m, q0, k0 in zip(s["lq"], s["lk"], _starts(s["lq"]), starts_k):
        if n == 0 or m == 0:
            continue
        for i in range(h):
            j = i // (h // hk)
            f64 = lambda t, at, count, head: t[at:at + count, head].to(torch.float64)
            o, sums, dq, dk, dv = _exact_head(f64(s["q"], q0, n, i), f64(s["k"], k0, m, j), f64(s["v"], k0, m, j),
                                              f64(s["do"], q0, n, i) if train else None, m - n if s["causal"] else None)
            out["o"][q0:q0 + n, i], out["lse"][q0:q0 + n, i] = o, sums
            if train:
                out["dq"][q0:q0 + n, i] = dq
                out["dk"][k0:k0 + m, j] += dk
                out["dv"][k0:k0 + m, j] += dv
    return out
