"""The two ends of a training step, as measured cases: the embedding lookup and
its gradient, the clipped policy loss with a KL term and its gradient, the norm
of all gradients, and the AdamW step over many tensors.

Operators, each with a plain form in elementary torch operations (FP32, rounded
once at the end) and, where ``own`` is true, the library's call:

  lookup            out[i] = scale * weight[token[i]]
  lookup_backward   dweight[v] (+)= scale * sum of dout[i] over token[i] = v
  policy            with d = old_nll - nll and r = exp(d):
                    l = -min(r A, clip(r) A) + beta (exp(q) - q - 1),
                    q = nll - ref_nll, averaged over tokens or over sequences
  policy_backward   dnll
  norm              n = scale |all gradients|_2, factor = scale min(1, max / n)
  adamw             m, v, p of every tensor; m and v in FP32, or in 8 bits with
                    a power of two for each 256 of them, rounded at random

``exact`` states the same definitions once more in FP64.
"""

import math

import torch

own = False

IGNORE = -100
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 256
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.95, 1e-8, 0.1
CLIP_LOW, CLIP_HIGH, KL = 0.2, 0.28, 0.04


def listed():
    return [
        # four sequences decode: one token each
        {"name": "lookup 4x2048 bf16", "op": "lookup", "rows": 4, "width": 2048, "vocab": 32768,
         "type": "bf16", "scale": 1.0, "ignored": 0.0},
        # a training batch against a large vocabulary, scaled by sqrt(width)
        {"name": "lookup 32768x4096 bf16", "op": "lookup", "rows": 32768, "width": 4096,
         "vocab": 131072, "type": "bf16", "scale": 64.0, "ignored": 0.0},
        # a short fine-tuning sequence: its gradient is added to the one that
        # the head, whose weight is the same tensor, has left
        {"name": "lookup bwd 48x1024 f16", "op": "lookup_backward", "rows": 48, "width": 1024,
         "vocab": 32768, "type": "f16", "into": "f16", "add": True, "scale": 1.0, "ignored": 0.0},
        # a ragged batch, a third of it padding; odd rows
        {"name": "lookup bwd 5000x1537 f32", "op": "lookup_backward", "rows": 5000, "width": 1537,
         "vocab": 50001, "type": "f32", "into": "f32", "add": False, "scale": 0.7, "ignored": 0.3},
        # a training batch against a large vocabulary
        {"name": "lookup bwd 32768x4096 bf16", "op": "lookup_backward", "rows": 32768,
         "width": 4096, "vocab": 131072, "type": "bf16", "into": "bf16", "add": False,
         "scale": 64.0, "ignored": 0.0},
        # a large rollout batch of packed sequences, advantages by token
        {"name": "policy 512 of 1048576", "op": "policy", "rows": 1 << 20, "sequences": 512,
         "advantage": "token", "mean": "token", "ref": True, "ignored": 0.3},
        # the answers of one prompt group: an advantage for each of 16
        # sequences, averaged over sequences
        {"name": "policy bwd 16 of 8191", "op": "policy_backward", "rows": 8191, "sequences": 16,
         "advantage": "sequence", "mean": "sequence", "ref": True, "ignored": 0.3},
        # the gradients of a small model, its tensors one behind the other in a
        # buffer: odd starts
        {"name": "norm 11 tensors f32", "op": "norm", "layers": 1, "width": 65, "vocab": 1001,
         "grad": "f32", "packed": True},
        # all gradients of a model of 1.2e9 parameters
        {"name": "norm 1.2e9 bf16", "op": "norm", "layers": 4, "width": 4096, "vocab": 32768,
         "grad": "bf16", "packed": False},
        # the step of the small model
        {"name": "adamw 11 tensors f32", "op": "adamw", "layers": 1, "width": 65, "vocab": 1001,
         "grad": "f32", "state": 32, "copy": "none", "packed": True},
        # 1.2e9 parameters in FP32 with the BF16 weights that the model runs on
        {"name": "adamw 1.2e9 bf16", "op": "adamw", "layers": 4, "width": 4096, "vocab": 32768,
         "grad": "bf16", "state": 32, "copy": "bf16", "packed": False},
        # states in 8 bits, odd widths
        {"name": "adamw 8-bit 1.9e8 f16", "op": "adamw", "layers": 3, "width": 1537,
         "vocab": 50001, "grad": "f16", "state": 8, "copy": "f16", "packed": False},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["lookup", "lookup_backward", "policy", "policy_backward", "norm", "adamw",
                     "adamw"])
    if op.startswith("lookup"):
        width = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            width = max(64, width // 64 * 64)
        kind = rng.choice(["f32", "bf16", "f16"])
        vocab = _log(rng, 100, min(131072, (1 << 29) // width))
        rows = _log(rng, 1, min(32768, (1 << 27) // width))
        case = {"op": op, "rows": rows, "width": width, "vocab": vocab, "type": kind,
                "scale": rng.choice([1.0, 0.7, round(math.sqrt(width), 3)]),
                "ignored": rng.choice([0.0, 0.0, 0.3]) if rows > 8 else 0.0}
        if op == "lookup_backward":
            case["into"] = rng.choice([kind, kind, "f32"])
            case["add"] = rng.random() < 0.5
        return case
    if op.startswith("policy"):
        rows = _log(rng, 8, 1 << 20)
        return {"op": op, "rows": rows, "sequences": min(rows // 4, _log(rng, 1, 2048)),
                "advantage": rng.choice(["token", "sequence"]),
                "mean": rng.choice(["token", "sequence"]), "ref": rng.random() < 0.6,
                "ignored": rng.choice([0.0, 0.3])}
    width = _log(rng, 64, 4096)
    if rng.random() < 0.6:
        width = max(64, width // 64 * 64)
    case = {"op": op, "layers": rng.randint(1, 4), "width": width, "vocab": _log(rng, 100, 32768),
            "grad": rng.choice(["f32", "bf16", "f16"]), "packed": rng.random() < 0.3}
    if op == "adamw":
        case["state"] = rng.choice([32, 32, 8])
        case["copy"] = rng.choice(["none", "bf16", "f16"])
        case["packed"] = case["packed"] and case["state"] == 32
    return case


# ---- what a program has in hand -----------------------------------------------


def _tokens(case, gen):
    """Tokens of frequencies about 1 / rank, in an order of their own."""
    rows, vocab = case["rows"], case["vocab"]
    u = torch.rand(rows, device="cuda", generator=gen, dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1.0)) - 1.0).long().clamp_(0, vocab - 1)
    token = torch.randperm(vocab, device="cuda", generator=gen)[rank]
    if case["ignored"]:
        token[torch.rand(rows, device="cuda", generator=gen) < case["ignored"]] = IGNORE
    return token


def _lookup_inputs(case, gen):
    t, shape = TYPES[case["type"]], (case["vocab"], case["width"])
    s = {"case": case, "token": _tokens(case, gen)}
    if case["op"] == "lookup":
        s["weight"] = (torch.randn(*shape, device="cuda", generator=gen) * 0.02).to(t)
        return s
    s["dout"] = (torch.randn(case["rows"], case["width"], device="cuda", generator=gen)
                 * 0.01).to(t)
    if case["add"]:
        s["dweight"] = (torch.randn(*shape, device="cuda", generator=gen)
                        * 0.01).to(TYPES[case["into"]])
    return s


def _policy_inputs(case, gen):
    rows, count = case["rows"], case["sequences"]

    def rand(n):
        return torch.rand(n, device="cuda", generator=gen)

    def normal(n):
        return torch.randn(n, device="cuda", generator=gen)

    # packed sequences of uneven lengths, a few of them empty; some rows
    # behind the last one are nobody's
    last = rows - rows // 50
    cuts = torch.randint(last + 1, (count - 1,), device="cuda", generator=gen).sort().values
    offsets = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), last)])
    target = torch.randint(32768, (rows,), device="cuda", generator=gen)
    if case["ignored"]:                          # the prompts
        row = torch.arange(rows, device="cuda")
        of = (torch.searchsorted(offsets, row, right=True) - 1).clamp_(0, count - 1)
        length = (offsets[1:] - offsets[:-1])[of]
        target[(row - offsets[of]).double() < case["ignored"] * length.double()] = IGNORE
    nll = -torch.log(rand(rows).clamp_(min=1e-6)) * 0.8
    # the sampling policy is a few updates behind, the reference further away
    old = (nll + normal(rows) * 0.15).clamp_(min=0.0)
    ref = (nll + normal(rows) * 0.4).clamp_(min=0.0) if case["ref"] else None
    s = {"case": case, "nll": nll, "old": old, "ref": ref, "offsets": offsets, "target": target,
         "advantage": normal(rows if case["advantage"] == "token" else count),
         "kl": KL if case["ref"] else 0.0}
    if case["op"] == "policy_backward":
        s["weights"] = _plain_policy(s)[1]
        s["dloss"] = 0.5 + rand(1)
    return s


def _sizes(case):
    """Elements of a model's tensors: the embedding and, for each layer, four
    projections and three products of a block four times as wide, which decay;
    then two norms for each layer and the last one, which do not."""
    w, layers = case["width"], case["layers"]
    return ([case["vocab"] * w] + [w * w, w * w, w * w, w * w, 4 * w * w, 4 * w * w,
                                   4 * w * w] * layers, [w] * (2 * layers + 1))


def _views(flat, sizes, packed, unit=1):
    """The tensors of a flat buffer, each from a place that is a multiple of
    256 on, or one behind the other."""
    at, out = 0, []
    for n in sizes:
        out.append(flat[at // unit:at // unit + -(-n // unit)])
        at += n if packed else -(-n // BLOCK) * BLOCK
    return out


def _padded(case):
    """(elements that decay, elements in all) of the flat buffers."""
    first, second = ([n if case["packed"] else -(-n // BLOCK) * BLOCK for n in part]
                     for part in _sizes(case))
    return sum(first), sum(first) + sum(second)


def _grads(case, gen):
    """Gradients, about log-normal in size over the tensors; zero between them."""
    sizes, total = sum(_sizes(case), []), _padded(case)[1]
    flat = torch.zeros(total, device="cuda", dtype=TYPES[case["grad"]])
    size = torch.exp(torch.randn(len(sizes), generator=gen, device="cuda")) * 1e-3
    views = _views(flat, sizes, case["packed"])
    for k, v in enumerate(views):
        v.copy_(torch.randn(v.numel(), device="cuda", generator=gen) * size[k])
    return flat, views


def _adamw_inputs(case, gen):
    first, second = _sizes(case)
    sizes, total = first + second, _padded(case)[1]
    grad, grads = _grads(case, gen)
    s = {"case": case, "grad": grad, "grads": grads, "step": 1000,
         "factor": 0.5 + torch.rand(1, device="cuda", generator=gen),
         "decay": [DECAY] * len(first) + [0.0] * len(second)}

    def flat(name, values):
        s[name] = values
        s[name + "s"] = _views(values, sizes, case["packed"])

    live = torch.zeros(total, device="cuda")
    for v in _views(live, sizes, case["packed"]):
        v.fill_(1.0)
    flat("param", torch.randn(total, device="cuda", generator=gen) * 0.02 * live)
    m = (grad.float() * 0.3 + grad.float().abs().mean() * 0.3
         * torch.randn(total, device="cuda", generator=gen)) * live
    v = (m * m * (1.0 + torch.rand(total, device="cuda", generator=gen)))
    del live
    if case["state"] == 8:
        for name, x in (("m", m), ("v", torch.sqrt(v))):
            scale = _block_scale(x)
            flat(name, (x.view(-1, BLOCK) / scale[:, None]).view(-1).to(torch.float8_e4m3fn))
            s[name + "_scale"] = scale
            s[name + "_scales"] = _views(scale, sizes, False, BLOCK)
    else:
        flat("m", m)
        flat("v", v)
    if case["copy"] != "none":
        flat("copy", s["param"].to(TYPES[case["copy"]]))
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"].startswith("lookup"):
        return _lookup_inputs(case, gen)
    if case["op"].startswith("policy"):
        return _policy_inputs(case, gen)
    if case["op"] == "norm":
        flat, views = _grads(case, gen)
        return {"case": case, "grad": flat, "grads": views, "max": 1.0, "scale": 0.5}
    return _adamw_inputs(case, gen)


# ---- the plain forms -----------------------------------------------------------


def _plain_lookup(s):
    valid = s["token"] != IGNORE
    out = s["weight"][torch.where(valid, s["token"], 0)].float() * s["case"]["scale"]
    return torch.where(valid[:, None], out, 0.0).to(s["weight"].dtype)


def _plain_lookup_backward(s):
    case = s["case"]
    valid = s["token"] != IGNORE
    total = torch.zeros(case["vocab"], case["width"], device="cuda")
    rows = torch.where(valid[:, None], s["dout"].float(), 0.0)
    total.index_add_(0, torch.where(valid, s["token"], 0), rows)
    total *= case["scale"]
    if not case["add"]:
        return total.to(TYPES[case["into"]])
    return s["dweight"].copy_(s["dweight"].float() + total)


def _sequence_of_rows(s):
    """The sequence of each row, and whether the row counts."""
    row = torch.arange(s["nll"].shape[0], device=s["nll"].device)
    of = torch.searchsorted(s["offsets"], row, right=True) - 1
    count = s["offsets"].shape[0] - 1
    return of.clamp(0, count - 1), (of >= 0) & (of < count) & (s["target"] != IGNORE)


def _policy_parts(s):
    of, counts = _sequence_of_rows(s)
    adv = s["advantage"] if s["case"]["advantage"] == "token" else s["advantage"][of]
    log_ratio = s["old"].double() - s["nll"].double()
    high = log_ratio > math.log1p(torch.tensor(CLIP_HIGH).item())
    low = log_ratio < math.log1p(-torch.tensor(CLIP_LOW).item())
    clipped = counts & ((high & (adv > 0)) | (low & (adv < 0)))
    return of, counts, adv, log_ratio.float(), clipped


def _plain_policy(s):
    of, counts, adv, log_ratio, clipped = _policy_parts(s)
    ratio = torch.where(clipped, torch.where(adv > 0, 1.0 + CLIP_HIGH, 1.0 - CLIP_LOW),
                        torch.exp(log_ratio))
    surrogate = torch.where(counts, -ratio * adv, 0.0)
    kl = torch.zeros_like(surrogate)
    if s["ref"] is not None:
        q = s["nll"] - s["ref"]
        kl = torch.where(counts, torch.expm1(q) - q, 0.0)
    per = torch.zeros(s["offsets"].shape[0] - 1, device="cuda", dtype=torch.float64)
    n = per.index_add(0, of, counts.double())
    if s["case"]["mean"] == "token":
        weights = (1.0 / n.sum().clamp(min=1.0)).expand_as(n)
    else:
        weights = torch.where(n > 0, 1.0 / (n.clamp(min=1.0) * (n > 0).sum().clamp(min=1)), 0.0)
    w = weights[of]
    means = [(w * x.double()).sum() for x in (surrogate, kl, clipped)]
    stats = torch.stack([means[0] + s["kl"] * means[1], *means])
    return stats.float(), weights.float()


def _plain_policy_backward(s):
    of, counts, adv, log_ratio, clipped = _policy_parts(s)
    d = torch.where(clipped, 0.0, torch.exp(log_ratio) * adv)
    if s["ref"] is not None:
        d = d + s["kl"] * torch.expm1(s["nll"] - s["ref"])
    return torch.where(counts, d * s["weights"][of] * s["dloss"], 0.0)


def _plain_norm(s):
    g = s["grad"].float()
    norm = (torch.sqrt((g * g).sum(dtype=torch.float64)) * s["scale"]).float()
    factor = s["scale"] * torch.where(norm > s["max"], s["max"] / norm, 1.0)
    return torch.stack([norm, factor])


def _block_scale(x):
    """A power of two for each 256 values: the largest comes to 128 to 256 of it."""
    top = x.view(-1, BLOCK).abs().amax(1)
    power = torch.ldexp(torch.ones_like(top), torch.frexp(top).exponent - 8)
    return torch.where(top < 2.0 ** -100, 1.0, power)


def _mix(z):
    """SplitMix64's finalizer on int64 tensors (products wrap, shifts are made logical)."""
    z = (z ^ ((z >> 30) & ((1 << 34) - 1))) * -0x40A7B892E31B1A47
    z = (z ^ ((z >> 27) & ((1 << 37) - 1))) * -0x6B2FB644ECCEEE15
    return z ^ ((z >> 31) & ((1 << 33) - 1))


GOLDEN = -0x61C8864680B583EB


def _random_words(s):
    """32 random bits for each element: of the step, the tensor and the element."""
    sizes = sum(_sizes(s["case"]), [])
    room = torch.tensor([-(-n // BLOCK) * BLOCK for n in sizes], device="cuda")
    which = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), room)
    element = torch.arange(which.shape[0], device="cuda") - (room.cumsum(0) - room)[which]
    key = _mix(torch.full((), s["step"], device="cuda", dtype=torch.int64) * GOLDEN)
    key = _mix(key + (which + 1) * GOLDEN)
    word = _mix(key + ((element >> 1) + 1) * GOLDEN)
    return torch.where((element & 1) == 1, word >> 32, word) & 0xFFFFFFFF


def _round_at_random(x, scale, bits, never_zero):
    """x / scale in e4m3, up with the probability of what is cut off: 16 random
    bits are added below the three mantissa bits that stay.  Magnitudes under
    2^-6 are moved up by 2^-6, where these three bits are the type's last step."""
    y = (x.view(-1, BLOCK) / scale[:, None]).view(-1)
    size = y.abs()
    base = torch.where(size < 2.0 ** -6, 2.0 ** -6, 0.0)
    word = (size + base).view(torch.int32) + (bits << 4).to(torch.int32)
    size = (word & -0x100000).view(torch.float32) - base
    if never_zero:
        size = torch.where(y > 0, size.clamp(min=2.0 ** -9), size)
    return torch.where(y < 0, -size, size).to(torch.float8_e4m3fn)


def _plain_adamw(s):
    case, step = s["case"], s["step"]
    split, p = _padded(case)[0], s["param"]
    g = s["grad"].float() * s["factor"]
    if case["state"] == 8:
        m = (s["m"].float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        v = (s["v"].float().view(-1, BLOCK) * s["v_scale"][:, None]).view(-1).square_()
    else:
        m, v = s["m"], s["v"]
    m.mul_(BETA1).add_(g * (1.0 - BETA1))
    v.mul_(BETA2).add_(g * g * (1.0 - BETA2))
    denominator = torch.sqrt(v) / math.sqrt(1.0 - BETA2 ** step) + EPS
    p[:split].mul_(1.0 - LR * DECAY)
    p.sub_(m / denominator * (LR / (1.0 - BETA1 ** step)))
    if case["state"] == 8:
        words = _random_words(s)
        for name, x, bits in (("m", m, words & 0xFFFF), ("v", torch.sqrt(v), words >> 16)):
            scale = _block_scale(x)
            s[name].copy_(_round_at_random(x, scale, bits, name == "v"))
            s[name + "_scale"].copy_(scale)
    if case["copy"] != "none":
        s["copy"].copy_(p)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    return {k: s[k] for k in ("param", "copy", "m", "v", "m_scale", "v_scale") if k in s}


# ---- the library's calls ---------------------------------------------------------


def _own(s):
    import tile_compiler_row_gb300 as tile
    case, op = s["case"], s["case"]["op"]
    if op == "lookup":
        return tile.embedding(s["token"], s["weight"], scale=case["scale"], ignore_index=IGNORE)
    if op == "lookup_backward":
        return tile.embedding_backward(
            s["token"], s["dout"], case["vocab"], scale=case["scale"], ignore_index=IGNORE,
            dtype=TYPES[case["into"]], dweight=s["dweight"] if case["add"] else None)
    if op.startswith("policy"):
        common = dict(ref_nll=s["ref"], target=s["target"], offsets=s["offsets"],
                      per_sequence=case["advantage"] == "sequence", clip_low=CLIP_LOW,
                      clip_high=CLIP_HIGH, kl_coef=s["kl"], ignore_index=IGNORE)
        if op == "policy":
            return tile.policy_loss(s["nll"], s["old"], s["advantage"], mean=case["mean"],
                                    **common)
        return tile.policy_loss_backward(s["nll"], s["old"], s["advantage"], s["weights"],
                                         s["dloss"], **common)
    if op == "norm":
        return tile.grad_norm(s["grads"], max_norm=s["max"], scale=s["scale"])
    tile.adamw(s["params"], s["grads"], s["ms"], s["vs"], step=s["step"], lr=LR,
               betas=(BETA1, BETA2), eps=EPS, weight_decay=s["decay"], factor=s["factor"],
               copies=s.get("copys"), exp_avg_scales=s.get("m_scales"),
               exp_avg_sq_scales=s.get("v_scales"))
    return _adamw_outputs(s)


def run(state):
    if own:
        return _own(state)
    return {"lookup": _plain_lookup, "lookup_backward": _plain_lookup_backward,
            "policy": _plain_policy, "policy_backward": _plain_policy_backward,
            "norm": _plain_norm, "adamw": _plain_adamw}[state["case"]["op"]](state)


def _distinct(case):
    """Expected number of different tokens."""
    vocab, n = case["vocab"], case["rows"] * (1.0 - case["ignored"])
    v = torch.arange(vocab, dtype=torch.float64)
    p = (torch.log(v + 2.0) - torch.log(v + 1.0)) / math.log(vocab + 1.0)
    return float((1.0 - torch.exp(n * torch.log1p(-p))).sum()) if vocab > 1 else 1.0


def work(case):
    if case["op"].startswith("lookup"):
        rows, width, size = case["rows"], case["width"], BYTES[case["type"]]
        if case["op"] == "lookup":
            return {"bytes": (rows + _distinct(case)) * width * size + 8 * rows,
                    "flops": rows * width}
        valid = rows * (1.0 - case["ignored"])
        into = 2 * _distinct(case) if case["add"] else case["vocab"]
        return {"bytes": (valid * size + into * BYTES[case["into"]]) * width + 8 * rows,
                "flops": valid * width}
    if case["op"].startswith("policy"):
        rows, count = case["rows"], case["sequences"]
        read = 3 + (1 if case["ref"] else 0) + (1 if case["op"] == "policy_backward" else 0)
        read += 1 if case["advantage"] == "token" else 0
        return {"bytes": 4 * rows * (read + 1) + 16 * count, "flops": 20 * rows}
    n = sum(sum(_sizes(case), []))
    if case["op"] == "norm":
        return {"bytes": n * BYTES[case["grad"]], "flops": 2 * n}
    state = 16 if case["state"] == 32 else 4 + 16 / BLOCK
    copy = 0 if case["copy"] == "none" else 2
    return {"bytes": n * (8 + state + BYTES[case["grad"]] + copy), "flops": 15 * n}


# ---- the definitions in 64 bits ------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"lookup": _exact_lookup, "lookup_backward": _exact_lookup_backward,
            "policy": _exact_policy, "policy_backward": _exact_policy_backward,
            "norm": _exact_norm, "adamw": _exact_adamw}[case["op"]](s)


def _exact_lookup(s):
    out = s["weight"].double()[s["token"].clamp(min=0)] * s["case"]["scale"]
    out[s["token"] == IGNORE] = 0.0
    return out


def _exact_lookup_backward(s):
    case = s["case"]
    out = s["dweight"].double() if case["add"] else torch.zeros(
        case["vocab"], case["width"], device="cuda", dtype=torch.float64)
    keep = s["token"] != IGNORE
    return out.index_put_((s["token"][keep],), s["dout"][keep].double() * case["scale"],
                          accumulate=True)


def _exact_rows(s):
    """Each row's sequence (-1: none), from the lengths, and whether it counts."""
    start, end = s["offsets"][:-1], s["offsets"][1:]
    of = torch.full_like(s["target"], -1)
    of[int(start[0]):int(end[-1])] = torch.repeat_interleave(
        torch.arange(start.shape[0], device="cuda"), end - start)
    keep = (of >= 0) & (s["target"] != IGNORE)
    adv = s["advantage"].double()
    adv = adv if s["case"]["advantage"] == "token" else adv[of.clamp(min=0)]
    ratio = torch.exp(s["old"].double() - s["nll"].double())
    return of, keep, adv, ratio


def _exact_policy(s):
    of, keep, adv, ratio = _exact_rows(s)
    lo, hi = (1.0 + torch.tensor([-CLIP_LOW, CLIP_HIGH]).double()).tolist()
    plain, bounded = ratio * adv, ratio.clamp(lo, hi) * adv
    q = (s["nll"].double() - s["ref"].double()) if s["ref"] is not None else 0.0 * adv
    parts = torch.stack([-torch.minimum(plain, bounded), torch.exp(q) - q - 1.0,
                         (bounded < plain).double()], 1)
    count = s["offsets"].shape[0] - 1
    n = torch.bincount(of[keep], minlength=count).double()
    if s["case"]["mean"] == "token":
        weights = torch.ones_like(n) / max(1.0, float(n.sum()))
    else:
        weights = (n > 0) / n.clamp(min=1.0) / max(1, int((n > 0).sum()))
    means = (parts[keep] * weights[of[keep]][:, None]).sum(0)
    return torch.cat([(means[0] + s["kl"] * means[1])[None], means]), weights


def _exact_policy_backward(s):
    of, keep, adv, ratio = _exact_rows(s)
    lo, hi = (1.0 + torch.tensor([-CLIP_LOW, CLIP_HIGH]).double()).tolist()
    held = ratio.clamp(lo, hi) * adv < ratio * adv
    d = ratio * adv * (~held)
    if s["ref"] is not None:
        d += s["kl"] * (torch.exp(s["nll"].double() - s["ref"].double()) - 1.0)
    d *= s["weights"].double()[of.clamp(min=0)] * s["dloss"].double()
    return d * keep


def _exact_norm(s):
    norm = s["scale"] * torch.linalg.vector_norm(s["grad"].double())
    return torch.stack([norm, s["scale"] * (s["max"] / norm).clamp(max=1.0)])


def _exact_adamw(s):
    case, step = s["case"], s["step"]
    g = s["grad"].double() * s["factor"].double()
    eight = case["state"] == 8
    if eight:
        m, v = (s[k].double() * s[k + "_scale"].double().repeat_interleave(BLOCK) for k in "mv")
        v = v * v
    else:
        m, v = s["m"].double(), s["v"].double()
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * g.square()
    decay = torch.zeros_like(g)
    decay[:_padded(case)[0]] = DECAY
    p = s["param"].double()
    p = p - LR * (decay * p + m / (1.0 - BETA1 ** step)
                  / ((v / (1.0 - BETA2 ** step)).sqrt() + EPS))
    out = {"param": p, "m": m, "v": v}
    if case["copy"] != "none":
        out["copy"] = p
    if eight:
        words = _random_words(s)
        for name, x, bits in (("m", m, words % 65536), ("v", v.sqrt(), words // 65536)):
            top = x.reshape(-1, BLOCK).abs().amax(1)
            scale = torch.where(top < 2.0 ** -100, 1.0, torch.exp2(
                torch.floor(torch.log2(top.clamp(min=2.0 ** -126))) - 7.0))
            y = x / scale.repeat_interleave(BLOCK)
            place = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
            unit = torch.exp2(place - 3.0)
            code = torch.floor(y.abs() / unit + bits / 65536.0) * unit
            if name == "v":
                code = torch.where(y > 0, code.clamp(min=2.0 ** -9), code)
            out[name], out[name + "_scale"] = code * y.sign(), scale
    return out
