"""The block norm and the linear cross entropy, forward and backward, as
measured cases.

Four operators, each with a plain form in elementary torch operations (FP32,
rounded once at the end) and, where ``own`` is true, the library's call:

  block_norm            h = a r + gate * post(b), y = pre(h): the RMSNorm after
                        a block's output, its gate, the scaled residual sum and
                        the RMSNorm before the next block
  block_norm_backward   its input and parameter gradients
  cross_entropy         lse = log sum exp(x W^T), loss = lse - (x W^T)[target]
                        for every token, the logits of the vocabulary not kept
  cross_entropy_backward  dx = g W, dW = g^T x, g = (softmax - onehot) dloss

``exact`` states the same definitions once more in FP64.
"""

import math

import torch

own = False

EPS = 1e-5
IGNORE = -100
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # four sequences decode one token each: between two blocks, one call
        {"name": "norm 4x2048 bf16", "op": "block_norm", "rows": 4, "width": 2048, "type": "bf16",
         "post": True, "pre": True, "gate": 0, "scale": 1.0},
        # a training step's residual stream, norms on both sides, a learned
        # gate for each channel
        {"name": "norm 16384x4096 bf16", "op": "block_norm", "rows": 16384, "width": 4096,
         "type": "bf16", "post": True, "pre": True, "gate": 16384, "scale": 1.0},
        # FP32 rows of an odd width, gates conditioned on each sequence of
        # 600 tokens (the last one shorter), a residual scale
        {"name": "norm 5000x1537 f32", "op": "block_norm", "rows": 5000, "width": 1537,
         "type": "f32", "post": True, "pre": True, "gate": 600, "scale": 0.7},
        # a small batch, no norm after the block and no gate: the ordinary
        # residual sum with its norm, odd width
        {"name": "norm bwd 511x1537 f16", "op": "block_norm_backward", "rows": 511, "width": 1537,
         "type": "f16", "post": False, "pre": True, "gate": 0, "scale": 1.0},
        # FP32 training rows with a gate for each sequence of 512 tokens
        {"name": "norm bwd 4096x8192 f32", "op": "block_norm_backward", "rows": 4096,
         "width": 8192, "type": "f32", "post": True, "pre": True, "gate": 512, "scale": 0.7},
        # the backward pass of a long training batch
        {"name": "norm bwd 32768x4096 bf16", "op": "block_norm_backward", "rows": 32768,
         "width": 4096, "type": "bf16", "post": True, "pre": True, "gate": 32768, "scale": 1.0},
        # scoring the few tokens of an answer
        {"name": "loss 5x2048x32768 bf16", "op": "cross_entropy", "rows": 5, "width": 2048,
         "vocab": 32768, "type": "bf16", "ignored": 0.0},
        # a ragged fine-tuning batch with prompts masked out; nothing is a
        # multiple of a tile
        {"name": "loss 1000x1537x50001 f16", "op": "cross_entropy", "rows": 1000, "width": 1537,
         "vocab": 50001, "type": "f16", "ignored": 0.3},
        # a training step's tokens against a large vocabulary
        {"name": "loss 4096x4096x131072 bf16", "op": "cross_entropy", "rows": 4096, "width": 4096,
         "vocab": 131072, "type": "bf16", "ignored": 0.0},
        # one short sequence
        {"name": "loss bwd 48x1024x32768 bf16", "op": "cross_entropy_backward", "rows": 48,
         "width": 1024, "vocab": 32768, "type": "bf16", "ignored": 0.0},
        # a fine-tuning batch, two fifths of it masked; an odd vocabulary
        {"name": "loss bwd 2047x2048x65537 f16", "op": "cross_entropy_backward", "rows": 2047,
         "width": 2048, "vocab": 65537, "type": "f16", "ignored": 0.4},
        # a training step's tokens against a large vocabulary
        {"name": "loss bwd 4096x4096x131072 bf16", "op": "cross_entropy_backward", "rows": 4096,
         "width": 4096, "vocab": 131072, "type": "bf16", "ignored": 0.0},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["block_norm", "block_norm_backward", "cross_entropy",
                     "cross_entropy_backward"])
    if op.startswith("block"):
        kind = rng.choice(["f32", "bf16", "f16"])
        width = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            width = max(64, width // 64 * 64)
        rows = _log(rng, 1, max(1, min(32768, (1 << 26) // width)))
        post = rng.random() < 0.7
        pre = rng.random() < 0.8 or not post
        gate = rng.choice([0, rows, max(1, rows // 8), max(1, rows // 3)])
        return {"op": op, "rows": rows, "width": width, "type": kind, "post": post, "pre": pre,
                "gate": gate, "scale": rng.choice([1.0, 0.7])}
    kind = rng.choice(["bf16", "f16"])
    rows = _log(rng, 1, 4096)
    width = _log(rng, 64, 4096)
    if rng.random() < 0.7:
        width = max(64, width // 64 * 64)
    vocab = _log(rng, 1000, 131072)
    if rng.random() < 0.5:
        vocab = vocab // 8 * 8
    return {"op": op, "rows": rows, "width": width, "vocab": vocab, "type": kind,
            "ignored": rng.choice([0.0, 0.0, 0.25, 0.6])}


def _block_inputs(case, gen):
    rows, width, t = case["rows"], case["width"], TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    s = {"case": case, "x": (normal(rows, width) * 1.5).to(t),
         # the residual stream is larger than a block's output, and has a few
         # channels that stand out
         "residual": (normal(rows, width) * (1.0 + 8.0 * (torch.rand(width, device="cuda", generator=gen) < 0.01))
                      * 3.0).to(t),
         "gamma_post": 1.0 + 0.2 * normal(width) if case["post"] else None,
         "gamma_pre": 1.0 + 0.2 * normal(width) if case["pre"] else None,
         "gate": None}
    if case["gate"]:
        s["gate"] = 0.5 + 0.25 * normal(-(-rows // case["gate"]), width)
    if case["op"] == "block_norm_backward":
        s["hidden"] = _plain_block(s)[0]
        s["dhidden"] = (normal(rows, width) * 0.01).to(t)
        s["dout"] = (normal(rows, width) * 0.02).to(t) if case["pre"] else None
        del s["residual"]
    return s


def _loss_inputs(case, gen):
    rows, width, vocab, t = case["rows"], case["width"], case["vocab"], TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    weight = (normal(vocab, width) * (1.5 / math.sqrt(width))).to(t)
    target = torch.randint(vocab, (rows,), device="cuda", generator=gen)
    # hidden rows that lean towards their target, as a trained model's do (by
    # up to 0.7 log vocab): some targets are likely, some are not
    lean = 0.7 * math.log(vocab) / 1.5 ** 2 * torch.rand(rows, 1, device="cuda", generator=gen)
    x = (normal(rows, width) + lean * weight[target].float()).to(t)
    if case["ignored"]:
        target[torch.rand(rows, device="cuda", generator=gen) < case["ignored"]] = IGNORE
    s = {"case": case, "x": x, "weight": weight, "target": target}
    if case["op"] == "cross_entropy_backward":
        s["lse"] = _plain_loss(s)[1]
        valid = target != IGNORE
        s["dloss"] = valid.float() / valid.sum().clamp(min=1)      # of the mean loss
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return _block_inputs(case, gen) if case["op"].startswith("block") else _loss_inputs(case, gen)


# ---- the plain forms -----------------------------------------------------------


def _rstd(v):
    return 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)


def _gate_of_rows(s):
    if s["gate"] is None:
        return 1.0
    rows = torch.arange(s["x"].shape[0], device=s["x"].device)
    return s["gate"][rows // s["case"]["gate"]]


def _plain_block(s):
    case, t = s["case"], s["x"].dtype
    n = s["x"].float()
    if case["post"]:
        n = n * _rstd(n) * s["gamma_post"]
    h = case["scale"] * s["residual"].float() + _gate_of_rows(s) * n
    y = (h * _rstd(h) * s["gamma_pre"]).to(t) if case["pre"] else None
    return h.to(t), y


def _plain_block_backward(s):
    case, t = s["case"], s["x"].dtype
    b, h, gate = s["x"].float(), s["hidden"].float(), _gate_of_rows(s)
    dh, dgamma_pre = s["dhidden"].float(), None
    if case["pre"]:
        dy, r = s["dout"].float(), _rstd(h)
        hat, g = h * r, dy * s["gamma_pre"]
        dh = dh + r * (g - hat * (g * hat).mean(1, keepdim=True))
        dgamma_pre = (dy * hat).sum(0)
    dresidual = case["scale"] * dh
    dn, dgamma_post, n = dh * gate, None, b
    if case["post"]:
        r = _rstd(b)
        hat, g = b * r, dn * s["gamma_post"]
        db = r * (g - hat * (g * hat).mean(1, keepdim=True))
        dgamma_post = (dn * hat).sum(0)
        n = hat * s["gamma_post"]
    else:
        db = dn
    dgate = None
    if s["gate"] is not None:
        rows, per = b.shape[0], case["gate"]
        group = torch.arange(rows, device=b.device) // per
        dgate = torch.zeros_like(s["gate"])
        if dgate.shape[0] == 1:
            dgate = (dh * n).sum(0, keepdim=True)
        else:
            dgate.index_add_(0, group, dh * n)
    return {"din": db.to(t), "dresidual": dresidual.to(t), "dgamma_post": dgamma_post,
            "dgate": dgate, "dgamma_pre": dgamma_pre}


def _logits(s):
    return s["x"].float() @ s["weight"].float().t()


def _plain_loss(s):
    valid = s["target"] != IGNORE
    logits = _logits(s)
    top = logits.amax(1)
    lse = top + torch.log(torch.exp(logits - top[:, None]).sum(1))
    at = logits.gather(1, torch.where(valid, s["target"], 0)[:, None])[:, 0]
    zero = torch.zeros_like(lse)
    return torch.where(valid, lse - at, zero), torch.where(valid, lse, zero)


def _plain_loss_backward(s):
    t, valid = s["x"].dtype, s["target"] != IGNORE
    g = torch.exp(_logits(s) - s["lse"][:, None])
    rows = torch.arange(g.shape[0], device=g.device)
    g[rows, torch.where(valid, s["target"], 0)] -= 1.0
    g *= torch.where(valid, s["dloss"], 0.0)[:, None]
    return {"dx": (g @ s["weight"].float()).to(t), "dweight": (g.t() @ s["x"].float()).to(t)}


# ---- the library's calls ---------------------------------------------------------


def _own(s):
    import tile_compiler_row_gb300 as tile
    case = s["case"]
    if case["op"] == "block_norm":
        return tile.block_norm(s["x"], s["residual"], s["gamma_post"], s["gate"], s["gamma_pre"],
                               post=case["post"], pre=case["pre"], rows_per_gate=case["gate"],
                               residual_scale=case["scale"], eps=EPS)
    if case["op"] == "block_norm_backward":
        din, dresidual, dgamma_post, dgate, dgamma_pre = tile.block_norm_backward(
            s["x"], s["hidden"], s["gamma_post"], s["gate"], s["gamma_pre"], s["dhidden"],
            s["dout"], post=case["post"], pre=case["pre"], rows_per_gate=case["gate"],
            residual_scale=case["scale"], eps=EPS)
        return {"din": din, "dresidual": dresidual, "dgamma_post": dgamma_post, "dgate": dgate,
                "dgamma_pre": dgamma_pre}
    if case["op"] == "cross_entropy":
        return tile.linear_cross_entropy(s["x"], s["weight"], s["target"], ignore_index=IGNORE)
    dx, dweight = tile.linear_cross_entropy_backward(s["x"], s["weight"], s["target"], s["lse"],
                                                     s["dloss"], ignore_index=IGNORE)
    return {"dx": dx, "dweight": dweight}


def run(state):
    if own:
        return _own(state)
    return {"block_norm": _plain_block, "block_norm_backward": _plain_block_backward,
            "cross_entropy": _plain_loss,
            "cross_entropy_backward": _plain_loss_backward}[state["case"]["op"]](state)


def work(case):
    rows, width, size = case["rows"], case["width"], BYTES[case["type"]]
    if case["op"].startswith("block"):
        gates = -(-rows // case["gate"]) if case["gate"] else 0
        params = 4 * width * (case["post"] + case["pre"] + gates)
        matrix = rows * width * size
        if case["op"] == "block_norm":
            return {"bytes": matrix * (4 if case["pre"] else 3) + params,
                    "flops": 10 * rows * width}
        # x, hidden (only its norm's gradient needs it), dhidden, dout, din, dresidual
        read = (2 if case["post"] or case["gate"] else 1) + (2 if case["pre"] else 0)
        return {"bytes": matrix * (read + 2) + 2 * params, "flops": 24 * rows * width}
    vocab = case["vocab"]
    valid = rows * (1.0 - case["ignored"])
    io = (valid * width + vocab * width) * size
    if case["op"] == "cross_entropy":
        return {"bytes": io + 16 * rows, "flops": 2.0 * valid * width * vocab}
    return {"bytes": io + (rows * width + vocab * width) * size + 16 * rows,
            "flops": 6.0 * valid * width * vocab}


# ---- the definitions in 64 bits ------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "block_norm":
        return _exact_block(s)
    if case["op"] == "block_norm_backward":
        return _exact_block_backward(s)
    # FP64 products run at about 1 TFLOP/s
    if 2.0 * case["rows"] * case["width"] * case["vocab"] > 5e12:
        return None
    return _exact_loss(s) if case["op"] == "cross_entropy" else _exact_loss_backward(s)


def _exact_gate(s):
    rows, width = s["x"].shape
    if s["gate"] is None:
        return torch.ones(1, 1, device="cuda", dtype=torch.float64)
    return s["gate"].double().repeat_interleave(s["case"]["gate"], 0)[:rows]


def _exact_block(s):
    case, width = s["case"], s["x"].shape[1]
    b, r = s["x"].double(), s["residual"].double()
    if case["post"]:
        b = b * (b.pow(2).sum(1, keepdim=True) / width + EPS).pow(-0.5) * s["gamma_post"].double()
    h = r * case["scale"] + b * _exact_gate(s)
    if not case["pre"]:
        return h, None
    return h, h * (h.pow(2).sum(1, keepdim=True) / width + EPS).pow(-0.5) * s["gamma_pre"].double()


def _exact_block_backward(s):
    """Jacobians of the norms applied as (I - v v^T / (n (ms + eps))) / rms."""
    case, width = s["case"], s["x"].shape[1]
    b, h, gate = s["x"].double(), s["hidden"].double(), _exact_gate(s)
    flow, dgamma_pre = s["dhidden"].double(), None
    if case["pre"]:
        power = h.pow(2).sum(1, keepdim=True) / width + EPS
        up = s["dout"].double() * s["gamma_pre"].double()
        flow = flow + (up - h * ((up * h).sum(1, keepdim=True) / (width * power))) / power.sqrt()
        dgamma_pre = (s["dout"].double() * h / power.sqrt()).sum(0)
    normed, dgamma_post, din = b, None, flow * gate
    if case["post"]:
        power = b.pow(2).sum(1, keepdim=True) / width + EPS
        unit = b / power.sqrt()
        dgamma_post = (din * unit).sum(0)
        normed = unit * s["gamma_post"].double()
        up = din * s["gamma_post"].double()
        din = (up - b * ((up * b).sum(1, keepdim=True) / (width * power))) / power.sqrt()
    dgate = None
    if s["gate"] is not None:
        dgate = torch.stack([p.sum(0) for p in (flow * normed).split(case["gate"])])
    return {"din": din, "dresidual": flow * case["scale"], "dgamma_post": dgamma_post,
            "dgate": dgate, "dgamma_pre": dgamma_pre}


def _exact_loss(s):
    weight, loss, lse = s["weight"].double(), [], []
    for x, target in zip(s["x"].split(512), s["target"].split(512)):
        logits = torch.einsum("th,vh->tv", x.double(), weight)
        z = torch.logsumexp(logits, 1)
        picked = (x.double() * weight[target.clamp(min=0)]).sum(1)
        loss.append(torch.where(target == IGNORE, 0.0, z - picked))
        lse.append(torch.where(target == IGNORE, 0.0, z))
    return torch.cat(loss), torch.cat(lse)


def _exact_loss_backward(s):
    weight, dweight, dx = s["weight"].double(), 0.0, []
    columns = torch.arange(weight.shape[0], device="cuda")
    for x, target, lse, dloss in zip(s["x"].split(512), s["target"].split(512),
                                     s["lse"].split(512), s["dloss"].split(512)):
        x = x.double()
        p = torch.exp(torch.einsum("th,vh->tv", x, weight) - lse.double()[:, None])
        g = (p - (columns == target[:, None]).double()) * dloss.double()[:, None]
        g[target == IGNORE] = 0.0
        dx.append(torch.einsum("tv,vh->th", g, weight))
        dweight = dweight + torch.einsum("tv,th->vh", g, x)
    return {"dx": torch.cat(dx), "dweight": dweight}
