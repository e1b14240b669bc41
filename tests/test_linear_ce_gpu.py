"""The linear cross entropy and its gradients against FP64.

Tolerances count roundings.  Products of 16-bit elements are exact; a logit
is a sum over the width that the tensor cores add 16 products at a time,
each step truncated to no fewer than FP32's 24 bits: with L = sum |x w| its
error is at most e = (width / 16 + 2) 2^-22 L.  lse is off by at most the
largest e of its row, and by 2^-17 for the exponentials and their sum
(ex2 2^-22, at most 256 + vocab / 256 / 32 + 16 additions of 2^-24) and
logarithm.  A gradient g = (p - onehot) dloss has p off by p (e + the lse's
2^-20 |lse|) and is rounded once to 16 bits, and what it is summed into adds
FP32 roundings (the same bound as a logit's) and one rounding."""

import pytest
import torch

import tile_compiler_row_gb300 as tile

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def device():
    from tile_compiler_row_gb300 import _build
    _build.build()
    tile.load()
    torch.cuda.set_device(0)


def make(rows, width, vocab, kind, ignored=0.0, seed=3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[kind]
    weight = (torch.randn(vocab, width, device="cuda", generator=gen) * 1.5 / width ** 0.5).to(t)
    target = torch.randint(vocab, (rows,), device="cuda", generator=gen)
    x = (torch.randn(rows, width, device="cuda", generator=gen) + weight[target].float()).to(t)
    if ignored:
        target[torch.rand(rows, device="cuda", generator=gen) < ignored] = -100
    dloss = torch.rand(rows, device="cuda", generator=gen) / rows
    return x, weight, target, dloss


def sum_error(n):
    """Relative error of a sum of n exact products against the sum of their
    absolute values."""
    return (n / 16 + 2) * 2.0 ** -22


def reference(x, weight, target):
    x, weight = x.double(), weight.double()
    logits, mag = x @ weight.t(), x.abs() @ weight.abs().t()
    valid = target != -100
    lse = torch.logsumexp(logits, 1)
    at = logits.gather(1, target.clamp(min=0)[:, None])[:, 0]
    tol = sum_error(x.shape[1]) * mag.amax(1) + 2.0 ** -17
    zero = torch.zeros_like(lse)
    return (torch.where(valid, lse - at, zero), torch.where(valid, lse, zero), tol, logits, mag)


def check_loss(x, weight, target, loss, lse):
    want, want_lse, tol, _, _ = reference(x, weight, target)
    assert loss.dtype == lse.dtype == torch.float32
    assert ((lse.double() - want_lse).abs() <= tol + 2.0 ** -23 * want_lse.abs()).all()
    assert ((loss.double() - want).abs() <= 2 * tol + 2.0 ** -23 * want.abs()).all()
    assert not loss[target == -100].any() and not lse[target == -100].any()


def check_gradients(x, weight, target, lse, dloss, dx, dweight):
    _, _, _, logits, mag = reference(x, weight, target)
    valid = (target != -100)[:, None]
    p = torch.where(valid, torch.exp(logits - lse.double()[:, None]), 0.0)
    off = sum_error(x.shape[1]) * mag + 2.0 ** -20 * (1 + lse.double().abs()[:, None])
    onehot = torch.zeros_like(p)
    onehot.scatter_(1, target.clamp(min=0)[:, None], 1.0)
    onehot *= valid
    dl = dloss.double()[:, None]
    g = (p - onehot) * dl
    half = torch.finfo(x.dtype).eps / 2
    # FP16 g: values are held to a step of 2^-39 of the largest dloss
    least = 2.0 ** -39 * dloss.abs().max().double() if x.dtype == torch.float16 else 0.0
    gerr = half * g.abs() + (p * off + 2.0 ** -22 * onehot) * dl.abs() + least * valid
    tiny = torch.finfo(x.dtype).smallest_normal * torch.finfo(x.dtype).eps
    for got, ref, err, name in (
            (dx, g @ weight.double(),
             gerr @ weight.double().abs() + sum_error(p.shape[1]) * (g.abs() @ weight.double().abs()),
             "dx"),
            (dweight, g.t() @ x.double(),
             gerr.t() @ x.double().abs() + sum_error(p.shape[0]) * (g.abs().t() @ x.double().abs()),
             "dweight")):
        tol = half * ref.abs() + 1.01 * err + tiny
        bad = ~((got.double() - ref).abs() <= tol)
        assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} values off, the first "
                               f"at {bad.nonzero()[0].tolist()}: {got[bad][0].item()} for "
                               f"{ref[bad][0].item()}, tolerance {tol[bad][0].item():.3e}")
        # in the 2-norm the roundings are independent: no more than the
        # output's and g's together
        if ref.norm() > 0 and name == "dx":
            assert (got.double() - ref).norm() <= 4 * half * ref.norm() + tiny * ref.numel() ** 0.5


# one token, one column, one class; around the tiles of 128 rows, 64 and 256
# columns; odd widths and vocabularies; vocabularies split among CTAs
# (few rows of many columns, many rows and entries of few)
SHAPES = [(3, 9001, 700), (70, 16384, 300), (17000, 64, 520), (2, 64, 300001), (1, 1, 1), (1, 8, 2), (2, 3, 5), (1, 64, 1000), (5, 72, 257), (17, 100, 256),
          (127, 64, 255), (128, 128, 512), (129, 136, 511), (130, 65, 777), (256, 256, 300),
          (300, 520, 1025), (3, 2048, 9000), (64, 333, 20011), (1000, 96, 3001), (257, 1537, 640)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,width,vocab", SHAPES)
def test_loss_and_gradients(rows, width, vocab, kind):
    x, weight, target, dloss = make(rows, width, vocab, kind, 0.3 if rows > 2 else 0.0)
    loss, lse = tile.linear_cross_entropy(x, weight, target)
    check_loss(x, weight, target, loss, lse)
    dx, dweight = tile.linear_cross_entropy_backward(x, weight, target, lse, dloss)
    assert dx.dtype == dweight.dtype == x.dtype
    check_gradients(x, weight, target, lse, dloss, dx, dweight)
    assert tile.tile_check_device_status() == 0


def test_pieces_of_the_vocabulary():
    """More columns than one piece holds, in both element types; one of the
    two gradients alone is the same as with the other."""
    rows, width, vocab = 4100, 64, 70001
    for kind in TYPES:
        x, weight, target, dloss = make(rows, width, vocab, kind, 0.1)
        loss, lse = tile.linear_cross_entropy(x, weight, target)
        check_loss(x, weight, target, loss, lse)
        dx, dweight = tile.linear_cross_entropy_backward(x, weight, target, lse, dloss)
        check_gradients(x, weight, target, lse, dloss, dx, dweight)
        only, none = tile.linear_cross_entropy_backward(x, weight, target, lse, dloss,
                                                        need_dweight=False)
        assert none is None and torch.equal(only, dx)
        none, only = tile.linear_cross_entropy_backward(x, weight, target, lse, dloss,
                                                        need_dx=False)
        assert none is None and torch.equal(only, dweight)


@pytest.mark.parametrize("kind", list(TYPES))
def test_ignored_rows_cost_nothing_even_with_nan(kind):
    """Rows that are ignored, or whose dloss is 0, may hold anything: the
    gradients are those of the other rows alone."""
    x, weight, target, dloss = make(200, 96, 700, kind, 0.4)
    target[7] = -100
    dloss[[3, 50]] = 0.0
    lse = tile.linear_cross_entropy(x, weight, target)[1]
    out = (target == -100) | (dloss == 0)
    x[out] = float("nan")
    x[7] = float("inf")
    lse[out] = float("nan")
    dloss[target == -100] = float("nan")
    dx, dweight = tile.linear_cross_entropy_backward(x, weight, target, lse, dloss)
    assert not dx[out].any()
    keep = ~out
    check_gradients(x[keep], weight, target[keep], lse[keep], dloss[keep], dx[keep], dweight)
    loss, lse2 = tile.linear_cross_entropy(x, weight, target)
    assert not loss[target == -100].any()
    fine = keep & (target != -100)
    check_loss(x[fine], weight, target[fine], loss[fine], lse2[fine])


def test_everything_ignored_and_no_rows():
    x, weight, target, dloss = make(40, 72, 300, "bf16")
    target[:] = -100
    loss, lse = tile.linear_cross_entropy(x, weight, target)
    assert not loss.any() and not lse.any()
    dx, dweight = tile.linear_cross_entropy_backward(x, weight, target, lse, dloss)
    assert not dx.any() and not dweight.any()
    loss, lse = tile.linear_cross_entropy(x[:0], weight, target[:0])
    assert loss.numel() == lse.numel() == 0
    dx, dweight = tile.linear_cross_entropy_backward(x[:0], weight, target[:0], lse, dloss[:0])
    assert dx.numel() == 0 and not dweight.any()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,width,vocab", [(3, 2048, 1000), (200, 2048, 5000), (300, 1001, 777)])
def test_tokens_the_head_is_sure_of(rows, width, vocab, kind):
    """Losses from 1e-2 down to 1e-5 keep their digits, and the target's
    gradient, which is as small.  Both logits of a difference l_v - l_target
    are off by at most e = sum_error L (the target's, an FP32 sum of width / 32
    terms in each lane, by less), so a loss of log1p(d) is off by
    d (2 e + 2^-17).  e^(l - lse) - 1 takes the target's error, and that of an
    lse rounded to 24 bits, but the tensor cores' error of 1e-5 and more of
    the logit itself reaches neither."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    t = TYPES[kind]
    weight = (torch.randn(vocab, width, device="cuda", generator=gen) / width ** 0.5).to(t)
    target = torch.randint(vocab, (rows,), device="cuda", generator=gen)
    scale = torch.linspace(12, 18, rows, device="cuda")[:, None]
    x = (weight[target].float() * scale).to(t)
    loss, lse = tile.linear_cross_entropy(x, weight, target)
    l = x.double() @ weight.double().t()
    mag = (x.double().abs() @ weight.double().abs().t()).amax(1)
    at = l.gather(1, target[:, None])
    others = torch.exp(l - at)
    others.scatter_(1, target[:, None], 0.0)
    want = torch.log1p(others.sum(1))
    assert (loss >= 0).all() and want.max() < 0.2 and want.min() < 1e-3
    e = (width / 32 + 6) * 2.0 ** -23 * mag   # FP32 sums of a lane, and over lanes
    e_tc = sum_error(width) * mag
    rel = (e + e_tc).clamp(max=0.5)
    assert ((loss.double() - want).abs() <= want * (1.1 * rel + 2.0 ** -17)).all()
    # one row's dx: g_t w_t + sum of the others, with p from the lse handed over
    dx, _ = tile.linear_cross_entropy_backward(x, weight, target, lse, torch.ones(rows, device="cuda"),
                                               need_dweight=False)
    p = torch.exp(l - lse.double()[:, None])
    g = p.clone()
    miss = torch.expm1(at[:, 0] - lse.double())
    g.scatter_(1, target[:, None], miss[:, None])
    ref = g @ weight.double()
    half = torch.finfo(t).eps / 2
    gerr = half * g.abs() + p * (rel + 2.0 ** -20 * lse.double().abs())[:, None]
    gerr.scatter_(1, target[:, None], (half * miss.abs() + e + 2.0 ** -23 * lse.double())[:, None])
    if t == torch.float16:
        gerr += 2.0 ** -39
    tol = half * ref.abs() + 1.01 * gerr @ weight.double().abs() + \
        sum_error(vocab) * (g.abs() @ weight.double().abs()) + 2.0 ** -24
    assert ((dx.double() - ref).abs() <= tol).all()
    # the same, in the 2-norm, where the roundings of g and of dx are
    # independent: no worse than 4 roundings and the target's own error
    off = (dx.double() - ref).norm(dim=1)
    own = (e + 2.0 ** -23 * lse.double()) * weight[target].double().norm(dim=1)
    assert (off <= 4 * half * ref.norm(dim=1) + own + 1e-6).all()
    assert tile.tile_check_device_status() == 0


def test_another_ignore_index():
    x, weight, target, dloss = make(50, 64, 300, "f16")
    target[::3] = 0
    loss, lse = tile.linear_cross_entropy(x, weight, target, ignore_index=0)
    assert not loss[::3].any()
    t = torch.where(target == 0, -100, target)
    check_loss(x, weight, t, loss, lse)
    dx, dweight = tile.linear_cross_entropy_backward(x, weight, target, lse, dloss, ignore_index=0)
    check_gradients(x, weight, t, lse, dloss, dx, dweight)


def test_target_out_of_range_is_reported():
    x, weight, target, dloss = make(20, 64, 300, "bf16")
    target[4], target[9] = 300, -1
    loss, lse = tile.linear_cross_entropy(x, weight, target)
    assert loss[[4, 9]].isnan().all() and loss.isnan().sum() == 2
    assert tile.tile_check_device_status() == -9
    assert tile.tile_check_device_status() == 0
    dx, dweight = tile.linear_cross_entropy_backward(x, weight, target, lse, dloss)
    assert tile.tile_check_device_status() == -9
    t = target.clone()
    t[[4, 9]] = -100
    check_gradients(x, weight, t, lse, dloss, dx, dweight)


def test_large_logits_and_infinities():
    """Logits far apart (the sum is the largest one's), a vocabulary entry
    masked out with -inf through its row, a row that overflows."""
    x, weight, target, _ = make(64, 64, 600, "bf16")
    x *= 30
    loss, lse = tile.linear_cross_entropy(x, weight, target)
    check_loss(x, weight, target, loss, lse)
    x = x.abs() + 1
    weight[100:400] = 0.0
    weight[100:400, 5] = float("-inf")      # whole tiles and a part of one
    target.clamp_(max=99)
    loss, lse = tile.linear_cross_entropy(x, weight, target)
    keep = torch.cat([torch.arange(100), torch.arange(400, 600)]).cuda()
    check_loss(x, weight[keep], target, loss, lse)
    x[3] = float("inf")
    loss2, _ = tile.linear_cross_entropy(x, weight.abs(), target)
    assert not loss2[3].isfinite()


def test_gradients_against_differences():
    """Along a random direction of x and of weight, in FP64 differences."""
    x, weight, target, dloss = make(30, 40, 90, "f16", 0.2)
    loss, lse = tile.linear_cross_entropy(x, weight, target)
    dx, dweight = tile.linear_cross_entropy_backward(x, weight, target, lse, dloss * 1000)

    def value(dxs, dws):
        z = (x.double() + dxs) @ (weight.double() + dws).t()
        at = z.gather(1, target.clamp(min=0)[:, None])[:, 0]
        each = torch.where(target == -100, 0.0, torch.logsumexp(z, 1) - at)
        return (each * dloss.double() * 1000).sum()

    gen = torch.Generator(device="cuda").manual_seed(9)
    for t, grad, which in ((x, dx, 0), (weight, dweight, 1)):
        d = torch.randn(t.shape, device="cuda", generator=gen, dtype=torch.float64)
        e = 1e-5
        a, b = ((e * d, 0.0), (-e * d, 0.0)) if which == 0 else ((0.0, e * d), (0.0, -e * d))
        slope = (value(*a) - value(*b)) / (2 * e)
        want = (grad.double() * d).sum()
        # two FP16 roundings of each term
        assert (slope - want).abs() <= 2.0 ** -10 * (grad.double() * d).abs().sum()


@pytest.mark.parametrize("kind", list(TYPES))
def test_small_and_large_row_gradients(kind):
    """dloss over ten orders of magnitude, down to 2^-60."""
    x, weight, target, _ = make(96, 64, 500, kind)
    dloss = 2.0 ** -torch.arange(96, device="cuda").float().mul(60 / 95).floor()
    _, lse = tile.linear_cross_entropy(x, weight, target)
    dx, dweight = tile.linear_cross_entropy_backward(x, weight, target, lse, dloss)
    check_gradients(x, weight, target, lse, dloss, dx, dweight)


def test_repeats_streams_and_graph():
    x, weight, target, dloss = make(300, 200, 5000, "bf16", 0.2)

    def both():
        loss, lse = tile.linear_cross_entropy(x, weight, target)
        return (loss, lse) + tile.linear_cross_entropy_backward(x, weight, target, lse, dloss)
    first = both()
    for a, b in zip(first, both()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = tile.linear_cross_entropy(x, weight, target, stream=side)
    side.synchronize()
    assert torch.equal(other[0], first[0]) and torch.equal(other[1], first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = both()
    for k in range(2):
        x.mul_(0.5)
        target.copy_(torch.roll(target, 1))
        graph.replay()
        for a, b in zip(captured, both()):
            assert torch.equal(a, b)


def test_two_calls_at_once():
    """Calls on two streams with no synchronisation between them, each with a
    workspace of its own, forward and backward, small beside large."""
    calls = [make(700, 256, 9000, "bf16", 0.2, seed=5), make(9, 136, 3000, "f16", seed=6)]

    def both(x, weight, target, dloss, stream=None):
        loss, lse = tile.linear_cross_entropy(x, weight, target, stream=stream)
        return (loss, lse) + tile.linear_cross_entropy_backward(x, weight, target, lse, dloss,
                                                                stream=stream)
    alone = [both(*c) for c in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [both(*c, stream=s) for c, s in zip(calls, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_rows_behind_are_left_as_they_were():
    """The outputs' neighbours in memory are not written."""
    x, weight, target, dloss = make(37, 72, 300, "bf16")
    big = torch.full((40, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    wbig = torch.full((310, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    losses = torch.full((2, 64), 7.0, device="cuda")
    need = tile.tile_linear_cross_entropy_backward_workspace_bytes(37, 72, 300)
    ws = torch.full((need + 4096,), 3, dtype=torch.uint8, device="cuda")
    tile.tile_linear_cross_entropy(x, weight, target, losses[0, :37], losses[1, :37], ws[:need])
    tile.tile_linear_cross_entropy_backward(x, weight, target, losses[1, :37], dloss, big[:37],
                                            wbig[:300], ws[:need])
    assert (big[37:] == 7).all() and (wbig[300:] == 7).all()
    assert (losses[:, 37:] == 7).all() and (ws[need:] == 3).all()
    check_gradients(x, weight, target, losses[1, :37], dloss, big[:37], wbig[:300])


@pytest.mark.parametrize("rows,width,vocab", [(6, 4096, 530000), (6, 4095, 530000),
                                              (600000, 4096, 140), (530000, 64, 4100)])
def test_past_two_to_the_31_elements(rows, width, vocab):
    """A weight, a copy of it, an x and a piece's gradients of more than 2^31
    elements: the loss of every row, dx of the last rows and dweight of the
    last entries (and of some targets) against FP64, in blocks."""
    assert max(rows, vocab) * width > 1 << 31 or rows * 4096 > 1 << 31
    gen = torch.Generator(device="cuda").manual_seed(8)
    weight = torch.empty(vocab, width, dtype=torch.bfloat16, device="cuda")
    weight.normal_(0.0, 1.5 / width ** 0.5, generator=gen)
    target = torch.randint(vocab, (rows,), device="cuda", generator=gen)
    target[-2:] = vocab - 1
    x = torch.empty(rows, width, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=gen)
    dloss = torch.rand(rows, device="cuda", generator=gen) + 0.5
    loss, lse = tile.linear_cross_entropy(x, weight, target)
    dx, dweight = tile.linear_cross_entropy_backward(x, weight, target, lse, dloss)
    last = torch.arange(max(0, rows - 40), rows, device="cuda")
    cols = torch.cat([torch.arange(max(0, vocab - 40), vocab, device="cuda"), target[:5]]).unique()
    dw = torch.zeros(len(cols), width, dtype=torch.float64, device="cuda")
    dw_sq = torch.zeros_like(dw)
    for r0 in range(0, rows, 30000):
        r1 = min(rows, r0 + 30000)
        xr, t = x[r0:r1].double(), target[r0:r1]
        parts, top = [], []
        for v0 in range(0, vocab, 60000):
            l = xr @ weight[v0:v0 + 60000].double().t()
            parts.append(torch.logsumexp(l, 1))
            top.append(l.abs().amax(1))
        want_lse = torch.logsumexp(torch.stack(parts), 0)
        at = (xr * weight[t].double()).sum(1)
        # |x w| sums below 1.5 sqrt(width) 8, in place of each logit's own
        tol = sum_error(width) * 1.5 * 8 * width ** 0.5 + 2.0 ** -17
        assert ((lse[r0:r1] - want_lse).abs() <= tol + 2.0 ** -23 * want_lse.abs()).all()
        assert ((loss[r0:r1] - (want_lse - at)).abs() <= 2 * tol + 2.0 ** -22 * want_lse.abs()).all()
        g = torch.exp(xr @ weight[cols].double().t() - lse[r0:r1, None].double())
        g -= (t[:, None] == cols).double()
        g *= dloss[r0:r1, None].double()
        dw += g.t() @ xr
        dw_sq += g.square().t() @ xr.square()
    half = 2.0 ** -8
    # each of the n terms is rounded to half a step on its own: their errors
    # add like the root of their squares (within 8 times that), on top of
    # sum_error of the whole and the output's own rounding
    tol = half * dw.abs() + 8 * half * dw_sq.sqrt() + sum_error(rows) * dw_sq.sqrt() * rows ** 0.5
    assert ((dweight[cols].double() - dw).abs() <= tol).all()
    want = torch.zeros(len(last), width, dtype=torch.float64, device="cuda")
    want_sq = torch.zeros_like(want)
    for v0 in range(0, vocab, 60000):
        w = weight[v0:v0 + 60000].double()
        g = torch.exp(x[last].double() @ w.t() - lse[last, None].double())
        g -= (target[last, None] == torch.arange(v0, v0 + len(w), device="cuda")).double()
        g *= dloss[last, None].double()
        want += g @ w
        want_sq += g.square() @ w.square()
    tol = half * want.abs() + 8 * half * want_sq.sqrt() + \
        sum_error(vocab) * want_sq.sqrt() * vocab ** 0.5
    assert ((dx[last].double() - want).abs() <= tol).all()
    assert tile.tile_check_device_status() == 0


def test_end_of_a_training_step():
    """Block norm, loss and both backward passes as a training step runs
    them: the last block's hidden rows are scored, and the gradients reach
    the block's output, the residual stream and every parameter.  Against
    FP64 autograd of the same chain, in the 2-norm."""
    rows, width, vocab = 260, 192, 1500
    gen = torch.Generator(device="cuda").manual_seed(11)
    b, r = (torch.randn(rows, width, device="cuda", generator=gen).bfloat16() for _ in range(2))
    gp, gn = (1 + 0.2 * torch.randn(width, device="cuda", generator=gen) for _ in range(2))
    gate = 0.5 + 0.2 * torch.randn(2, width, device="cuda", generator=gen)
    weight = (torch.randn(vocab, width, device="cuda", generator=gen) / width ** 0.5).bfloat16()
    target = torch.randint(vocab, (rows,), device="cuda", generator=gen)
    target[::7] = -100
    hidden, y = tile.block_norm(b, r, gp, gate, gn, rows_per_gate=130)
    loss, lse = tile.linear_cross_entropy(y, weight, target)
    n = (target != -100).sum()
    dloss = (target != -100).float() / n
    dy, dweight = tile.linear_cross_entropy_backward(y, weight, target, lse, dloss)
    got = tile.block_norm_backward(b, hidden, gp, gate, gn, None, dy, rows_per_gate=130)

    leaves = [t.double().requires_grad_() for t in (b, r, gp, gate, gn, weight)]
    B, R, GP, GATE, GN, W = leaves
    h = R + GATE.repeat_interleave(130, 0) * B / (B.square().mean(1, keepdim=True) + 1e-5).sqrt() * GP
    z = (h / (h.square().mean(1, keepdim=True) + 1e-5).sqrt() * GN) @ W.t()
    each = torch.logsumexp(z, 1) - z.gather(1, target.clamp(min=0)[:, None])[:, 0]
    total = each[target != -100].sum() / n
    total.backward()
    # y, hidden, dy and the outputs are rounded to bf16 (2^-8 each at most)
    assert (loss.sum() / n - total).abs() <= 2.0 ** -8 * total
    for name, g, leaf in zip(("din", "dresidual", "dgamma_post", "dgate", "dgamma_pre"), got, leaves):
        assert (g.double() - leaf.grad).norm() <= 4 * 2.0 ** -8 * leaf.grad.norm(), name
    assert (dweight.double() - W.grad).norm() <= 4 * 2.0 ** -8 * W.grad.norm()
