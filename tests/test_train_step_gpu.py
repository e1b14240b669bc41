"""A whole training step from tokens to updated weights: the lookup, a block norm,
the linear cross entropy with the head's weight shared by the embedding, the policy
loss, every gradient, their norm and the AdamW step; eager and captured, against
FP64 autograd."""

import math

import pytest
import torch

import tile_compiler_row_gb300 as tile

pytestmark = pytest.mark.gpu

IGNORE = -100
ROWS, WIDTH, VOCAB, SEQUENCES = 200, 96, 300, 5


@pytest.fixture(scope="module", autouse=True)
def device():
    from tile_compiler_row_gb300 import _build
    _build.build()
    tile.load()
    torch.cuda.set_device(0)


def make(seed=1, rows=ROWS):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)
    token = torch.randint(VOCAB, (rows,), device="cuda", generator=g)
    token[::17] = IGNORE
    target = torch.randint(VOCAB, (rows,), device="cuda", generator=g)
    target[::7] = IGNORE
    cuts = torch.randint(rows, (SEQUENCES - 1,), device="cuda", generator=g).sort().values
    s = {"token": token, "target": target,
         "offsets": torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), rows - 3)]),
         "advantage": normal(SEQUENCES), "mixed": normal(rows, WIDTH).bfloat16(),
         "params": [normal(VOCAB, WIDTH) / WIDTH ** 0.5, 1 + 0.1 * normal(WIDTH), 1 + 0.1 * normal(WIDTH)]}
    s["weight"] = s["params"][0].bfloat16()
    s["old"] = 5.7 + 0.2 * normal(rows)
    s["ref"] = 5.7 + 0.3 * normal(rows)
    s["state"] = tile.adamw_state(s["params"])
    s["gammas"] = [torch.empty(WIDTH, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    return s


def step(s, count):
    """One step in place; its gradients and the loss."""
    w, (_, post, pre) = s["weight"], s["params"]
    policy = dict(ref_nll=s["ref"], target=s["target"], offsets=s["offsets"], per_sequence=True, kl_coef=0.05)
    x = tile.embedding(s["token"], w, scale=WIDTH ** 0.5)
    hidden, y = tile.block_norm(s["mixed"], x, post, None, pre)
    nll, lse = tile.linear_cross_entropy(y, w, s["target"])
    stats, weights = tile.policy_loss(nll, s["old"], s["advantage"], mean="sequence", **policy)
    dnll = tile.policy_loss_backward(nll, s["old"], s["advantage"], weights, **policy)
    dy, dw = tile.linear_cross_entropy_backward(y, w, s["target"], lse, dnll)
    dmixed, dx, dpost, _, dpre = tile.block_norm_backward(s["mixed"], hidden, post, None, pre, None, dy)
    tile.embedding_backward(s["token"], dx, scale=WIDTH ** 0.5, dweight=dw)
    grads = [dw, dpost, dpre]
    norm = tile.grad_norm(grads, 0.05)
    tile.adamw(s["params"], grads, **s["state"], step=count, lr=1e-2, factor=norm[1:],
               weight_decay=[0.1, 0.0, 0.0], copies=[w, *s["gammas"]])
    return stats, grads, norm


def reference(s):
    """(loss, gradients) by FP64 autograd."""
    leaves = [t.double().requires_grad_() for t in (s["weight"], *s["params"][1:])]
    w, post, pre = leaves
    keep = s["token"] != IGNORE
    x = torch.where(keep[:, None], w[s["token"].clamp(min=0)] * WIDTH ** 0.5, 0.0)
    m = s["mixed"].double()
    h = x + m / (m.square().mean(1, keepdim=True) + 1e-5).sqrt() * post
    z = h / (h.square().mean(1, keepdim=True) + 1e-5).sqrt() * pre @ w.t()
    valid = s["target"] != IGNORE
    nll = torch.logsumexp(z, 1) - z.gather(1, s["target"].clamp(min=0)[:, None])[:, 0]
    of = torch.full((len(nll),), -1, device="cuda", dtype=torch.int64)
    for k in range(SEQUENCES):
        of[int(s["offsets"][k]):int(s["offsets"][k + 1])] = k
    counts = valid & (of >= 0)
    r = torch.exp(s["old"].double() - nll)
    adv = s["advantage"].double()[of.clamp(min=0)]
    q = nll - s["ref"].double()
    term = -torch.minimum(r * adv, r.clamp(0.8, 1.2) * adv) + 0.05 * (torch.exp(q) - q - 1)
    means = [term[counts & (of == k)].mean() for k in range(SEQUENCES) if (counts & (of == k)).any()]
    loss = torch.stack(means).mean()
    loss.backward()
    return loss.detach(), [t.grad for t in leaves]


def test_step_against_autograd():
    """Rows pass through four tensors of BF16 (the lookup, the hidden rows, the
    block's result and its gradient), each off by 2^-9 rms or 2^-8 at most,
    and the weight's gradient through two more: six of 2^-8 in the 2-norm.  Ratios next to
    the clip's bounds may fall on the other side, so none may lie that near."""
    s = make()
    with torch.no_grad():
        want = {k: [t.clone() for t in v] if isinstance(v, list) else v for k, v in s.items() if k != "state"}
        want["weight"] = s["weight"].clone()
    stats, grads, norm = step(s, 1)
    loss, ref = reference(want)
    assert abs(stats[0].double() - loss) <= 6 * 2.0 ** -8 * loss.abs() + 6 * 2.0 ** -8
    total = torch.stack([g.square().sum() for g in ref]).sum().sqrt()
    assert abs(norm[0].double() - total) <= 6 * 2.0 ** -8 * total
    for g, r in zip(grads, ref):
        assert (g.double() - r).norm() <= 6 * 2.0 ** -8 * r.norm()
    assert torch.equal(s["weight"], s["params"][0].bfloat16())
    # a first step moves each element by lr, or next to none where its gradient is 0
    moved = (s["params"][1] - want["params"][1]).abs()
    assert (moved <= 1e-2 * (1 + 2.0 ** -10)).all() and (moved > 0.9e-2).float().mean() > 0.9


@pytest.mark.parametrize("rows", [ROWS, 3000])
def test_captured_step_equals_eager_steps(rows):
    """Two programs at once, each captured on its own, replayed in turn."""
    eager, captured, other = make(1, rows), make(1, rows), make(2, rows)
    counts = [torch.ones(1, dtype=torch.int64, device="cuda") for _ in range(3)]
    graphs = []
    for s, count in ((captured, counts[1]), (other, counts[2])):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(s, count)
            count.add_(1)
        graphs.append(graph)
    for _ in range(3):
        step(eager, counts[0])
        counts[0].add_(1)
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager["params"] + eager["gammas"], captured["params"] + captured["gammas"]):
        assert torch.equal(a, b)
    assert torch.equal(eager["weight"], captured["weight"])
    assert tile.tile_check_device_status() == 0


def log_probabilities(s):
    """nll of the step's rows in FP64."""
    w, post, pre = (t.double() for t in (s["weight"], *s["params"][1:]))
    x = torch.where((s["token"] != IGNORE)[:, None], w[s["token"].clamp(min=0)] * WIDTH ** 0.5, 0.0)
    m = s["mixed"].double()
    h = x + m / (m.square().mean(1, keepdim=True) + 1e-5).sqrt() * post
    z = h / (h.square().mean(1, keepdim=True) + 1e-5).sqrt() * pre @ w.t()
    return torch.logsumexp(z, 1) - z.gather(1, s["target"].clamp(min=0)[:, None])[:, 0]


def counted_rows(s):
    row = torch.arange(len(s["target"]), device="cuda")
    return (s["target"] != IGNORE) & (row >= s["offsets"][0]) & (row < s["offsets"][-1])


def held(s, nll):
    """The rows that the clip holds back."""
    of = (torch.searchsorted(s["offsets"], torch.arange(len(nll), device="cuda"), right=True) - 1).clamp(0, SEQUENCES - 1)
    r, adv = torch.exp(s["old"].double() - nll.double()), s["advantage"].double()[of]
    return counted_rows(s) & (r.clamp(0.8, 1.2) * adv < r * adv)


def own_log_probabilities(s):
    w, (_, post, pre) = s["weight"], s["params"]
    x = tile.embedding(s["token"], w, scale=WIDTH ** 0.5)
    _, y = tile.block_norm(s["mixed"], x, post, None, pre)
    return tile.linear_cross_entropy(y, w, s["target"])[0]


def test_no_ratio_of_the_step_crosses_a_bound():
    """What test_step_against_autograd rests on: its rows are held back by the clip
    in BF16 exactly where they are in FP64."""
    s = make()
    assert torch.equal(held(s, own_log_probabilities(s)), held(s, log_probabilities(s)))


@pytest.mark.parametrize("seed", [1, 2, 3, 4])
def test_step_of_ratios_away_from_the_bounds(seed):
    """The same step with old_nll placed around FP64's nll, no log ratio within 0.08
    of a bound's: BF16's errors of nll (asserted to be below) move no row over it."""
    s = make(seed)
    if (s["offsets"].diff() < 0).any():    # a cut behind the last row of all (seed 3): noted, not computed
        assert torch.isnan(step(s, 1)[0]).all()
        assert tile.tile_check_device_status() == -9 and tile.tile_check_device_status() == 0
        return
    exact = log_probabilities(s)
    x = 0.3 * torch.randn(ROWS, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed + 50)).double()
    for ratio in (0.8, 1.2):
        bound = math.log(ratio)
        near = (x - bound).abs() < 0.08
        x = torch.where(near, bound + torch.where(x < bound, -0.08, 0.08), x)
    s["old"] = (exact + x).float()
    nll = own_log_probabilities(s)
    assert (nll.double() - exact)[counted_rows(s)].abs().max() < 0.07
    rows_held = held(s, exact)
    assert torch.equal(held(s, nll), rows_held)
    assert 0 < rows_held.sum() < counted_rows(s).sum()
    want = {k: [t.clone() for t in v] if isinstance(v, list) else v for k, v in s.items() if k != "state"}
    want["weight"] = s["weight"].clone()
    stats, grads, norm = step(s, 1)
    loss, ref = reference(want)
    # (six roundings of 2^-8, as in test_step_against_autograd)
    assert abs(stats[0].double() - loss) <= 6 * 2.0 ** -8 * loss.abs() + 6 * 2.0 ** -8
    total = torch.stack([g.square().sum() for g in ref]).sum().sqrt()
    assert abs(norm[0].double() - total) <= 6 * 2.0 ** -8 * total
    for g, r in zip(grads, ref):
        assert (g.double() - r).norm() <= 6 * 2.0 ** -8 * r.norm()
