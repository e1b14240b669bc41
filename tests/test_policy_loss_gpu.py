"""The clipped policy loss and its gradient against FP64.

Bounds.  x = old_nll - nll and q = nll - ref_nll are off by 2^-24 of themselves, expf
and expm1f by 2 ulp (2^-22), each product and sum by 2^-24.  So r is off by (2^-22
+ |x| 2^-24) r, r A by 2^-24 more, and e^q - 1 - q by 2^-22 |e^q - 1| + |q (e^q - 1)|
2^-24 + 2^-24 of itself; a held-back r A by 2^-23 (its bound and the product).  A
weight is rounded once or twice, and the gradient has three more products.  A mean
adds at most 511 FP32 roundings of partial sums of a tile's magnitudes.
"""

import math

import pytest
import torch

import tile_compiler_row_gb300 as tile

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
IGNORE = -100


@pytest.fixture(scope="module", autouse=True)
def device():
    from tile_compiler_row_gb300 import _build
    _build.build()
    tile.load()
    torch.cuda.set_device(0)


def inputs(rows, sequences=None, per_sequence=False, ref=True, ignored=0.0, seed=1, margin=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(n):
        return torch.randn(n, device="cuda", generator=g)
    nll = normal(rows).abs()
    kw = {"old_nll": nll + 0.25 * normal(rows), "advantage": normal(sequences if per_sequence else rows),
          "ref_nll": nll + 0.5 * normal(rows) if ref else None, "target": None, "offsets": None,
          "per_sequence": per_sequence, "kl_coef": 0.1 if ref else 0.0, "clip_low": 0.2, "clip_high": 0.3}
    if sequences is not None:
        cuts = torch.randint(margin, rows - margin + 1, (sequences + 1,), device="cuda", generator=g).sort().values
        if margin == 0:
            cuts[0], cuts[-1] = 0, rows
        kw["offsets"] = cuts
    if ignored:
        kw["target"] = torch.randint(100, (rows,), device="cuda", generator=g)
        kw["target"][torch.rand(rows, device="cuda", generator=g) < ignored] = IGNORE
    return nll, kw


def reference(nll, kw, mean, dloss=1.0):
    """(stats, weights, dnll) and bounds of stats and dnll, in FP64."""
    rows = nll.shape[0]
    f = lambda t: t.double()
    offsets = kw["offsets"]
    if offsets is None:
        offsets = torch.tensor([0, rows], device="cuda")
    count = offsets.shape[0] - 1
    of = torch.full((rows,), -1, device="cuda", dtype=torch.int64)
    for s, (b, e) in enumerate(zip(offsets[:-1].tolist(), offsets[1:].tolist())):
        of[b:e] = s
    keep = of >= 0
    if kw["target"] is not None:
        keep &= kw["target"] != IGNORE
    adv = f(kw["advantage"])
    if kw["per_sequence"]:
        adv = adv[of.clamp(min=0)]
    x = f(kw["old_nll"]) - f(nll)
    r = torch.exp(x)
    lo, hi = 1 - f(torch.tensor(kw["clip_low"])).item(), 1 + f(torch.tensor(kw["clip_high"])).item()
    held = r.clamp(lo, hi) * adv < r * adv
    ra = torch.where(held, r.clamp(lo, hi) * adv, r * adv)
    ra_off = ra.abs() * torch.where(held, 2 * U, 5 * U + x.abs() * U)
    q = f(nll) - f(kw["ref_nll"]) if kw["ref_nll"] is not None else torch.zeros_like(x)
    e = torch.expm1(q)
    kl = e - q
    kl_off = 4 * U * e.abs() + U * (q * e).abs() + U * kl.abs()
    beta = f(torch.tensor(kw["kl_coef"])).item()
    n = torch.bincount(of[keep], minlength=count).double()
    if mean == "token":
        weights = torch.full_like(n, 1 / max(1.0, n.sum().item()) if n.sum() > 0 else 0.0)
    else:
        weights = torch.where(n > 0, 1 / n.clamp(min=1) / max(1, int((n > 0).sum())), 0.0)
    w = torch.where(keep, weights[of.clamp(min=0)], 0.0)
    means, off = [], []
    for t, t_off in ((-ra, ra_off), (kl, kl_off), (held.double(), 0 * kl)):
        t = torch.where(keep, t, 0.0)
        means.append((w * t).sum())
        off.append((w * torch.where(keep, t_off, 0.0)).sum() + 512 * U * (w * t.abs()).sum() + U * means[-1].abs())
    stats = torch.stack([means[0] + beta * means[1], *means])
    off = torch.stack([off[0] + beta * off[1] + U * stats[0].abs(), *off])
    d = torch.where(held, 0.0, ra) + beta * e
    d_off = torch.where(held, 0.0, ra_off) + beta * (5 * U * e.abs() + U * (q * e + q).abs()) + U * d.abs()
    up = w * dloss
    dnll = torch.where(keep, d * up, 0.0)
    d_off = torch.where(keep, (d_off + 5 * U * d.abs()) * up.abs(), 0.0)
    return stats, weights, dnll, off * (1 + 2.0 ** -10), d_off * (1 + 2.0 ** -10) + 1e-44


def check(nll, kw, mean="token", dloss=None):
    stats, weights = tile.policy_loss(nll, mean=mean, **kw)
    up = 1.0 if dloss is None else float(dloss)
    want, want_weights, dnll, off, d_off = reference(nll, kw, mean, up)
    assert ((weights.double() - want_weights).abs() <= 3 * U * want_weights).all()
    assert ((stats.double() - want).abs() <= off).all(), (stats, want, off)
    got = tile.policy_loss_backward(nll, weights=weights, dloss=dloss, **kw)
    assert ((got.double() - dnll).abs() <= d_off).all(), float(((got.double() - dnll).abs() - d_off).max())
    assert (got[dnll == 0] == 0).all()
    assert tile.tile_check_device_status() == 0
    again, w2 = tile.policy_loss(nll, mean=mean, **kw)
    assert torch.equal(stats, again) and torch.equal(weights, w2)


@pytest.mark.parametrize("mean", ["token", "sequence"])
@pytest.mark.parametrize("ref", [True, False])
@pytest.mark.parametrize("rows", [1, 2, 31, 255, 1023, 1024, 1025, 5000, 8191, 8192, 8193, 30001])
def test_one_sequence(rows, ref, mean):
    check(*inputs(rows, ref=ref), mean=mean)
    check(*inputs(rows, ref=ref, ignored=0.4, seed=2), mean=mean,
          dloss=torch.tensor([0.37], device="cuda"))


@pytest.mark.parametrize("mean", ["token", "sequence"])
@pytest.mark.parametrize("per_sequence", [True, False])
@pytest.mark.parametrize("rows,sequences", [(1, 1), (5, 9), (700, 3), (1024, 64), (1025, 65),
                                            (2000, 1999), (3000, 5000), (9000, 2), (9001, 700),
                                            (70000, 12), (50000, 3000), (4000, 1), (300000, 3)])
def test_sequences(rows, sequences, per_sequence, mean):
    check(*inputs(rows, sequences, per_sequence, ignored=0.3), mean=mean)
    margin = rows // 7     # rows in front of the first sequence and behind the last
    check(*inputs(rows, sequences, per_sequence, ref=False, margin=margin, seed=3), mean=mean)


@pytest.mark.parametrize("mean", ["token", "sequence"])
@pytest.mark.parametrize("rows", [300, 20000])
def test_rows_that_do_not_count_are_not_used(rows, mean):
    nll, kw = inputs(rows, 6, True, ignored=0.5, margin=20)
    out = torch.ones(rows, dtype=torch.bool, device="cuda")
    out[int(kw["offsets"][0]):int(kw["offsets"][-1])] = False
    out |= kw["target"] == IGNORE
    for k, bad in ((0, float("nan")), (1, float("inf")), (2, -float("inf"))):
        with_bad = dict(kw)
        n = nll.clone()
        n[out] = bad
        for name in ("old_nll", "ref_nll"):
            with_bad[name] = kw[name].clone()
            with_bad[name][out] = bad
        a, wa = tile.policy_loss(nll, mean=mean, **kw)
        b, wb = tile.policy_loss(n, mean=mean, **with_bad)
        assert torch.equal(a, b) and torch.equal(wa, wb)
        assert torch.equal(tile.policy_loss_backward(nll, weights=wa, **kw),
                           tile.policy_loss_backward(n, weights=wa, **with_bad))


@pytest.mark.parametrize("mean", ["token", "sequence"])
@pytest.mark.parametrize("rows", [50, 9000])
def test_nothing_counts(rows, mean):
    nll, kw = inputs(rows, 5, True)
    kw["target"] = torch.full((rows,), IGNORE, device="cuda")
    stats, weights = tile.policy_loss(nll, mean=mean, **kw)
    assert (stats == 0).all() and (weights == 0).all()
    assert (tile.policy_loss_backward(nll, weights=weights, **kw) == 0).all()
    kw["target"], kw["offsets"] = None, torch.full((6,), rows // 2, device="cuda")
    stats, weights = tile.policy_loss(nll, mean=mean, **kw)
    assert (stats == 0).all() and (weights == 0).all()
    kw["offsets"] = torch.zeros(6, device="cuda", dtype=torch.int64)
    empty = torch.empty(0, device="cuda")
    kw.update(old_nll=empty, ref_nll=empty, target=None)
    stats, weights = tile.policy_loss(empty, mean=mean, **kw)
    assert (stats == 0).all() and (weights == 0).all()
    assert tile.policy_loss_backward(empty, weights=weights, **kw).numel() == 0


def test_at_the_border():
    """Ratios next to the bounds, decided as FP64 decides the unrounded
    differences; old and nll of sizes that make the difference round."""
    high, low = 0.3, 0.2
    up = math.log1p(float(torch.tensor(high)))
    down = math.log1p(-float(torch.tensor(low)))
    nll, old = [], []
    for bound in (up, down):
        for base in (0.0, 1e-3, 0.7, 5.0, 1000.0):
            o = torch.tensor(base + bound)
            for k in range(-3, 4):
                near = o.clone()
                for _ in range(abs(k)):
                    near = torch.nextafter(near, torch.tensor(math.copysign(1e9, k)))
                nll.append(torch.tensor(base)), old.append(near)
    nll, old = torch.stack(nll).cuda(), torch.stack(old).cuda()
    x = old.double() - nll.double()
    for a in (1.0, -1.0):
        adv = torch.full_like(nll, a)
        held = (x > up) if a > 0 else (x < down)
        kw = dict(old_nll=old, advantage=adv, clip_low=low, clip_high=high)
        stats, weights = tile.policy_loss(nll, **kw)
        assert abs(float(stats[3]) - held.double().mean().item()) <= U
        d = tile.policy_loss_backward(nll, weights=weights, **kw)
        assert torch.equal(d == 0, held)
        assert held.any() and not held.all()


def test_extreme_ratios():
    """Ratios of 0 and infinity, advantages of 0, and bounds of no clip."""
    nll = torch.tensor([0.0, 300.0, 0.0, 300.0, 0.0, 300.0], device="cuda")
    old = torch.tensor([300.0, 0.0, 300.0, 0.0, 300.0, 0.0], device="cuda")
    adv = torch.tensor([1.0, 1.0, -1.0, -1.0, 0.0, 0.0], device="cuda")
    for mask, loss, share in ((0, -1.5, 1), (1, 0.0, 0), (2, float("inf"), 0), (3, 0.5, 1), (4, 0, 0), (5, 0, 0)):
        target = torch.full((6,), IGNORE, device="cuda")
        target[mask] = 1
        kw = dict(old_nll=old, advantage=adv, target=target, clip_low=0.5, clip_high=0.5)
        stats, weights = tile.policy_loss(nll, **kw)
        assert float(stats[0]) == loss and float(stats[3]) == share
        d = tile.policy_loss_backward(nll, weights=weights, **kw)
        assert float(d[mask]) == (-float("inf") if mask == 2 else 0.0)
    kw = dict(old_nll=old, advantage=adv, clip_low=1.0, clip_high=float("inf"))
    stats, _ = tile.policy_loss(nll[1:2], **{k: v[1:2] if torch.is_tensor(v) else v for k, v in kw.items()})
    assert stats.tolist() == [0.0, 0.0, 0.0, 0.0]
    stats, _ = tile.policy_loss(nll[:1], **{k: v[:1] if torch.is_tensor(v) else v for k, v in kw.items()})
    assert stats[1] == -float("inf") and stats[3] == 0


def test_offsets_that_fall_are_noted():
    nll, kw = inputs(5000, 4, True)
    for offsets in ([0, 100, 50, 200, 5000], [-1, 5, 6, 7, 8], [0, 1, 2, 3, 5001],
                    [0, 1 << 62, 3, 4, 5000], [-(1 << 63), 5, (1 << 63) - 1, 7, 9]):
        kw["offsets"] = torch.tensor(offsets, device="cuda")
        for mean in ("token", "sequence"):
            stats, _ = tile.policy_loss(nll, mean=mean, **kw)
            assert torch.isnan(stats).all()
            assert tile.tile_check_device_status() == -9 and tile.tile_check_device_status() == 0
            tile.policy_loss_backward(nll, weights=torch.zeros(4, device="cuda"), **kw)
            assert tile.tile_check_device_status() == 0


def test_gradient_against_differences():
    """Central differences of the FP64 loss at the FP32 inputs, a step h of 1e-5
    (error h^2 / 6 times a third derivative of at most 2 r |A| + beta e^q, and
    2^-50 / h of the loss's terms), away from the borders."""
    nll, kw = inputs(40, 5, True, ignored=0.2)
    x = kw["old_nll"].double() - nll.double()
    for b in (math.log(1.3), math.log(0.8)):
        assert ((x - b).abs() > 1e-4).all()
    stats, weights = tile.policy_loss(nll, mean="sequence", **kw)
    got = tile.policy_loss_backward(nll, weights=weights, **kw)
    h = 1e-5

    def loss(v):
        return reference(v, kw, "sequence")[0][0].item()
    off = reference(nll, kw, "sequence")[4]
    for i in range(0, 40, 3):
        v = nll.double().clone()
        v[i] += h
        w = nll.double().clone()
        w[i] -= h
        diff = (loss(v) - loss(w)) / (2 * h)
        assert abs(diff - float(got[i])) <= float(off[i]) + 3e-9


def test_workspace_streams_and_graphs():
    nll, kw = inputs(20000, 300, True, ignored=0.3)
    n = tile.tile_policy_loss_workspace_bytes(20000, 300)
    room = torch.full((n + 512,), 0xAB, dtype=torch.uint8, device="cuda")
    stats, weights = torch.empty(4, device="cuda"), torch.empty(300, device="cuda")
    names = {k: v for k, v in kw.items() if k not in ("per_sequence", "old_nll", "advantage")}
    tile.tile_policy_loss(nll, kw["old_nll"], kw["advantage"], stats, weights, room[256:256 + n],
                          sequence_advantage=True, sequence_mean=True, **names)
    want, want_weights = tile.policy_loss(nll, mean="sequence", **kw)
    assert torch.equal(stats, want) and torch.equal(weights, want_weights)
    assert (room[:256] == 0xAB).all() and (room[256 + n:] == 0xAB).all()
    small, small_kw = inputs(3000, 20, True)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [(tile.policy_loss(nll, mean="sequence", stream=s, **kw),
            tile.policy_loss(small, mean="sequence", stream=s.cuda_stream, **small_kw)) for s in streams * 2]
    torch.cuda.synchronize()
    small_want = tile.policy_loss(small, mean="sequence", **small_kw)
    for big, little in got:
        assert torch.equal(big[0], want) and torch.equal(little[0], small_want[0])
    for data, k in ((nll, kw), (small, small_kw)):
        held = data.clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s, w = tile.policy_loss(held, mean="sequence", **k)
            d = tile.policy_loss_backward(held, weights=w, **k)
        for shift in (0.0, 0.05):
            held.copy_(data + shift)
            graph.replay()
            torch.cuda.synchronize()
            s2, w2 = tile.policy_loss(held, mean="sequence", **k)
            assert torch.equal(s, s2) and torch.equal(w, w2)
            assert torch.equal(d, tile.policy_loss_backward(held, weights=w2, **k))


@pytest.mark.parametrize("mean", ["token", "sequence"])
@pytest.mark.parametrize("rows", [1, 300, 20000])
@pytest.mark.parametrize("size", [1e-6, 1e-4, 1e-3, 0.05, 0.3, 0.5, 0.7, 1.0, 3.0])
def test_kl_of_a_policy_near_its_reference(size, rows, mean):
    """The KL term against itself: e^q - q - 1 is about q^2 / 2 there, so nothing of the
    size of q's own ulp may be left in it.  In roundings of 2^-24 of the term: q is
    off by one of itself, which is q (e^q - 1) / kl of the term, 3.6 at most up to
    |q| = 3.  Then five of the term's own up to 1/2, or beyond it expm1f's ulp, up to
    2 |e^q - 1| / kl = 8.8, and one of the difference: 14 in all.  The terms are
    positive, so each of the sums over a tile (16 to a lane and 5 between lanes, or 2, 5
    and 8) adds one at most: 21; the sums beyond are compensated, 1; two quotients,
    and three of the weights that the reference takes: 41."""
    g = torch.Generator(device="cuda").manual_seed(7)

    def uniform(n):
        return torch.rand(n, device="cuda", generator=g)
    nll = 0.1 + uniform(rows)
    ref = nll - (2 * uniform(rows) - 1) * size
    offsets = torch.tensor([0, rows // 3, rows // 3, rows], device="cuda")
    stats, weights = tile.policy_loss(nll, nll.clone(), torch.ones_like(nll), ref_nll=ref, offsets=offsets,
                                      kl_coef=1.0, mean=mean)
    q = nll.double() - ref.double()
    q2 = q * q     # e^q - q - 1: the series up to 1/2 (the first term left out: 2^-60 of it), else expm1
    series = torch.zeros_like(q)
    for k in range(16, 1, -1):
        series = series * q + 1.0 / math.factorial(k)
    kl = torch.where(q.abs() <= 0.5, q2 * series, torch.expm1(q) - q)
    w = torch.repeat_interleave(weights.double(), offsets[1:] - offsets[:-1])
    want = (w * kl).sum().item()
    assert float(stats[2]) >= 0 and abs(float(stats[2]) - want) <= 41 * U * want, (float(stats[2]), want)


@pytest.mark.parametrize("mean", ["token", "sequence"])
@pytest.mark.parametrize("rows", [40, 9000])
def test_no_kl_term_whatever_the_reference_holds(rows, mean):
    """kl_coef 0 with a reference (its term is looked at, not trained on): loss and
    gradient are those without one, where e^q overflows or is NaN too."""
    nll, kw = inputs(rows, 6, ignored=0.3)
    kw["kl_coef"] = 0.0
    nll[::5] += 150.0
    kw["old_nll"] = kw["old_nll"] + torch.where(nll > 100.0, 150.0, 0.0)
    without = dict(kw, ref_nll=None)
    want, weights = tile.policy_loss(nll, mean=mean, **without)
    want_d = tile.policy_loss_backward(nll, weights=weights, **without)
    assert torch.isfinite(want).all() and torch.isfinite(want_d).all()
    for bad in (None, float("nan"), float("inf"), -float("inf")):
        if bad is not None:
            kw["ref_nll"] = torch.full_like(nll, bad)
        stats, w = tile.policy_loss(nll, mean=mean, **kw)
        assert torch.equal(w, weights)
        assert torch.equal(stats[[0, 1, 3]], want[[0, 1, 3]])
        assert not torch.isfinite(stats[2])
        assert torch.equal(tile.policy_loss_backward(nll, weights=w, **kw), want_d)
