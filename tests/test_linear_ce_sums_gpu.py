"""How exact the linear cross entropy's sums are, beyond the worst case that a
sum of `width` products allows (test_linear_ce_gpu.py).

A logit is added up in parts of at most 4096 columns, which the tensor cores add
16 products at a time; parts are joined in FP32 with rounding, and 2^-26 of a
part is put back for each of its n <= 256 steps.  What a step may lose, by the
model that Fasi, Higham, Mikaitis and Pranesh measured on earlier tensor cores
(Numerical behavior of NVIDIA tensor cores, 2021): every product and the sum so
far is cut off 2 bits below the 24 of the largest of them, and the new sum at
its 24 bits, in all at most 16 2^-25 + 2^-23 = 5 2^-23 of it, toward 0.

* Sums that are exact lose nothing: what is put back is n 2^-26 of the logit.
* Rows of random signs: what the products lose is as often added as taken, and
  of the sums' own cuts, half a unit or 2^-25 to 2^-24 of a sum that grows to
  its end, 2^-26 to 2^-25 of the end, the least is put back: at most n 2^-26 is
  left of a logit.  Of lse less: it goes with the mean logit under p, half of
  it or less in these rows, and 4096 columns lost 3.9e-6 to 4.4e-6 for the
  3.8e-6 put back: 3e-7 is left of lse, 2^-21 with a margin.
* Products of one sign: a part that grows evenly is (n + 1) / 2n of its end on
  average, so it loses at most (n + 1) / 2 5 2^-23 of itself.

What comes to lse on top: log2(e) and its product with a logit, 3 roundings of
the largest logit, and one for each join of two parts; the exponentials and
their sums, below 64 roundings of 1 (2^-22 for each of 6 factors; chains of at
most 40 additions); the logarithm, 3 roundings of lse.

    2^-18 + (n 2^-26 + (4 + parts) 2^-24) max|l| + 2^-22 |lse|

holds the first two cases, and for a difference of two logits twice that."""

import pytest
import torch

import tile_compiler_row_gb300 as tile
from test_linear_ce_gpu import TYPES, check_gradients, check_loss, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    from tile_compiler_row_gb300 import _build
    _build.build()
    tile.load()
    torch.cuda.set_device(0)


def steps(width):
    return min(256, -(-width // 16))


def of_logit(width):
    return steps(width) * 2.0 ** -26 + (4 + width // 4096) * 2.0 ** -24


def check_exact(x, weight, target, more=0.0):
    """loss and lse within the bound above; `more`: what each row's sums may
    lose besides."""
    loss, lse = tile.linear_cross_entropy(x, weight, target)
    l = x.double() @ weight.double().t()
    want = torch.logsumexp(l, 1)
    tol = 2.0 ** -18 + of_logit(x.shape[1]) * l.abs().amax(1) + 2.0 ** -22 * want.abs() + more
    off = (lse.double() - want).abs()
    assert (off <= tol).all(), f"lse off by {(off / tol).max():.2f} of the tolerance"
    at = l.gather(1, target[:, None])[:, 0]
    off = (loss.double() - (want - at)).abs()
    assert (off <= 2 * tol).all(), f"loss off by {(off / tol).max() / 2:.2f} of the tolerance"
    assert tile.tile_check_device_status() == 0
    return l, lse


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,width,vocab", [(40, 64, 300), (300, 1000, 600), (40, 4096, 700),
                                              (40, 4097, 300), (20, 131072, 300)])
def test_one_product_to_a_logit(rows, width, vocab, kind):
    """Rows with a single column: a logit is one product, exact."""
    gen = torch.Generator(device="cuda").manual_seed(21)
    weight = torch.randn(vocab, width, device="cuda", generator=gen).to(TYPES[kind])
    x = torch.zeros(rows, width, dtype=TYPES[kind], device="cuda")
    at = torch.randint(width, (rows,), device="cuda", generator=gen)
    at[0], at[1] = 0, width - 1
    x[torch.arange(rows, device="cuda"), at] = 12.0
    target = torch.randint(vocab, (rows,), device="cuda", generator=gen)
    l, _ = check_exact(x, weight, target)
    assert l.abs().max() > 30


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("width", [2048, 8192, 65536])
def test_sums_of_small_integers(width, kind):
    """Every partial sum is a small multiple of 1/8: nothing is rounded."""
    gen = torch.Generator(device="cuda").manual_seed(22)
    x = torch.randint(-2, 3, (50, width), device="cuda", generator=gen).to(TYPES[kind])
    weight = torch.randint(-1, 2, (600, width), device="cuda", generator=gen).to(TYPES[kind]) / 8
    # rows that agree with an entry more often than by chance
    x[::2] = (x[::2].float() + (weight[:25].float() * 8) * (torch.rand(
        25, width, device="cuda", generator=gen) < 200 / width)).to(TYPES[kind])
    target = torch.randint(600, (50,), device="cuda", generator=gen)
    check_exact(x, weight, target)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("width", [1024, 4096, 16384])
def test_a_column_that_stands_out_at_the_end(width, kind):
    """Sums that stay below 1 until their last columns bring them to 40."""
    gen = torch.Generator(device="cuda").manual_seed(23)
    t = TYPES[kind]
    weight = torch.randn(600, width, device="cuda", generator=gen).to(t)
    x = (torch.randn(50, width, device="cuda", generator=gen) / width).to(t)
    x[:, -3] = 12.0
    target = torch.randint(600, (50,), device="cuda", generator=gen)
    # the steps before cut off sums of at most sum |x w|
    low = (x.double().abs()[:, :-3] @ weight.double().abs()[:, :-3].t()).amax(1)
    check_exact(x, weight, target, steps(width) * 5 * 2.0 ** -23 * low)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,width,vocab", [(300, 4096, 9000), (5, 2048, 9000), (600, 1024, 3000),
                                              (300, 4095, 3000), (200, 16384, 2000)])
def test_rows_of_a_trained_head(rows, width, vocab, kind):
    """Dense rows that lean towards their target (whose logit is a sum of its
    own), random beside the other entries."""
    gen = torch.Generator(device="cuda").manual_seed(24)
    t = TYPES[kind]
    weight = (torch.randn(vocab, width, device="cuda", generator=gen) * 1.5 / width ** 0.5).to(t)
    target = torch.randint(vocab, (rows,), device="cuda", generator=gen)
    x = (torch.randn(rows, width, device="cuda", generator=gen) +
         4 * torch.rand(rows, 1, device="cuda", generator=gen) * weight[target].float()).to(t)
    l, lse = check_exact(x, weight, target)
    want = torch.logsumexp(l, 1)
    off = lse.double() - want
    assert off.norm() <= 2.0 ** -20 * want.norm()
    assert off.mean().abs() <= 2.0 ** -21 * want.mean()
    loss, _ = tile.linear_cross_entropy(x, weight, target)
    each = want - l.gather(1, target[:, None])[:, 0]
    assert (loss.double() - each).norm() <= 2.0 ** -20 * want.norm()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("width,vocab", [(2048, 1000), (1537, 3001), (4096, 777), (1024, 32769),
                                         (512, 19456), (600, 9728), (8192, 777), (4097, 1000)])
def test_every_border_of_the_vocabulary_counts(width, vocab, kind):
    """One entry far above the others, at the borders of tiles of 192, 224 and
    256 entries, their halves and their pieces of 32, and at the end: lse is
    that entry's logit, which no sum without it comes near.  And so the
    gradients: the entry's g is dloss itself."""
    places = {0, 1, vocab - 1, vocab - 2, vocab // 256 * 256, vocab // 224 * 224, vocab // 192 * 192}
    for tile_width in (32, 96, 112, 128, 192, 224, 256):
        for i in (1, 2, 3, vocab // tile_width - 1, vocab // tile_width):
            places |= {i * tile_width - 1, i * tile_width}
    places = torch.tensor(sorted(p for p in places if 0 <= p < vocab), device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(25)
    t = TYPES[kind]
    weight = (torch.randn(vocab, width, device="cuda", generator=gen) / width ** 0.5).to(t)
    x = (30 * weight[places].float()).to(t)
    target = (places + vocab // 2) % vocab
    # products of one sign: squares
    own = 30 * weight[places].double().square().sum(1)
    l, lse = check_exact(x, weight, target, (steps(width) + 1) / 2 * 5 * 2.0 ** -23 * own)
    rows = torch.arange(len(places), device="cuda")
    assert (l[rows, places] > torch.logsumexp(l.scatter(1, places[:, None], -1e9), 1) + 2).all()
    dloss = torch.rand(len(places), device="cuda", generator=gen) + 0.5
    loss, lse = tile.linear_cross_entropy(x, weight, target)
    check_loss(x, weight, target, loss, lse)
    dx, dweight = tile.linear_cross_entropy_backward(x, weight, target, lse, dloss)
    check_gradients(x, weight, target, lse, dloss, dx, dweight)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,width,vocab", [(300, 4104, 1000), (70, 8191, 3001), (257, 12288, 511),
                                              (1, 4097, 5), (33, 20000, 700)])
def test_sums_of_several_parts(rows, width, vocab, kind):
    """Loss and gradients of rows a little and much wider than a part, every
    element, with ignored rows."""
    x, weight, target, dloss = make(rows, width, vocab, kind, 0.3 if rows > 2 else 0.0)
    loss, lse = tile.linear_cross_entropy(x, weight, target)
    check_loss(x, weight, target, loss, lse)
    dx, dweight = tile.linear_cross_entropy_backward(x, weight, target, lse, dloss)
    check_gradients(x, weight, target, lse, dloss, dx, dweight)
    again = tile.linear_cross_entropy(x, weight, target)
    assert torch.equal(loss, again[0]) and torch.equal(lse, again[1])
    assert tile.tile_check_device_status() == 0


@pytest.mark.parametrize("kind", list(TYPES))
def test_a_single_entry_of_several_parts(kind):
    """Nothing to choose from: the loss is 0, and what the gradient holds is
    the roundings of two FP32 sums of the logit, lse and the backward pass's
    own, in orders that differ (of padded rows, and of rows as they lie): each
    (width / 32 + 6) 2^-24 of sum |x w|; and its own (half of FP16's least step,
    2^-24, is more than these)."""
    x, weight, target, dloss = make(3, 4097, 1, kind)
    loss, lse = tile.linear_cross_entropy(x, weight, target)
    assert not loss.any()
    dx, dweight = tile.linear_cross_entropy_backward(x, weight, target, lse, dloss)
    mag = x.double().abs() @ weight.double().abs().t()
    off = ((4097 / 32 + 6) * 2.0 ** -23 * mag + 2.0 ** -23) * dloss.double()[:, None]
    least = torch.finfo(x.dtype).smallest_normal * torch.finfo(x.dtype).eps / 2
    assert (dx.double().abs() <= 1.01 * off * weight.double().abs() + least).all()
    assert (dweight.double().abs() <= 1.01 * (off * x.double().abs()).sum(0) + least).all()


@pytest.mark.parametrize("kind", list(TYPES))
def test_gradients_of_wide_exact_rows(kind):
    """The recomputed logits of the backward pass are as exact: with a
    single product to a logit, p is off by the roundings of a logit
    (of_logit) and of lse, not by a share that grows with the width."""
    rows, width, vocab = 20, 131072, 300
    gen = torch.Generator(device="cuda").manual_seed(26)
    t = TYPES[kind]
    weight = torch.randn(vocab, width, device="cuda", generator=gen).to(t)
    x = torch.zeros(rows, width, dtype=t, device="cuda")
    at = torch.randint(width, (rows,), device="cuda", generator=gen)
    r = torch.arange(rows, device="cuda")
    x[r, at] = 12.0
    target = torch.randint(vocab, (rows,), device="cuda", generator=gen)
    loss, lse = tile.linear_cross_entropy(x, weight, target)
    dloss = torch.rand(rows, device="cuda", generator=gen) + 0.5
    dx, _ = tile.linear_cross_entropy_backward(x, weight, target, lse, dloss, need_dweight=False)
    l = x.double() @ weight.double().t()
    p = torch.exp(l - lse.double()[:, None])
    g = p.clone()
    g[r, target] -= 1.0
    g *= dloss.double()[:, None]
    half = torch.finfo(t).eps / 2
    gerr = half * g.abs() + p * dloss.double()[:, None] * (
        2.0 ** -18 + of_logit(width) * l.abs() + 2.0 ** -22 * lse.double().abs()[:, None])
    # the target's, from an FP32 dot product and expm1
    gerr[r, target] += 2.0 ** -20 * (1 + lse.double().abs()) * dloss.double()
    if t == torch.float16:
        gerr += 2.0 ** -39 * dloss.max().double()
    ref = g @ weight.double()
    tol = half * ref.abs() + 1.01 * gerr @ weight.double().abs() + \
        (vocab / 16 + 2) * 2.0 ** -22 * (g.abs() @ weight.double().abs())
    assert ((dx.double() - ref).abs() <= tol).all()
    # and in the 2-norm, where roundings of 16 bits would hide a bias of p
    off = p * dloss.double()[:, None] * (2.0 ** -18 + 2 * of_logit(width) * l.abs().amax())
    roundings = half * ((g.square() @ weight.double().square()).sqrt().norm() + ref.norm())
    assert (dx.double() - ref).norm() <= roundings + (off @ weight.double().abs()).norm()
