"""The embedding lookup and its gradient against FP64.

Bounds, element by element.  The lookup rounds its FP32 product and then the
output: 2^-24 + eps / 2 of the value.  The gradient of a token that occurs n times
sums n values in FP32 in some order, n - 1 roundings of partial sums that are at
most the sum of magnitudes, then the scale's fused multiply-add: (n + 1) 2^-24 of
scale times that sum (and of what it is added to), and the output's eps / 2.  A
subnormal FP16 result is off by half its step, 2^-25, instead.
"""

import pytest
import torch

import tile_compiler_row_gb300 as tile

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
IGNORE = -100
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def device():
    from tile_compiler_row_gb300 import _build
    _build.build()
    tile.load()
    torch.cuda.set_device(0)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, device="cuda", generator=gen(seed)).to(dtype)


def half_step(dtype, value):
    return value.abs() * (torch.finfo(dtype).eps / 2) + (2.0 ** -25 if dtype is torch.float16 else 0.0)


def offset_view(t, elements):
    """The same values from a place that is so many elements off the 16-byte grid."""
    flat = torch.empty(t.numel() + elements, dtype=t.dtype, device=t.device)
    view = flat[elements:].view(t.shape)
    view.copy_(t)
    return view


def check_lookup(token, weight, scale, out):
    ref = weight.double()[token.clamp(0, weight.shape[0] - 1)] * scale
    ref[token == IGNORE] = 0.0
    bound = (ref.abs() * U + half_step(weight.dtype, ref)) * (1 + 2.0 ** -7)
    assert torch.isfinite(out).all()
    worst = ((out.double() - ref).abs() - bound).max()
    assert worst <= 0, float(worst)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width,vocab", [(1, 1, 1), (1, 2048, 50), (3, 7, 5), (4, 64, 300),
                                              (5, 1537, 1001), (17, 8, 9), (64, 4097, 33),
                                              (1000, 96, 5000), (33, 131072, 3), (2, 131071, 4)])
def test_lookup(dtype, rows, width, vocab):
    weight = normal(rows, vocab, width, dtype=dtype)
    token = torch.randint(vocab, (rows,), device="cuda", generator=gen(2))
    token[::5] = IGNORE
    for scale in (1.0, -0.3, 64.0):
        check_lookup(token, weight, scale, tile.embedding(token, weight, scale=scale))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("source", [0, 1, 3, 8])
@pytest.mark.parametrize("target", [0, 1, 6])
def test_lookup_from_any_alignment(dtype, source, target):
    """Rows that begin anywhere, read and written; neighbours are left alone."""
    for width in (1, 5, 8, 33, 257, 1024):
        weight = offset_view(normal(1, 40, width, dtype=dtype), source)
        token = torch.randint(40, (29,), device="cuda", generator=gen(2))
        room = torch.full((29 * width + 32,), 7.0, dtype=dtype, device="cuda")
        out = room[target:target + 29 * width].view(29, width)
        tile.tile_embedding(token, weight, out, 0.7)
        check_lookup(token, weight, 0.7, out)
        assert (room[:target] == 7.0).all() and (room[target + 29 * width:] == 7.0).all()


def test_lookup_of_ignored_and_bad_tokens():
    weight = normal(1, 10, 40)
    weight[0] = float("nan")     # entry 0 is not read by a row that ignores it
    token = torch.tensor([3, 0, 0, 9], device="cuda")
    out = tile.embedding(token, weight, scale=2.0, ignore_index=0)
    assert (out[1:3] == 0).all() and torch.equal(out[0], weight[3] * 2) and torch.equal(out[3], weight[9] * 2)
    assert tile.tile_check_device_status() == 0
    for bad in (10, -1, 1 << 40, -(1 << 62)):
        token = torch.tensor([3, bad, 9], device="cuda")
        out = tile.embedding(token, weight)
        assert torch.isnan(out[1]).all() and torch.equal(out[2], weight[9])
        assert tile.tile_check_device_status() == -9 and tile.tile_check_device_status() == 0
    # an infinite value times a scale of 0 is the product's NaN, but not in an ignored row
    weight[1] = float("inf")
    out = tile.embedding(torch.tensor([1, IGNORE], device="cuda"), weight, scale=0.0)
    assert torch.isnan(out[0]).all() and (out[1] == 0).all()


def check_gradient(token, dout, scale, got, old=None):
    vocab, width = got.shape
    keep = (token >= 0) & (token < vocab) & (token != IGNORE)
    t, d = token[keep], dout[keep].double()
    total = torch.zeros(vocab, width, device="cuda", dtype=torch.float64).index_add_(0, t, d)
    size = torch.zeros(vocab, width, device="cuda", dtype=torch.float64).index_add_(0, t, d.abs())
    n = torch.bincount(t, minlength=vocab)[:, None].double()
    ref = total * scale + (old.double() if old is not None else 0.0)
    spread = size * abs(scale) + (old.double().abs() if old is not None else 0.0)
    bound = (n + 1) * U * spread
    bound = (bound + half_step(got.dtype, ref.abs() + bound)) * (1 + 2.0 ** -7)
    bound[n[:, 0] == 0] = 0.0    # what no token touches is exactly zero, or as it was
    worst = ((got.double() - ref).abs() - bound).max()
    assert worst <= 0, float(worst)


def tokens(rows, vocab, kind, seed=5):
    g = gen(seed)
    t = torch.randint(vocab, (rows,), device="cuda", generator=g)
    if kind == "one":            # every row the same entry
        t.fill_(vocab // 2)
    elif kind == "padded":       # half the rows one entry, a tenth ignored
        pick = torch.rand(rows, device="cuda", generator=g)
        t[pick < 0.5] = vocab - 1
        t[pick > 0.9] = IGNORE
    elif kind == "rare":         # tokens by frequency
        t = (torch.exp(torch.rand(rows, device="cuda", generator=g)
                       * torch.log(torch.tensor(float(vocab)))) - 1).long().clamp_(0, vocab - 1)
    elif kind == "none":
        t.fill_(IGNORE)
    return t


SHAPES = [(1, 1, 1), (1, 64, 7), (48, 1024, 200), (300, 1537, 100), (2048, 65, 5000),
          (2049, 65, 5000), (2500, 8, 1), (5000, 257, 513), (4097, 1000, 512), (256, 8200, 40),
          (257, 64, 3000), (6144, 40, 900), (6145, 40, 900), (20000, 24, 70000), (9000, 8, 300001),
          (50000, 24, 700), (140000, 16, 300)]


@pytest.mark.parametrize("rows,vocab,kind", [(1 << 20, 100000, "rare"), (1 << 20, 3, "uniform"),
                                             (1 << 24, 100000, "padded")])
def test_gradient_of_many_rows(rows, vocab, kind):
    token = tokens(rows, vocab, kind)
    dout = normal(3, rows, 3)
    check_gradient(token, dout, 0.7, tile.embedding_backward(token, dout, vocab, scale=0.7))


@pytest.mark.parametrize("kind", ["uniform", "one", "padded", "rare", "none"])
@pytest.mark.parametrize("rows,width,vocab", SHAPES)
def test_gradient(rows, width, vocab, kind):
    token = tokens(rows, vocab, kind)
    for dtype, into in ((torch.float32, None), (torch.bfloat16, None), (torch.float16, torch.float32)):
        dout = normal(3, rows, width, dtype=dtype)
        got = tile.embedding_backward(token, dout, vocab, scale=0.7, dtype=into)
        assert got.dtype is (into or dtype)
        check_gradient(token, dout, 0.7, got)
        old = normal(4, vocab, width, dtype=into or dtype)
        dweight = old.clone()
        assert tile.embedding_backward(token, dout, scale=-2.0, dweight=dweight) is dweight
        check_gradient(token, dout, -2.0, dweight, old)
    assert tile.tile_check_device_status() == 0


@pytest.mark.parametrize("rows", [100, 3000])
@pytest.mark.parametrize("dtype,into", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                        (torch.float16, torch.float32)])
def test_gradient_from_any_alignment(rows, dtype, into):
    """Every pair of alignments of the rows read and written; rows that no token
    touches, and what lies around the matrix, are left alone when adding."""
    for width, source, target in ((1, 0, 1), (7, 1, 0), (40, 3, 5), (64, 1, 1), (129, 0, 2), (513, 7, 3)):
        token = tokens(rows, 60, "uniform")
        token[token == 11] = 12
        dout = offset_view(normal(3, rows, width, dtype=dtype), source)
        room = torch.full((60 * width + 32,), 7.0, dtype=into, device="cuda")
        dweight = room[target:target + 60 * width].view(60, width)
        old = normal(4, 60, width, dtype=into)
        old[11] = float("nan")
        dweight.copy_(old)
        ws = torch.empty(tile.tile_embedding_backward_workspace_bytes(rows, width, 60) or 1,
                         dtype=torch.uint8, device="cuda")
        tile.tile_embedding_backward(token, dout, dweight, ws, 1.5, accumulate=True)
        assert torch.isnan(dweight[11]).all()
        dweight[11] = old[11] = 0.0
        check_gradient(token, dout, 1.5, dweight, old)
        assert (room[:target] == 7.0).all() and (room[target + 60 * width:] == 7.0).all()


@pytest.mark.parametrize("rows", [200, 4000])
def test_gradient_does_not_read_rows_that_take_no_part(rows):
    token = tokens(rows, 50, "padded")
    token[7] = 50
    token[8] = -3
    dout = normal(3, rows, 70)
    out = (token < 0) | (token >= 50)
    dout[out] = float("nan")
    got = tile.embedding_backward(token, dout, 50)
    assert tile.tile_check_device_status() == -9 and tile.tile_check_device_status() == 0
    check_gradient(torch.where(out, IGNORE, token), dout.nan_to_num(0.0), 1.0, got)
    # a NaN that takes part reaches its token's row and column alone
    dout = dout.nan_to_num(0.0)
    at = int((token == 49).nonzero()[3])
    dout[at, 5] = float("inf")
    bad = ~torch.isfinite(tile.embedding_backward(torch.where(out, IGNORE, token), dout, 50))
    assert bad.sum() == 1 and bad[49, 5]


def test_a_workspace_is_what_is_written():
    """Nothing in front of the workspace or behind it, whatever it holds."""
    for rows, width, vocab in ((2049, 33, 100), (9000, 64, 70000), (140000, 8, 3)):
        n = tile.tile_embedding_backward_workspace_bytes(rows, width, vocab)
        room = torch.full((n + 512,), 0xAB, dtype=torch.uint8, device="cuda")
        token, dout = tokens(rows, vocab, "padded"), normal(3, rows, width)
        got = torch.empty(vocab, width, device="cuda")
        tile.tile_embedding_backward(token, dout, got, room[256:256 + n])
        check_gradient(token, dout, 1.0, got)
        assert (room[:256] == 0xAB).all() and (room[256 + n:] == 0xAB).all()
        again = torch.empty_like(got)
        tile.tile_embedding_backward(token, dout, again, room[256:256 + n])
        assert torch.equal(got, again)


def test_no_rows():
    weight, none = normal(1, 7, 40), torch.empty(0, dtype=torch.int64, device="cuda")
    assert tile.embedding(none, weight).shape == (0, 40)
    dout = torch.empty(0, 40, device="cuda")
    assert not tile.embedding_backward(none, dout, 7).any()
    old = weight.clone()
    assert torch.equal(tile.embedding_backward(none, dout, dweight=weight), old)


@pytest.mark.parametrize("vocab", [300, 300001])
@pytest.mark.parametrize("rows", [3000, 20000])
def test_calls_one_after_another_in_one_workspace(rows, vocab):
    """Each launch is set up while the one before it runs: what a call finds in
    the workspace is its own, not the last call's."""
    width = 72
    sets = [(tokens(rows, vocab, kind, seed), normal(seed, rows, width)) for kind, seed in
            (("rare", 1), ("uniform", 2), ("padded", 3))]
    want = [tile.embedding_backward(t, d, vocab) for t, d in sets]
    ws = torch.empty(tile.tile_embedding_backward_workspace_bytes(rows, width, vocab), dtype=torch.uint8,
                     device="cuda")
    got = [[torch.empty(vocab, width, device="cuda") for _ in sets] for _ in range(4 if vocab > 1000 else 20)]
    torch.cuda.synchronize()
    for outs in got:
        for (t, d), o in zip(sets, outs):
            tile.tile_embedding_backward(t, d, o, ws)
    torch.cuda.synchronize()
    for outs in got:
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def test_gradient_against_differences():
    """(L(w + h d) - L(w - h d)) / 2h of L = sum(out c) is linear in w: FP64 sums
    of the FP32 lookups agree with <dweight, d> to their roundings, 2^-24 of
    each of the terms (twice, over 2h) and the gradient's own."""
    token = tokens(500, 40, "padded")
    w, c, d = normal(1, 40, 33), normal(2, 500, 33), normal(3, 40, 33)
    h = 0.5
    up, down = ((tile.embedding(token, (w + s * h * d), scale=0.7).double() * c.double()).sum()
                for s in (1, -1))
    grad = tile.embedding_backward(token, c, 40, scale=0.7)
    inner = (grad.double() * d.double()).sum()
    terms = (tile.embedding(token, w.abs() + d.abs(), scale=0.7).double() * c.double().abs()).sum()
    n = int(torch.bincount(token[token >= 0]).max())
    bound = 4 * U * terms / h + (n + 1) * U * (d.abs().double()[token.clamp(min=0)] * c.abs().double()).sum()
    assert abs((up - down) / (2 * h) - inner) <= bound


def test_large_offsets():
    """Rows of the weight and of the output that begin past 2^31 elements."""
    width = 65536
    weight = torch.zeros(40000, width, dtype=torch.float16, device="cuda")
    weight[39999] = normal(1, width, dtype=torch.float16)
    token = torch.tensor([39999, 0] * 17000, device="cuda")[:33000]
    out = tile.embedding(token, weight)
    assert torch.equal(out[32998], weight[39999]) and (out[32999] == 0).all()
    out[32998:] = normal(2, 2, width, dtype=torch.float16)
    token = torch.full((33000,), IGNORE, device="cuda")
    token[32998:] = 39999
    got = tile.embedding_backward(token, out, dweight=weight.zero_())
    check_gradient(token[32998:] - 39998, out[32998:], 1.0, got[39998:])
    assert not got[:39998].any()


def test_streams_graphs_and_calls_at_once():
    token, dout = tokens(3000, 500, "rare"), normal(3, 3000, 130, dtype=torch.bfloat16)
    few, fout = tokens(50, 500, "rare"), normal(5, 50, 130, dtype=torch.bfloat16)
    want = tile.embedding_backward(token, dout, 500), tile.embedding_backward(few, fout, 500)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for k, s in enumerate(streams * 3):
        args = (token, dout) if k % 2 == 0 else (few, fout)
        got.append(tile.embedding_backward(*args, 500, stream=s if k < 4 else s.cuda_stream))
    torch.cuda.synchronize()
    for k, g in enumerate(got):
        assert torch.equal(g, want[k % 2])
    # captured, replayed with other tokens and rows in the same place
    t, d = token.clone(), dout.clone()
    tile.embedding(t, want[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grad = tile.embedding_backward(t, d, 500)
        out = tile.embedding(t, grad)
    for seed in (11, 12):
        t.copy_(tokens(3000, 500, "padded", seed))
        d.copy_(normal(seed, 3000, 130, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(grad, tile.embedding_backward(t, d, 500))
        assert torch.equal(out, tile.embedding(t, grad))


# ---- sums that are exact ------------------------------------------------------------
#
# A bound of n roundings says nothing of a token that occurs a million times.  Of
# whole numbers, and a scale of 1/2, every sum in any order is exact in FP32 as long
# as the magnitudes add up to less than 2^24: the gradient is that of FP64, rounded
# once to its type.  One row left out, taken twice or put to another token shows.

PAIRS = [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
         (torch.float16, torch.float16), (torch.float16, torch.float32)]
LENGTHS = {"lengths": [1, 2, 7, 8, 9, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 192, 193, 256, 320, 1000],
           "whole runs": [64, 128, 64, 256, 192, 64, 64, 512, 1024, 320, 1536]}


def whole(seed, most, *shape, dtype=torch.float32):
    return torch.randint(-most, most + 1, shape, device="cuda", generator=gen(seed)).to(dtype)


def tokens_of_lengths(rows, vocab, lengths, seed=5):
    """Tokens that occur as often as `lengths` has it, one after another, shuffled: runs
    of the sorted list end in, at and next to them."""
    counts = torch.tensor(lengths, device="cuda").repeat(rows // sum(lengths) + 1)
    names = torch.arange(counts.numel(), device="cuda") % vocab
    t = torch.repeat_interleave(names.sort().values, counts)[:rows]
    return t[torch.randperm(rows, device="cuda", generator=gen(seed))]


def check_exact(rows, width, vocab, kind, pairs=PAIRS, most=2, source=0, target=0):
    token = tokens_of_lengths(rows, vocab, LENGTHS[kind]) if kind in LENGTHS else tokens(rows, vocab, kind)
    keep = token != IGNORE
    assert most * int(torch.bincount(token[keep], minlength=1).max()) + 200 < 1 << 24
    for dtype, into in pairs:
        dout = whole(3, most, rows, width, dtype=dtype)
        total = torch.zeros(vocab, width, device="cuda", dtype=torch.float64).index_add_(
            0, token[keep], dout[keep].double())
        dout = offset_view(dout, source)
        for old in (None, whole(4, 100, vocab, width, dtype=into)):
            room = torch.full((vocab * width + 32,), 7.0, dtype=into, device="cuda")
            got = room[target:target + vocab * width].view(vocab, width)
            if old is not None:
                got.copy_(old)
            need = tile.tile_embedding_backward_workspace_bytes(rows, width, vocab)
            ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None
            tile.tile_embedding_backward(token, dout, got, ws, 0.5, accumulate=old is not None)
            want = (total * 0.5 + (0.0 if old is None else old.double())).float().to(into)
            assert torch.equal(got, want), (dtype, into, old is not None, int((got != want).sum()))
            assert (room[:target] == 7.0).all() and (room[target + vocab * width:] == 7.0).all()
            del got, room, ws, want


@pytest.mark.parametrize("kind", ["uniform", "one", "padded", "rare", *LENGTHS])
@pytest.mark.parametrize("rows,width,vocab", SHAPES)
def test_exact_gradient(rows, width, vocab, kind):
    check_exact(rows, width, vocab, kind)


@pytest.mark.parametrize("kind", ["one", "padded", *LENGTHS])
@pytest.mark.parametrize("rows", [60, 3000, 9000])
@pytest.mark.parametrize("width,source,target", [(1, 0, 1), (33, 1, 0), (64, 1, 1), (129, 3, 2), (257, 0, 0)])
def test_exact_gradient_from_any_alignment(rows, width, source, target, kind):
    check_exact(rows, width, 60, kind, source=source, target=target)


@pytest.mark.parametrize("rows,vocab,kind", [(1 << 20, 100000, "rare"), (1 << 20, 3, "uniform"),
                                             (1 << 20, 900, "lengths"), (1 << 20, 900, "whole runs"), (131072, 70, "lengths"),
                                             (131073, 70, "lengths"), (1 << 20, 1, "one"),
                                             (1 << 24, 100000, "padded")])
def test_exact_gradient_of_many_rows(rows, vocab, kind):
    # (of 2^24 rows, half of one token and so 8.4e6 of them, -1 .. 1)
    check_exact(rows, 3, vocab, kind, PAIRS[:1], 2 if rows < 1 << 22 else 1)


# runs of more than 64 positions, where the partial sums would pass 64 MiB
@pytest.mark.parametrize("kind", ["one", "padded", "rare", *LENGTHS])
@pytest.mark.parametrize("rows,width,pair", [(131072, 4096, 1), (140001, 4001, 0), (1 << 20, 520, 4),
                                             (1 << 20, 1100, 2)])
def test_exact_gradient_of_long_runs(rows, width, kind, pair):
    assert rows * (width + 16) > 1 << 29
    check_exact(rows, width, 300, kind, PAIRS[pair:pair + 1])


@pytest.mark.parametrize("rows,width,vocab", [(7000, 5, 511), (7000, 5, 512), (7000, 3, 262143), (7000, 3, 262144),
                                              (9000, 1, (1 << 27) - 1), (9000, 1, (1 << 27) + 3), (3000, 1, (1 << 27) + 3)])
def test_exact_gradient_of_vocabularies_at_a_digit_end(rows, width, vocab):
    """1 to 4 passes of the sort, the last entries among the tokens."""
    token = tokens(rows, vocab, "uniform")
    token[::3] = vocab - 1 - token[::3] % 7
    dout = whole(3, 2, rows, width)
    for add in (False, True):
        got = torch.full((vocab, width), 3.0 if add else float("nan"), device="cuda")
        ws = torch.full((tile.tile_embedding_backward_workspace_bytes(rows, width, vocab),), 0xFF, dtype=torch.uint8,
                        device="cuda")
        tile.tile_embedding_backward(token, dout, got, ws, accumulate=add)
        want = torch.full((vocab, width), 3.0 if add else 0.0, device="cuda").index_add_(0, token, dout)
        assert torch.equal(got, want)
