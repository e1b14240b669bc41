"""The block norm and its gradients against a plain implementation in FP64.

Tolerances count roundings.  An output of type t is rounded once: half a
step, finfo(t).eps / 2 of its value.  Everything before that is FP32: each
quantity is a sum of a few terms whose scalars (means of at most 131072
squares or products, added by threads of at most 32 elements and trees of
10 and 3 levels, then square roots and products) carry at most 64 roundings
of 2^-24, relative to the same sum over absolute values.  Column sums add
at most 300 terms one after another (a program's rows, then runs of
programs): 400 roundings."""

import pytest
import torch

import tile_compiler_row_gb300 as tile

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def device():
    from tile_compiler_row_gb300 import _build
    _build.build()
    tile.load()
    torch.cuda.set_device(0)


def make(rows, width, kind, gate=0, seed=1, offset=0):
    """Inputs of a case; `offset` elements shift every row matrix off its
    16-byte alignment."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[kind]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    def matrix(scale):
        flat = torch.empty(rows * width + offset, dtype=t, device="cuda")
        m = flat[offset:].view(rows, width)
        m.copy_(normal(rows, width) * scale)
        return m

    s = {"x": matrix(1.5), "residual": matrix(3.0), "dhidden": matrix(0.5), "dout": matrix(1.0),
         "gamma_post": 1.0 + 0.3 * normal(width), "gamma_pre": 1.0 + 0.3 * normal(width),
         "gate": None}
    if gate:
        s["gate"] = 0.5 + 0.5 * normal(-(-rows // gate), width)
    return s


def half_step(t):
    return torch.finfo(t).eps / 2


def check(got, ref, mag, roundings, what):
    t = got.dtype
    tiny = torch.finfo(t).smallest_normal * torch.finfo(t).eps
    tol = half_step(t) * ref.abs() + roundings * F32 * mag.abs() + tiny
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values off, the first at "
                           f"{bad.nonzero()[0].tolist()}: {got[bad][0].item()} for "
                           f"{ref[bad][0].item()}, tolerance {tol[bad][0].item():.3e}")


def gates(s, per):
    rows = s["x"].shape[0]
    if s["gate"] is None:
        return torch.ones(1, 1, dtype=torch.float64, device="cuda")
    return s["gate"].double().repeat_interleave(per, 0)[:rows]


def reference(s, post, pre, per, scale, eps):
    b, r, gate = s["x"].double(), s["residual"].double(), gates(s, per)
    n = b
    if post:
        n = b / (b.square().mean(1, keepdim=True) + eps).sqrt() * s["gamma_post"].double()
    h = scale * r + gate * n
    mag = (scale * r).abs() + (gate * n).abs()
    if not pre:
        return h, mag, None, None
    r2 = 1 / (h.square().mean(1, keepdim=True) + eps).sqrt()
    g = s["gamma_pre"].double()
    # an error of h also moves its mean square
    shift = (h.abs() * mag).mean(1, keepdim=True) * r2 ** 2
    return h, mag, h * r2 * g, (mag + h.abs() * shift) * r2 * g


def reference_backward(s, hidden, post, pre, per, scale, eps, use_dhidden=True):
    """{name: (gradient, magnitude)}."""
    b, h, gate = s["x"].double(), hidden.double(), gates(s, per)
    dh = s["dhidden"].double() if use_dhidden else torch.zeros_like(h)
    gh, mag, out = dh, dh.abs(), {}
    if pre:
        r2 = 1 / (h.square().mean(1, keepdim=True) + eps).sqrt()
        gy = s["dout"].double() * s["gamma_pre"].double()
        gh = gh + r2 * gy - h * r2 ** 3 * (gy * h).mean(1, keepdim=True)
        mag = mag + r2 * gy.abs() + h.abs() * r2 ** 3 * (gy * h).abs().mean(1, keepdim=True)
        t = s["dout"].double() * h * r2
        out["dgamma_pre"] = (t.sum(0), t.abs().sum(0))
    out["dresidual"] = (scale * gh, abs(scale) * mag)
    w = gate * (s["gamma_post"].double() if post else 1.0)
    u, umag = w * gh, w.abs() * mag
    unit = b
    if post:
        r1 = 1 / (b.square().mean(1, keepdim=True) + eps).sqrt()
        unit = b * r1
        out["din"] = (r1 * u - b * r1 ** 3 * (u * b).mean(1, keepdim=True),
                      r1 * umag + b.abs() * r1 ** 3 * (umag * b.abs()).mean(1, keepdim=True))
    else:
        out["din"] = (u, umag)
    t, tm = gh * unit, mag * unit.abs()
    if post:
        out["dgamma_post"] = ((gate * t).sum(0), (gate.abs() * tm).sum(0))
    if s["gate"] is not None:
        g = s["gamma_post"].double() if post else torch.ones_like(t[0])
        out["dgate"] = (torch.stack([p.sum(0) for p in t.split(per)]) * g,
                        torch.stack([p.sum(0) for p in tm.split(per)]) * g.abs())
    return out


# rows, width, gate rows of a case: one row and one column, widths around the
# vectors, warps and CTAs of a row, clusters of 2, 4 and 8, the widest row;
# row counts below, at and above the programs
SHAPES = [(1, 1, 0), (3, 7, 2), (1, 8, 1), (5, 63, 0), (37, 64, 10), (200, 257, 7),
          (1000, 256, 1000), (700, 1537, 100), (64, 2048, 10), (9, 4095, 4), (64, 4096, 64), (11, 4104, 0),
          (6, 8192, 5), (5, 9001, 2), (7, 16384, 3), (3, 20000, 2), (3, 40008, 2), (2, 65536, 1),
          (2, 70001, 0), (2, 131072, 2), (2, 131071, 1), (5000, 136, 17),
          # odd widths with more gate rows than programs keep to
          (1000, 63, 3), (301, 129, 1), (1100, 68, 1)]


@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False)],
                         ids=["both", "pre", "post"])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,width,gate", SHAPES)
def test_block_norm(rows, width, gate, kind, post, pre):
    s = make(rows, width, kind, gate)
    scale = 0.7 if width % 2 else 1.0
    hidden, out = tile.block_norm(s["x"], s["residual"], s["gamma_post"] if post else None,
                                  s["gate"], s["gamma_pre"] if pre else None, post, pre, gate,
                                  scale)
    h, hm, y, ym = reference(s, post, pre, gate, scale, 1e-5)
    check(hidden, h, hm, 64, "hidden")
    if pre:
        check(out, y, ym, 128, "out")
    else:
        assert out is None
    dy = s["dout"] if pre else None
    din, dres, dgp, dgate, dgn = tile.block_norm_backward(
        s["x"], hidden, s["gamma_post"] if post else None, s["gate"],
        s["gamma_pre"] if pre else None, s["dhidden"], dy, post, pre, gate, scale)
    ref = reference_backward(s, hidden, post, pre, gate, scale, 1e-5)
    check(dres, *ref["dresidual"], 128, "dresidual")
    check(din, *ref["din"], 192, "din")
    for name, got in (("dgamma_post", dgp), ("dgate", dgate), ("dgamma_pre", dgn)):
        assert (got is not None) == (name in ref), name
        if got is not None:
            check(got, *ref[name], 400, name)
    assert tile.tile_check_device_status() == 0


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("offset", [1, 3])
def test_unaligned_rows(kind, offset):
    """Row matrices that start off a 16-byte boundary, and one that does
    while the others do not."""
    s = make(33, 512, kind, 33, offset=offset)
    s["x"] = s["x"].clone()
    hidden, out = tile.block_norm(s["x"], s["residual"], s["gamma_post"], s["gate"],
                                  s["gamma_pre"], rows_per_gate=33)
    h, hm, y, ym = reference(s, True, True, 33, 1.0, 1e-5)
    check(hidden, h, hm, 64, "hidden")
    check(out, y, ym, 128, "out")
    got = tile.block_norm_backward(s["x"], hidden, s["gamma_post"], s["gate"], s["gamma_pre"],
                                   s["dhidden"], s["dout"], rows_per_gate=33)
    ref = reference_backward(s, hidden, True, True, 33, 1.0, 1e-5)
    for name, g, n in zip(("din", "dresidual", "dgamma_post", "dgate", "dgamma_pre"), got,
                          (192, 128, 400, 400, 400)):
        check(g, *ref[name], n, name)


def test_unaligned_parameters():
    s = make(20, 256, "bf16", 20)
    for k in ("gamma_post", "gamma_pre"):
        s[k] = torch.cat([s[k][:1], s[k]])[1:]
    flat = torch.empty(257, device="cuda")
    flat[1:] = s["gate"][0]
    s["gate"] = flat[1:].view(1, 256)
    hidden, out = tile.block_norm(s["x"], s["residual"], s["gamma_post"], s["gate"],
                                  s["gamma_pre"], rows_per_gate=20)
    h, hm, y, ym = reference(s, True, True, 20, 1.0, 1e-5)
    check(hidden, h, hm, 64, "hidden")
    check(out, y, ym, 128, "out")


@pytest.mark.parametrize("gate", [0, 5])
def test_null_parameters_are_ones_and_dhidden_may_be_none(gate):
    s = make(23, 200, "f32", gate)
    hidden, out = tile.block_norm(s["x"], s["residual"], None, s["gate"], None, rows_per_gate=gate)
    ones = torch.ones(200, device="cuda")
    s["gamma_post"] = s["gamma_pre"] = ones
    h, hm, y, ym = reference(s, True, True, gate, 1.0, 1e-5)
    check(hidden, h, hm, 64, "hidden")
    check(out, y, ym, 128, "out")
    got = tile.block_norm_backward(s["x"], hidden, None, s["gate"], None, None, s["dout"],
                                   rows_per_gate=gate)
    ref = reference_backward(s, hidden, True, True, gate, 1.0, 1e-5, use_dhidden=False)
    check(got[0], *ref["din"], 192, "din")
    check(got[1], *ref["dresidual"], 128, "dresidual")
    assert got[2] is None and got[4] is None
    if gate:
        check(got[3], *ref["dgate"], 400, "dgate")


def test_zero_rows():
    x = torch.empty(0, 64, device="cuda")
    hidden, out = tile.block_norm(x, x, None, None, None)
    assert hidden.shape == out.shape == (0, 64)
    g = torch.ones(64, device="cuda")
    _, _, dgp, dgate, dgn = tile.block_norm_backward(x, x, g, None, g, x, x)
    assert dgate is None and not dgp.any() and not dgn.any()


def test_zero_rows_of_the_matrix_and_non_finite_rows_stay_apart():
    """A row of zeros gives zeros (the norm's eps); a row with a NaN or an
    infinity spoils itself only."""
    s = make(8, 320, "f32")
    s["x"][2] = 0.0
    s["residual"][2] = 0.0
    s["x"][4, 17] = float("nan")
    s["x"][6, 3] = float("inf")
    hidden, out = tile.block_norm(s["x"], s["residual"], s["gamma_post"], None, s["gamma_pre"])
    assert not hidden[2].any() and not out[2].any()
    assert out[4].isnan().all()
    keep = [0, 1, 2, 3, 5, 7]
    h, hm, y, ym = reference(s, True, True, 0, 1.0, 1e-5)
    check(hidden[keep], h[keep], hm[keep], 64, "hidden")
    check(out[keep], y[keep], ym[keep], 128, "out")


def test_cancelling_residual_sum():
    """h far smaller than its two terms: its norm is that of the h computed,
    not of a combination of sums."""
    s = make(16, 1024, "f32")
    b = s["x"].double()
    n = b / (b.square().mean(1, keepdim=True) + 1e-5).sqrt() * s["gamma_post"].double()
    s["residual"] = (-n).float()
    hidden, out = tile.block_norm(s["x"], s["residual"], s["gamma_post"], None, s["gamma_pre"])
    h, hm, _, _ = reference(s, True, True, 0, 1.0, 1e-5)
    check(hidden, h, hm, 64, "hidden")
    # given that hidden, out is its norm
    r2 = 1 / (hidden.double().square().mean(1, keepdim=True) + 1e-5).sqrt()
    y = hidden.double() * r2 * s["gamma_pre"].double()
    check(out, y, y, 64, "out")


def test_repeated_calls_are_bitwise_the_same():
    s = make(900, 1000, "bf16", 70)
    args = (s["x"], s["x"], s["gamma_post"], s["gate"], s["gamma_pre"], s["dhidden"], s["dout"])
    first = tile.block_norm_backward(*args, rows_per_gate=70)
    for _ in range(3):
        for a, b in zip(first, tile.block_norm_backward(*args, rows_per_gate=70)):
            assert torch.equal(a, b)


def test_gradients_against_differences():
    """d(sum(dh * hidden) + sum(dy * out)) along a direction of every input,
    from FP64 differences of the reference, against the library's gradients
    (FP32 rows)."""
    rows, width, per = 6, 48, 4
    s = make(rows, width, "f32", per)
    hidden, _ = tile.block_norm(s["x"], s["residual"], s["gamma_post"], s["gate"], s["gamma_pre"],
                                rows_per_gate=per, residual_scale=0.7)
    got = tile.block_norm_backward(s["x"], hidden, s["gamma_post"], s["gate"], s["gamma_pre"],
                                   s["dhidden"], s["dout"], rows_per_gate=per, residual_scale=0.7)
    grads = dict(zip(("x", "residual", "gamma_post", "gate", "gamma_pre"), got))

    def value(step):
        q = {k: (v.double() + step.get(k, 0.0)) if v is not None else None for k, v in s.items()}
        h, _, y, _ = reference(q, True, True, per, 0.7, 1e-5)
        return (s["dhidden"].double() * h).sum() + (s["dout"].double() * y).sum()

    gen = torch.Generator(device="cuda").manual_seed(5)
    for name, grad in grads.items():
        d = torch.randn(s[name].shape, device="cuda", generator=gen, dtype=torch.float64)
        e = 1e-5
        slope = (value({name: e * d}) - value({name: -e * d})) / (2 * e)
        want = (grad.double() * d).sum()
        # FP32 gradients (and hidden rounded to FP32): 1e-5 of the terms' sum
        assert (slope - want).abs() <= 1e-5 * (grad.double() * d).abs().sum(), name


def test_streams_and_graph():
    """A call on another stream, and a captured forward and backward pass
    replayed on changed inputs, against eager calls."""
    s = make(300, 768, "bf16", 100)
    eager = tile.block_norm(s["x"], s["residual"], s["gamma_post"], s["gate"], s["gamma_pre"],
                            rows_per_gate=100)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = tile.block_norm(s["x"], s["residual"], s["gamma_post"], s["gate"], s["gamma_pre"],
                            rows_per_gate=100, stream=side)
    side.synchronize()
    for a, b in zip(eager, other):
        assert torch.equal(a, b)

    def both():
        h, y = tile.block_norm(s["x"], s["residual"], s["gamma_post"], s["gate"], s["gamma_pre"],
                               rows_per_gate=100)
        return (h, y) + tile.block_norm_backward(s["x"], h, s["gamma_post"], s["gate"],
                                                 s["gamma_pre"], s["dhidden"], y,
                                                 rows_per_gate=100)
    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = both()
    for k in range(2):
        s["x"].add_(0.25 + k)
        graph.replay()
        for a, b in zip(captured, both()):
            assert torch.equal(a, b)


def test_rows_behind_are_left_as_they_were():
    """Outputs' neighbours in memory, and the workspace's, are not written
    (whole vectors, and rows that end inside one)."""
    for width in (96, 99):
        s = make(37, width, "bf16", 5)
        bufs = [torch.full((41, width), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        mats = [b[:37] for b in bufs]
        need = tile.tile_block_norm_backward_workspace_bytes(37, width)
        ws = torch.full((need + 512,), 3, dtype=torch.uint8, device="cuda")
        grads = torch.full((12, width), 7.0, device="cuda")
        tile.tile_block_norm(s["x"], s["residual"], mats[0], mats[1], s["gamma_post"], s["gate"],
                             s["gamma_pre"], rows_per_gate=5)
        tile.tile_block_norm_backward(s["x"], mats[0], s["dhidden"], s["dout"], mats[2], mats[3],
                                      ws[:need], s["gamma_post"], s["gate"], s["gamma_pre"],
                                      grads[0], grads[1:9], grads[9], rows_per_gate=5)
        assert all((b[37:] == 7).all() for b in bufs)
        assert (grads[10:] == 7).all() and (ws[need:] == 3).all()
        ref = reference_backward(s, mats[0], True, True, 5, 1.0, 1e-5)
        check(mats[2], *ref["din"], 192, "din")
        check(grads[1:9], *ref["dgate"], 400, "dgate")


# as many programs as run at once (rows / 4 and more), row classes among them,
# column sums over all of them
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,width,gate", [(30000, 64, 700), (20001, 257, 9000), (12000, 1001, 0),
                                             (11000, 1024, 11000), (9999, 1028, 5),
                                             # and rows split between CTAs
                                             (700, 5120, 9), (900, 5111, 0), (500, 6152, 500),
                                             (300, 9224, 20), (310, 12288, 0), (260, 14600, 7),
                                             (170, 20480, 3), (90, 32768, 0)])
def test_many_rows(rows, width, gate, kind):
    s = make(rows, width, kind, gate, seed=4)
    hidden, out = tile.block_norm(s["x"], s["residual"], s["gamma_post"], s["gate"], s["gamma_pre"],
                                  rows_per_gate=gate)
    h, hm, y, ym = reference(s, True, True, gate, 1.0, 1e-5)
    check(hidden, h, hm, 64, "hidden")
    check(out, y, ym, 128, "out")
    got = dict(zip(("din", "dresidual", "dgamma_post", "dgate", "dgamma_pre"),
                   tile.block_norm_backward(s["x"], hidden, s["gamma_post"], s["gate"],
                                            s["gamma_pre"], s["dhidden"], s["dout"],
                                            rows_per_gate=gate)))
    for name, (ref, mag) in reference_backward(s, hidden, True, True, gate, 1.0, 1e-5).items():
        # a column's sum has at most rows / 600 + 160 additions in a chain
        check(got[name], ref, mag, 400, name)
    assert tile.tile_check_device_status() == 0


@pytest.mark.parametrize("width", [16384, 16383])
def test_past_two_to_the_31_elements(width):
    """Rows below and above element 2^31, each against FP64; the gradients'
    rows that are not looked at are zero, so column sums are those of the
    rows that are."""
    rows = (1 << 31) // width + 1000
    look = torch.tensor([0, 1, (1 << 31) // width, (1 << 31) // width + 1, rows - 2, rows - 1],
                        device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    few = make(len(look), width, "bf16", 0, seed=9)
    few["gate"] = torch.randn(1, width, device="cuda", generator=gen)
    big = {}
    for name in ("x", "residual", "dhidden", "dout"):
        big[name] = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
        big[name][look] = few[name]
    args = few["gamma_post"], few["gate"], few["gamma_pre"]
    hidden, out = tile.block_norm(big["x"], big["residual"], *args)
    h, hm, y, ym = reference(few, True, True, len(look), 1.0, 1e-5)
    check(hidden[look], h, hm, 64, "hidden")
    check(out[look], y, ym, 128, "out")
    del out, big["residual"]
    names = "din", "dresidual", "dgamma_post", "dgate", "dgamma_pre"
    got = dict(zip(names, tile.block_norm_backward(big["x"], hidden, *args, big["dhidden"],
                                                   big["dout"])))
    ref = reference_backward(few, hidden[look], True, True, len(look), 1.0, 1e-5)
    for name in names:
        check(got[name][look] if name in ("din", "dresidual") else got[name], *ref[name], 400, name)
    assert tile.tile_check_device_status() == 0


def test_agrees_with_the_weighted_rmsnorm():
    """Without a block norm and with a zero residual the block norm is the
    library's weighted RMSNorm."""
    s = make(64, 1024, "f32")
    zero = torch.zeros_like(s["x"])
    hidden, out = tile.block_norm(s["x"], zero, None, None, s["gamma_pre"], post=False)
    assert torch.equal(hidden, s["x"])
    want = torch.empty_like(out)
    tile.tile_rmsnorm_weighted_f32(s["x"], s["gamma_pre"], want)
    assert torch.allclose(out, want, rtol=16 * F32, atol=0)
