"""The gradients' norm and the AdamW step.

The states are sums of two rounded products in FP32, which numpy's FP32 repeats
bit for bit on the host; so are the 8-bit codes, scales and random bits.  The
parameter's update u = rate m / (sqrt(v) root + eps) rounds rate, root and the
root of v once (2^-24 each), the quotient by 2 ulp (2^-22) and two products and
a sum around it: within 2^-20 of u, and 2^-22 of the parameter itself (its factor
1 - lr decay, the product and the sum).  The norm's squares and the 8 to 64 sums of a
chunk are FP32 and all positive: 2^-18 of the sum at most, and half of that of its root.
"""

import numpy as np
import pytest
import torch

import tile_compiler_row_gb300 as tile

pytestmark = pytest.mark.gpu

F32 = np.float32
TYPES = [torch.float32, torch.bfloat16, torch.float16]
SIZES = [1, 0, 3, 255, 256, 257, 4096, 4097, 10000, 33333]


@pytest.fixture(scope="module", autouse=True)
def device():
    from tile_compiler_row_gb300 import _build
    _build.build()
    tile.load()
    torch.cuda.set_device(0)


def normal(seed, n, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, device="cuda", generator=g) * scale).to(dtype)


def views(tensors, shift):
    """The same values, each tensor so many elements off the 16-byte grid, in
    one buffer with a value of its own between them."""
    if not tensors:
        return [], None
    room = torch.full((sum(t.numel() for t in tensors) + 64 * (len(tensors) + 1),), 7.0,
                      dtype=torch.float32, device="cuda").to(tensors[0].dtype)
    out, at = [], 0
    for t in tensors:
        at = -(-at // 32) * 32 + 16 + shift
        out.append(room[at:at + t.numel()].view(t.shape))
        out[-1].copy_(t)
        at += t.numel()
    return out, room


def norm64(tensors):
    return torch.stack([t.double().square().sum() for t in tensors]).sum().sqrt().item()


@pytest.mark.parametrize("shift", [0, 1, 5])
def test_norm(shift):
    for k, dtype in enumerate(TYPES):
        grads, _ = views([normal(i, n, dtype) for i, n in enumerate(SIZES)], shift)
        want = norm64(grads)
        for scale, most in ((1.0, None), (0.25, want / 8), (3.0, want * 4)):
            norm, factor = tile.grad_norm(grads, most, scale).tolist()
            assert abs(norm - want * scale) <= 2.0 ** -18 * want * scale
            bound = scale * min(1.0, (most or np.inf) / (want * scale))
            assert abs(factor - bound) <= 2.0 ** -18 * bound


@pytest.mark.parametrize("count", [1, 32, 33, 1024, 1025, 2500])
def test_norm_of_many(count):
    grads = [normal(i, 1 + 37 * i % 300, TYPES[i % 3]) for i in range(count)]
    got = tile.grad_norm(grads)
    assert abs(got[0].item() - norm64(grads)) <= 2.0 ** -18 * norm64(grads) and got[1] == 1.0
    assert torch.equal(got, tile.grad_norm(grads))


def test_norm_of_large_tensors():
    big = [normal(1, (1 << 26) + 5, torch.bfloat16), normal(2, 3000001)]
    assert abs(tile.grad_norm(big)[0].item() - norm64(big)) <= 2.0 ** -18 * norm64(big)
    past = torch.zeros((1 << 31) + 100, dtype=torch.bfloat16, device="cuda")
    past[-1], past[0] = 3.0, 4.0
    assert tile.grad_norm([past])[0] == 5.0


def test_norm_that_is_not_finite():
    for value in (float("inf"), -float("inf"), float("nan"), 1e30):
        grads = [normal(1, 5000), normal(2, 70, torch.bfloat16)]
        grads[0][4321] = value
        norm, factor = tile.grad_norm(grads, 1.0).tolist()
        assert not np.isfinite(norm) and np.isnan(factor)
    assert tile.grad_norm([torch.zeros(100, device="cuda")], 1.0, 0.5).tolist() == [0.0, 0.5]
    assert tile.grad_norm([torch.zeros(0, device="cuda")], 1.0, 0.5).tolist() == [0.0, 0.5]


# ---- the step ---------------------------------------------------------------------


def mix64(z):
    z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
    z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
    return z ^ (z >> np.uint64(31))


def random_words(n, tensor, step, seed):
    golden = np.uint64(0x9E3779B97F4A7C15)
    with np.errstate(over="ignore"):
        key = mix64(np.uint64(seed) + np.uint64(step) * golden)
        key = mix64(key + np.uint64(tensor + 1) * golden)
        i = np.arange(n, dtype=np.uint64)
        both = mix64(key + ((i >> np.uint64(1)) + np.uint64(1)) * golden)
    return np.where(i & np.uint64(1), both >> np.uint64(32), both & np.uint64(0xFFFFFFFF)).astype(np.uint32)


def block_scales(x):
    """2^(e - 7) for the exponent e of each 256 values' largest magnitude."""
    scales = np.ones(-(-x.size // 256), F32)
    for b in range(scales.size):
        top = np.abs(x[256 * b:256 * b + 256]).max()
        if top >= 2.0 ** -100:
            scales[b] = 2.0 ** (np.frexp(top)[1] - 1 - 7)
    return scales


def e4m3_at_random(y, bits):
    """Magnitudes below 256 rounded to e4m3's steps: up where the part cut off and
    bits / 2^16 pass 1."""
    y = y.astype(np.float64)
    place = np.floor(np.log2(np.maximum(y, 2.0 ** -6)))
    unit = 2.0 ** (place - 3)
    # bits join behind the 20 bits of the mantissa that are cut off (under 2^-6,
    # of y + 2^-6 rounded to FP32)
    low = y < 2.0 ** -6
    part = np.where(low, (y.astype(F32) + F32(2.0 ** -6)).astype(np.float64) - 2.0 ** -6, y) / unit
    return np.floor(part + bits / 65536.0) * unit


class Reference:
    """The step in numpy, FP32 as the kernel's, the update in FP64."""

    def __init__(self, p, grads, m, v, ms, vs, tensor, step, lr, betas, eps, decay, factor, seed):
        b1, b2 = F32(betas[0]), F32(betas[1])
        r1, r2 = F32(1.0 - betas[0]), F32(1.0 - betas[1])
        g = grads * F32(factor)
        if ms is not None:
            m = m * np.repeat(ms, 256)[:m.size]
            v = np.square(v * np.repeat(vs, 256)[:v.size])
        self.m = m * b1 + g * r1
        self.v = v * b2 + (g * g) * r2
        root = np.sqrt(self.v)
        assert self.m.dtype == F32 and self.v.dtype == F32 and root.dtype == F32
        u = lr / (1 - betas[0] ** step) * self.m.astype(np.float64) / (
            root.astype(np.float64) / np.sqrt(1 - betas[1] ** step) + np.float64(F32(eps)))
        self.p = p.astype(np.float64) * (1 - lr * decay) - u
        self.off = 2.0 ** -20 * np.abs(u) + 2.0 ** -22 * np.abs(p)
        if ms is not None:
            words = random_words(p.size, tensor, step, seed)
            self.m_scale, self.v_scale = block_scales(self.m), block_scales(root)
            y = np.abs(self.m) / np.repeat(self.m_scale, 256)[:p.size]
            self.m = e4m3_at_random(y, words & 0xFFFF) * np.sign(self.m)
            y = root / np.repeat(self.v_scale, 256)[:p.size]
            self.v = e4m3_at_random(y, words >> 16)
            self.v = np.where(y > 0, np.maximum(self.v, 2.0 ** -9), self.v)


def host(t):
    return t.float().cpu().numpy().reshape(-1)


def make(sizes, dtype, eight, copy, shift=0):
    """Parameters, gradients and states of a run under way."""
    s = {"params": views([normal(10 + i, n) for i, n in enumerate(sizes)], shift)[0],
         "grads": views([normal(50 + i, n, dtype, 10.0 ** (i % 5 - 4)) for i, n in enumerate(sizes)], shift)[0]}
    m = [normal(90 + i, n, scale=10.0 ** (i % 5 - 4)) for i, n in enumerate(sizes)]
    v = [t.square() * 2 + 1e-12 for t in m]
    if eight:
        for name, x in (("exp_avg", m), ("exp_avg_sq", [t.sqrt() for t in v])):
            scale = [torch.from_numpy(block_scales(host(t))).cuda() if t.numel() else
                     torch.zeros(0, device="cuda") for t in x]
            codes = [(t / c.repeat_interleave(256)[:t.numel()]).to(torch.float8_e4m3fn) for t, c in zip(x, scale)]
            room = torch.zeros(sum(sizes) + 64 * len(sizes), dtype=torch.float8_e4m3fn, device="cuda")
            at, s[name] = 0, []
            for c in codes:
                at = -(-at // 32) * 32 + shift
                s[name].append(room[at:at + c.numel()])
                s[name][-1].copy_(c)
                at += c.numel()
            s[name + "_scales"] = scale
    else:
        s["exp_avg"], s["exp_avg_sq"] = views(m, shift)[0], views(v, shift)[0]
    if copy is not None:
        s["copies"] = views([p.to(copy) for p in s["params"]], shift)[0]
    return s


def check_step(s, step, lr=1e-2, betas=(0.9, 0.95), eps=1e-8, decay=0.1, factor=None, seed=0):
    before = {k: [host(t) for t in v] for k, v in s.items()}
    count = len(s["params"])
    decays = decay if isinstance(decay, list) else [decay] * count
    f = None if factor is None else torch.tensor([factor], device="cuda")
    tile.adamw(**s, step=step, lr=lr, betas=betas, eps=eps, weight_decay=decay, factor=f, seed=seed)
    for i in range(count):
        if s["params"][i].numel() == 0:
            continue
        b = {k: v[i] for k, v in before.items()}
        r = Reference(b["params"], b["grads"], b["exp_avg"], b["exp_avg_sq"], b.get("exp_avg_scales"),
                      b.get("exp_avg_sq_scales"), i, step, lr, betas, eps, decays[i],
                      1.0 if factor is None else factor, seed)
        assert np.array_equal(host(s["exp_avg"][i]), r.m), i
        assert np.array_equal(host(s["exp_avg_sq"][i]), r.v), i
        if "exp_avg_scales" in s:
            assert np.array_equal(host(s["exp_avg_scales"][i]), r.m_scale)
            assert np.array_equal(host(s["exp_avg_sq_scales"][i]), r.v_scale)
        p = host(s["params"][i])
        assert (np.abs(p - r.p) <= r.off).all(), (i, np.abs(p - r.p).max())
        assert np.array_equal(host(s["grads"][i]), b["grads"])
        if "copies" in s:
            assert torch.equal(s["copies"][i], s["params"][i].to(s["copies"][i].dtype))


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("shift", [0, 1, 4])
@pytest.mark.parametrize("dtype", TYPES)
def test_step(dtype, shift, eight):
    for copy in (None, torch.bfloat16, torch.float16):
        s = make(SIZES, dtype, eight, copy, shift)
        check_step(s, step=3, factor=0.3, seed=9)
        check_step(s, step=4, decay=[0.1 * (i % 3) for i in range(len(SIZES))])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shifts", [(1, 2, 3, 1, 2), (0, 1, 0, 0, 0), (2, 2, 2, 2, 3), (3, 3, 3, 0, 3)])
def test_step_of_unlike_alignments(dtype, shifts):
    s = make(SIZES + [2, 4, 5, 1027], dtype, False, torch.bfloat16)
    for name, shift in zip(("params", "grads", "exp_avg", "exp_avg_sq", "copies"), shifts):
        s[name] = views(s[name], shift)[0]
    check_step(s, step=3, factor=0.3)


@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_step_of_like_alignments(shift):
    """Off the grid by the same elements, of every short length."""
    for copy in (None, torch.float16):
        check_step(make([*range(1, 12), 1023, 1024, 1025, 1027, 1028, 4099], torch.bfloat16, False, copy, shift), step=2)


@pytest.mark.parametrize("eight", [False, True])
def test_first_step_from_zero(eight):
    params = [normal(1, 1000).view(10, 100), normal(2, 257)]
    grads = [normal(3, 1000, scale=1e-6).view(10, 100), torch.zeros(257, device="cuda")]
    state = tile.adamw_state(params, 8 if eight else 32)
    assert state["exp_avg"][0].shape == (10, 100)
    check_step({"params": params, "grads": grads, **state}, step=1, betas=(0.9, 0.999))
    # no gradient at all: decay alone
    assert torch.allclose(params[1], normal(2, 257) * (1 - 1e-3), rtol=2.0 ** -21, atol=0)


@pytest.mark.parametrize("count", [31, 32, 33, 384, 385, 800])
@pytest.mark.parametrize("eight", [False, True])
def test_many_tensors(count, eight):
    s = make([1 + 53 * i % 400 for i in range(count)], torch.bfloat16, eight, torch.bfloat16)
    check_step(s, step=7)


@pytest.mark.parametrize("eight", [False, True])
def test_a_step_that_is_skipped(eight):
    s = make([5000, 300], torch.float32, eight, torch.bfloat16)
    before = {k: [t.clone() for t in v] for k, v in s.items()}
    for bad in (float("nan"), float("inf")):
        tile.adamw(**s, step=2, factor=torch.tensor([bad], device="cuda"))
        for k in s:
            for a, b in zip(s[k], before[k]):
                assert torch.equal(a.float(), b.float())
    s["grads"][0][17] = float("inf")
    tile.adamw(**s, step=2, factor=tile.grad_norm(s["grads"], 1.0)[1:])
    assert torch.equal(s["params"][0], before["params"][0])


def test_a_gradient_that_is_not_finite():
    """Without a factor that skips the step: its element in FP32 states, its
    block of 256 in 8-bit ones."""
    for eight in (False, True):
        s = make([1000], torch.float32, eight, None)
        s["grads"][0][300] = float("nan")
        tile.adamw(**s, step=2)
        bad = ~torch.isfinite(s["params"][0])
        assert bad.sum() == 1 and bad[300]
        m = s["exp_avg"][0].float()
        if eight:
            m = m * s["exp_avg_scales"][0].repeat_interleave(256)[:1000]
        bad = ~torch.isfinite(m)
        want = torch.zeros_like(bad)
        want[256:512 if eight else 257] = eight
        want[300] = True
        assert torch.equal(bad, want)


def test_eight_bits_move_as_they_should():
    """No gradient: v shrinks by beta2 a step, far less than half a step of e4m3.  The
    mean root over 2^16 elements is off by at most 6 standard deviations of a
    rounding at random: a step of e4m3 is at most 1/8 of the value, so each of 200
    roundings has at most 1/16 of it, of the mean 1/256 of that."""
    n = 1 << 16
    params, grads = [torch.zeros(n, device="cuda")], [torch.zeros(n, device="cuda")]
    s = tile.adamw_state(params, 8)
    s["exp_avg_sq"][0].copy_(torch.full((n,), 200.0, device="cuda"))
    s["exp_avg_sq_scales"][0].fill_(2.0 ** -10)
    for step in range(1, 201):
        tile.adamw(params, grads, **s, step=step, betas=(0.9, 0.99))
    root = s["exp_avg_sq"][0].float() * s["exp_avg_sq_scales"][0].repeat_interleave(256)
    # 200 in e4m3 is 192 or 208: torch rounds to the even one
    start = float(torch.tensor(200.0).to(torch.float8_e4m3fn)) * 2.0 ** -10
    want = start * 0.99 ** 100
    assert abs(root.mean().item() - want) <= 6 * start * 200 ** 0.5 / 16 / 256
    assert want < start / 2


def test_step_and_rate_on_the_device():
    """The same as from the host but for the rounding of the two corrections:
    expm1f's ulp, and a product t log(beta) of three roundings, 2^-21 of the update."""
    for eight in (False, True):
        a, b = (make([3000, 77], torch.bfloat16, eight, None) for _ in range(2))
        for step, lr in ((1, 1e-2), (5, 3e-3), (2000, 1e-3)):
            was = [p.clone() for p in a["params"]]
            tile.adamw(**a, step=step, lr=lr, seed=3)
            tile.adamw(**b, step=torch.tensor([step], device="cuda"), lr=torch.tensor([lr], device="cuda"), seed=3)
            for k in a:
                for x, y, w in zip(a[k], b[k], was if k == "params" else a[k]):
                    if k == "params":
                        assert ((x - y).abs() <= 2.0 ** -21 * (x - w).abs() + 2.0 ** -22 * w.abs()).all()
                        y.copy_(x)
                    else:
                        assert torch.equal(x.float(), y.float())


def test_large_tensor():
    """Elements past 2^31."""
    n = (1 << 31) + 1000
    p, m, v = (torch.zeros(n, device="cuda") for _ in range(3))
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-5:] = 1.0
    tile.adamw([p], [g], [m], [v], step=1, lr=0.5, weight_decay=0.0)
    assert torch.allclose(p[-5:], torch.full((5,), -0.5, device="cuda"), rtol=2.0 ** -19, atol=0)
    assert not p[:-5].any()
    del p, m, v
    p = torch.zeros(n, device="cuda")
    state = tile.adamw_state([p], 8)
    tile.adamw([p], [g], **state, step=1, lr=0.5, weight_decay=0.0)
    assert torch.allclose(p[-5:], torch.full((5,), -0.5, device="cuda"), rtol=2.0 ** -19, atol=0)
    assert not p[:-5].any()


def test_copies_of_some():
    s = make([300, 300], torch.float32, False, torch.float16)
    s["copies"][0] = None
    was = s["params"][1].clone()
    tile.adamw(**s, step=1)
    assert torch.equal(s["copies"][1], s["params"][1].half()) and not torch.equal(was, s["params"][1])


def test_neighbours_are_left_alone():
    for eight in (False, True):
        for shift in (0, 3):
            params, room = views([normal(i, n) for i, n in enumerate(SIZES)], shift)
            grads = [normal(i + 20, n) for i, n in enumerate(SIZES)]
            copies, copy_room = views([p.to(torch.float16) for p in params], shift)
            inside = torch.zeros_like(room, dtype=torch.bool)
            for p in params:
                at = (p.data_ptr() - room.data_ptr()) // 4
                inside[at:at + p.numel()] = True
            tile.adamw(params, grads, **tile.adamw_state(params, 8 if eight else 32), step=1, copies=copies)
            assert (room[~inside] == 7.0).all()
            inside = torch.zeros_like(copy_room, dtype=torch.bool)
            for p in copies:
                at = (p.data_ptr() - copy_room.data_ptr()) // 2
                inside[at:at + p.numel()] = True
            assert (copy_room[~inside] == 7.0).all()


def test_captured_steps():
    """A captured clip and step, replayed: the step counter and the gradients
    change in place."""
    for eight in (False, True):
        sizes = [3000, 129, 64]
        a, b = (make(sizes, torch.bfloat16, eight, torch.bfloat16) for _ in range(2))
        step = torch.ones(1, dtype=torch.int64, device="cuda")
        lr = torch.full((1,), 1e-2, device="cuda")

        def run(s):
            tile.adamw(**s, step=step, lr=lr, factor=tile.grad_norm(s["grads"], 0.5)[1:])
            step.add_(1)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            run(a)
        step.fill_(1)
        for k in range(3):
            for i in range(len(sizes)):
                g = normal(200 + 10 * k + i, sizes[i], torch.bfloat16)
                a["grads"][i].copy_(g), b["grads"][i].copy_(g)
            graph.replay()
        step.fill_(1)
        for k in range(3):
            for i in range(len(sizes)):
                b["grads"][i].copy_(normal(200 + 10 * k + i, sizes[i], torch.bfloat16))
            run(b)
        torch.cuda.synchronize()
        for k in a:
            for x, y in zip(a[k], b[k]):
                assert torch.equal(x.float(), y.float())


def test_streams():
    s = make([4000, 100], torch.float32, False, None)
    t = make([4000, 100], torch.float32, False, None)
    u = make([4000, 100], torch.float32, False, None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for k, stream in ((s, None), (t, side), (u, side.cuda_stream)):
        out = tile.grad_norm(k["grads"], 0.1, stream=stream)
        tile.adamw(**k, step=1, factor=out[1:], stream=stream)
    torch.cuda.synchronize()
    for k in s:
        for x, y, z in zip(s[k], t[k], u[k]):
            assert torch.equal(x, y) and torch.equal(x, z)


# ---- many elements --------------------------------------------------------------------
#
# From 152 x 16 chunks on a CTA takes several steps of the smallest chunk: 2 in FP32 from
# 5e6 elements on, with 8-bit states 2 from 1e7 and 4 from 2e7 on (a warp's second and
# later blocks, whose scales other lanes hold and whose copies lie in used stages).


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", TYPES)
def test_step_of_many_elements(dtype, shift):
    s = make([3000001, 77, 2100003], dtype, False, torch.bfloat16, shift)
    check_step(s, step=3, factor=0.3)


@pytest.mark.parametrize("dtype,total,copy,shift", [
    (torch.float32, 2.1e7, None, 0), (torch.bfloat16, 2.1e7, torch.bfloat16, 0),
    (torch.float16, 2.1e7, torch.float16, 0), (torch.float32, 1.1e7, torch.float16, 0),
    (torch.bfloat16, 1.1e7, None, 0), (torch.bfloat16, 2.1e7, torch.float16, 3)])
def test_eight_bit_step_of_many_elements(dtype, total, copy, shift):
    """Whole blocks, a last one that is cut, and blocks before it that a CTA's last warps have not."""
    sizes = [int(total * 0.7) // 8192 * 8192 + 2048 * 3 + 256 * 2 + 5, 77, int(total * 0.3) // 8192 * 8192 + 8192]
    s = make(sizes, dtype, True, copy, shift)
    check_step(s, step=3, factor=0.3, seed=9)


@pytest.mark.parametrize("eight", [False, True])
def test_an_eps_that_leaves_decay_alone(eight):
    """Above 2^126 the reciprocal is 0; the parameter's factor and product round once each."""
    params, grads = [normal(1, 1000)], [normal(2, 1000)]
    was = params[0].clone()
    tile.adamw(params, grads, **tile.adamw_state(params, 8 if eight else 32), step=1, lr=0.5, weight_decay=0.5, eps=1e38)
    assert ((params[0].double() - was.double() * 0.75).abs() <= 2.0 ** -23 * was.double().abs()).all()
