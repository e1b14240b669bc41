"""The gradients of the block norm for rows far from 1, and for an eps that
does not hold small rows up, against FP64.

The tolerances are those of rows of about 1: every scalar of a row is a
product of the same few factors, whatever their size, so it carries the same
roundings as long as no factor on the way leaves FP32's range.  None does
here: hidden rows have a root mean square R of 3.3 times `stream` (3 from the
residual, about 1 from the gated block), x of 1.5 times `block`, so sums of
20000 squares are below 2e4 (1e17)^2 = 2e38 (the widest rows stop at a third
of that stream: 7e4 (3.3e16)^2 = 8e37) and above (1e-16)^2 = 1e-32, and no
gradient is below 1 / R^2 = 1e-34 times 1e-3, 16 bits above FP32's least
value.  The row sum of gate x hidden, 2.5 block stream^2 where the gate is as
large as the stream and 5 block stream where not, has to stay in range as well:
the gate is left at 1 for large blocks, and small ones are chosen so that the
sum is above 1e-34."""

import pytest
import torch

import tile_compiler_row_gb300 as tile
from test_block_norm_gpu import check, make, reference, reference_backward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    from tile_compiler_row_gb300 import _build
    _build.build()
    tile.load()
    torch.cuda.set_device(0)


# the ring kernel (whole vectors, row classes, clusters) and the one for rows
# that it does not take
LAYOUTS = [(9, 4096, 0), (20, 1537, 0), (6, 20000, 0), (33, 512, 1), (3, 70001, 0)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows,width,offset", LAYOUTS)
@pytest.mark.parametrize("eps,block,stream", [
    (1e-5, 1.0, 1e14), (1e-5, 1.0, 1e15), (1e-5, 1.0, 3e16), (1e-5, 1e15, 1.0), (1e-5, 3e16, 1.0),
    (1e-5, 3e16, 3e16), (1e-30, 1.0, 1e-13), (0.0, 1.0, 1e-13), (0.0, 1e-13, 1.0),
    (0.0, 1e-8, 1e-13), (1e-30, 1e-10, 1e-12)])
def test_rows_far_from_one(rows, width, offset, kind, eps, block, stream):
    if width > 20000:
        stream = min(stream, 1e16)
    s = make(rows, width, kind, rows, offset=offset)
    s["x"].mul_(block)
    s["residual"].mul_(stream)
    if block <= 1:   # the block's part of the stream as large as the stream
        s["gate"].mul_(stream)
    args = s["gamma_post"], s["gate"], s["gamma_pre"]
    hidden, out = tile.block_norm(s["x"], s["residual"], *args, rows_per_gate=rows, eps=eps)
    h, hm, y, ym = reference(s, True, True, rows, 1.0, eps)
    check(hidden, h, hm, 64, "hidden")
    check(out, y, ym, 128, "out")
    got = tile.block_norm_backward(s["x"], hidden, *args, None, s["dout"], rows_per_gate=rows,
                                   eps=eps)
    ref = reference_backward(s, hidden, True, True, rows, 1.0, eps, use_dhidden=False)
    for name, g, n in zip(("din", "dresidual", "dgamma_post", "dgate", "dgamma_pre"), got,
                          (192, 128, 400, 400, 400)):
        check(g, *ref[name], n, name)


def test_the_projection_is_there():
    """din is orthogonal to x and dresidual to hidden but for eps: what the
    projection term is for.  Without it each is along them by a share of
    1 / sqrt(width) and more."""
    s = make(16, 256, "f32")
    s["x"].mul_(1e15)
    s["residual"].mul_(1e16)
    s["dout"].copy_(s["residual"] * 1e-16)
    hidden, _ = tile.block_norm(s["x"], s["residual"], s["gamma_post"], None, s["gamma_pre"])
    din, dresidual = tile.block_norm_backward(s["x"], hidden, s["gamma_post"], None, s["gamma_pre"],
                                              None, s["dout"])[:2]
    for v, g in ((s["x"], din), (hidden, dresidual)):
        v, g = v.double(), g.double()
        along = (v * g).sum(1).abs() / (v.norm(dim=1) * g.norm(dim=1))
        assert (along <= 1e-4).all()
