"""The bounded waits of the block norm's gradients and of the linear cross
entropy, made to run out without a fault: through the test entry points one
program's first row, or one CTA pair's first tiles, are never copied, and waits
give up after 16 ms (64 for a cluster's sums).  The kernels end, the device
status word reports it once, nothing but the call's own outputs is written, and
the next call on the same buffers is right."""

import time

import pytest
import torch

import tile_compiler_row_gb300 as tile
from test_block_norm_gpu import check, make, reference_backward
from test_linear_ce_gpu import check_loss
from test_linear_ce_gpu import make as make_loss

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    from tile_compiler_row_gb300 import _build
    _build.build()
    tile.load()
    torch.cuda.set_device(0)


def reported_once(call):
    torch.cuda.synchronize()
    assert tile.tile_check_device_status() == 0
    start = time.perf_counter()
    call()
    torch.cuda.synchronize()
    assert time.perf_counter() - start < 10.0
    assert tile.tile_check_device_status() == -9     # TILE_ERR_DEVICE, then cleared
    assert tile.tile_check_device_status() == 0


# a row to a program and several, one CTA and clusters of 2 and 8
@pytest.mark.parametrize("rows,width", [(9, 64), (2000, 4096), (100, 1024), (700, 5120), (64, 20000)])
def test_a_row_that_never_comes(rows, width):
    s = make(rows, width, "bf16", rows)
    need = tile.tile_block_norm_backward_gated_workspace_bytes(rows, width, 1)
    ws = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    mats = [torch.full((rows + 3, width), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    vecs = torch.full((5, width), 7.0, device="cuda")
    args = (s["x"], s["residual"], s["dhidden"], s["dout"], mats[0][:rows], mats[1][:rows], ws[:need],
            s["gamma_post"], s["gate"], s["gamma_pre"], vecs[0], vecs[1:2], vecs[2])
    reported_once(lambda: tile.tile_test_block_norm_backward_wait_timeout(*args, rows_per_gate=rows))
    assert (ws[need:] == 77).all() and (vecs[3:] == 7).all()
    assert all((m[rows:] == 7).all() for m in mats)
    tile.tile_block_norm_backward(*args, rows_per_gate=rows)
    ref = reference_backward(s, s["residual"], True, True, rows, 1.0, 1e-5)
    for name, got, n in (("din", mats[0][:rows], 192), ("dresidual", mats[1][:rows], 128),
                         ("dgamma_post", vecs[0], 400), ("dgate", vecs[1:2], 400),
                         ("dgamma_pre", vecs[2], 400)):
        check(got, *ref[name], n, name)
    assert tile.tile_check_device_status() == 0


# one tile to a pair and several; fewer k blocks than stages, and more
@pytest.mark.parametrize("rows,width,vocab", [(5, 64, 300), (5, 2048, 32768), (300, 1024, 1000),
                                              (700, 1001, 9000), (2000, 4096, 40000)])
def test_tiles_that_never_come(rows, width, vocab):
    x, weight, target, _ = make_loss(rows, width, vocab, "bf16", 0.2 if rows > 5 else 0.0)
    need = tile.tile_linear_cross_entropy_workspace_bytes(rows, width, vocab)
    ws = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    losses = torch.full((2, rows + 9), 7.0, device="cuda")
    args = x, weight, target, losses[0, :rows], losses[1, :rows], ws[:need]
    reported_once(lambda: tile.tile_test_linear_cross_entropy_wait_timeout(*args))
    assert (ws[need:] == 77).all() and (losses[:, rows:] == 7).all()
    tile.tile_linear_cross_entropy(*args)
    keep = slice(0, rows, max(1, rows // 100))
    check_loss(x[keep], weight, target[keep], losses[0, :rows][keep], losses[1, :rows][keep])
    assert tile.tile_check_device_status() == 0


def test_forms_that_are_not_built_for_it():
    for rows, width, kind in ((4, 64, "f32"), (4, 65, "bf16"), (4, 8192, "bf16"), (2, 131072, "bf16")):
        s = make(rows, width, kind)
        ws = torch.empty(tile.tile_block_norm_backward_workspace_bytes(rows, width),
                         dtype=torch.uint8, device="cuda")
        out = [torch.empty_like(s["x"]) for _ in range(2)]
        with pytest.raises(tile.TileError) as e:
            tile.tile_test_block_norm_backward_wait_timeout(s["x"], s["residual"], None, s["dout"],
                                                            *out, ws)
        assert e.value.status == -8      # TILE_ERR_PLAN
    for width, kind in ((64, "f16"), (4160, "bf16")):
        x, weight, target, loss = make_loss(4, width, 300, kind)
        ws = torch.empty(tile.tile_linear_cross_entropy_workspace_bytes(4, width, 300),
                         dtype=torch.uint8, device="cuda")
        with pytest.raises(tile.TileError) as e:
            tile.tile_test_linear_cross_entropy_wait_timeout(x, weight, target, loss,
                                                             torch.empty_like(loss), ws)
        assert e.value.status == -8
    assert tile.tile_check_device_status() == 0
