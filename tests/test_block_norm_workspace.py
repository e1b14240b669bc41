"""The workspace of the block norm's gradients: as much as the programs of a
call write, and no more of it than the call's own matrices explain."""

import ctypes

import pytest
import torch

import tile_compiler_row_gb300 as tile

MIB = 1 << 20
CUDA, WORKSPACE = -5, -10


@pytest.fixture(scope="module", autouse=True)
def lib():
    from tile_compiler_row_gb300 import _build
    _build.build()
    return tile.load()


def anyhow(rows, width):
    return tile.tile_block_norm_backward_workspace_bytes(rows, width)


def gated(rows, width, gates):
    return tile.tile_block_norm_backward_gated_workspace_bytes(rows, width, gates)


# (16 bytes a column and program)
@pytest.mark.parametrize("rows,width", [(90, 32768), (128, 131072), (1024, 65536), (2048, 32768),
                                        (4096, 16384), (1 << 20, 8192), (1 << 20, 2048), (5, 4096)])
def test_wide_rows_take_what_runs_at_once(rows, width):
    assert gated(rows, width, 0) == gated(rows, width, rows) == anyhow(rows, width)
    assert 0 < anyhow(rows, width) <= min(rows * 16 * width, 40 * MIB)


@pytest.mark.parametrize("rows,width", [(90, 32769), (2000, 20001), (800, 65535), (128, 131071),
                                        (1 << 20, 4097)])
def test_odd_widths_take_eight_programs_a_gate_row(rows, width):
    most = max(min(rows * 16 * width, 40 * MIB), 8 * 16 * width)
    assert 0 < gated(rows, width, 0) == gated(rows, width, 1) <= most
    for gates in (1, 3, 20, 100, rows):
        assert gated(rows, width, gates) <= max(most, 8 * gates * 16 * width)
        assert gated(rows, width, gates) <= anyhow(rows, width) <= 1024 * 16 * width
    assert gated(rows, width, rows) == anyhow(rows, width)


def test_no_workspace_for_what_a_call_refuses():
    for rows, width, gates in ((0, 64, 0), (-1, 64, 0), (4, 0, 0), (4, 131073, 0), (4, 64, -1),
                               (4, 64, 1 << 32), ((1 << 32) + 4, 64, 0)):
        assert gated(rows, width, gates) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers: CPU-only test")
@pytest.mark.parametrize("rows,width,per", [(90, 32768, 0), (90, 32769, 0), (90, 32769, 30),
                                            (90, 32769, 1), (2000, 200, 0), (2000, 201, 7)])
def test_a_call_checks_for_its_own_gate_rows(lib, rows, width, per):
    a = tile.TileBlockNormBackwardArgs()
    step = 1 << 32     # fake device addresses, never dereferenced
    (a.in_, a.hidden, a.dhidden, a.dout, a.gamma_post, a.gate, a.gamma_pre, a.din, a.dresidual,
     a.dgamma_post, a.dgate, a.dgamma_pre) = (step * (i + 1) for i in range(12))
    if not per:
        a.gate = a.dgate = None
    a.rows, a.width, a.rows_per_gate, a.norms, a.dtype = rows, width, per, 3, 1
    a.residual_scale, a.eps = 1.0, 1e-5
    need = gated(rows, width, -(-rows // per) if per else 0)
    f = lib.tile_block_norm_backward
    assert f(ctypes.byref(a), 13 * step, need - 1, None) == WORKSPACE
    lib.tile_inject_launch_failure(2, 0, 1)
    try:
        assert f(ctypes.byref(a), 13 * step, need, None) == CUDA
    finally:
        lib.tile_inject_launch_failure(2, 0, 0)


# every layout: whole vectors and row classes, clusters, programs of registers
# (rows off 16 bytes, many gate rows, the widest rows); fewer and more rows than
# programs
@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,width,per,offset", [
    (4, 64, 1, 0), (40, 2048, 0, 0), (3000, 4096, 700, 0), (600, 5120, 0, 0), (400, 8192, 11, 0),
    (90, 32768, 0, 0), (90, 32769, 0, 0), (90, 32769, 9, 0), (30, 32769, 1, 0), (300, 20004, 40, 0),
    (5000, 1537, 600, 0), (5000, 63, 3, 0), (20000, 65, 0, 0), (40000, 128, 0, 0), (700, 4097, 4, 0),
    (9, 65537, 0, 0), (64, 131072, 0, 0), (33, 131071, 20, 0), (3, 131071, 1, 0), (500, 512, 70, 1),
    (100, 10000, 0, 3), (40, 70000, 7, 1), (1, 1, 0, 0)])
def test_a_call_keeps_to_the_workspace_it_asks_for(rows, width, per, offset, kind):
    """The bytes behind it stay as they are, and the results are those of a
    call with as much as any number of gate rows needs."""
    from test_block_norm_gpu import TYPES, make
    s = make(rows, width, kind, per, offset=offset)
    gates = -(-rows // per) if per else 0

    def call(nbytes):
        ws = torch.full((nbytes + 4096,), 77, dtype=torch.uint8, device="cuda")
        mats = [torch.empty(rows, width, dtype=TYPES[kind], device="cuda") for _ in range(2)]
        vecs = [torch.empty(width, device="cuda") for _ in range(2)]
        dgate = torch.empty(gates, width, device="cuda") if per else None
        tile.tile_block_norm_backward(s["x"], s["residual"], s["dhidden"], s["dout"], *mats,
                                      ws[:nbytes], s["gamma_post"], s["gate"], s["gamma_pre"],
                                      vecs[0], dgate, vecs[1], rows_per_gate=per)
        assert (ws[nbytes:] == 77).all()
        return mats + vecs + ([dgate] if per else [])
    for a, b in zip(call(gated(rows, width, gates)), call(anyhow(rows, width))):
        assert torch.equal(a, b)
    assert tile.tile_check_device_status() == 0
