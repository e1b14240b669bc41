"""Host-only checks of the block norm's and the linear cross entropy's entry
points: bad arguments are refused before any CUDA call, and the binding
refuses tensors it cannot pass on."""

import ctypes

import pytest

import tile_compiler_row_gb300 as tile
from tile_compiler_row_gb300 import _build

OK, NULL, SHAPE, ALIAS, EPS, OP, ALIGN, WORKSPACE, DTYPE = 0, -1, -2, -3, -4, -6, -7, -10, -11


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return tile.load()


def _no_gpu():
    try:
        import torch
        return not torch.cuda.is_available()
    except Exception:
        return True


fake_pointers = pytest.mark.skipif(not _no_gpu(), reason="fake device pointers: CPU-only test")

# fake device addresses, 16 MiB apart, never dereferenced
A, B, C, D, E, F, G, H, I, J, K, L = (0x10000000 + 0x1000000 * i for i in range(12))


def forward_args(**kw):
    a = tile.TileBlockNormArgs()
    a.in_, a.residual, a.gamma_post, a.gate, a.gamma_pre, a.hidden, a.out = A, B, C, D, E, F, G
    a.rows, a.width, a.rows_per_gate, a.norms = 4, 64, 2, 3
    a.residual_scale, a.eps, a.dtype = 1.0, 1e-5, 1
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def backward_args(**kw):
    a = tile.TileBlockNormBackwardArgs()
    a.in_, a.hidden, a.dhidden, a.dout, a.gamma_post, a.gate, a.gamma_pre = A, B, C, D, E, F, G
    a.din, a.dresidual, a.dgamma_post, a.dgate, a.dgamma_pre = H, I, J, J + 65536, J + 2 * 65536
    a.rows, a.width, a.rows_per_gate, a.norms = 4, 64, 2, 3
    a.residual_scale, a.eps, a.dtype = 1.0, 1e-5, 1
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@fake_pointers
@pytest.mark.parametrize("change,status", [
    ({"in_": None}, NULL), ({"residual": None}, NULL), ({"hidden": None}, NULL),
    ({"out": None}, NULL), ({"rows": -1}, SHAPE), ({"width": 0}, SHAPE),
    ({"width": 131073}, SHAPE), ({"rows_per_gate": 0}, SHAPE), ({"norms": 0}, OP),
    ({"norms": 4}, OP), ({"dtype": 3}, DTYPE), ({"eps": -1.0}, EPS), ({"eps": float("nan")}, EPS),
    ({"residual_scale": float("inf")}, EPS), ({"in_": A + 1}, ALIGN), ({"gate": D + 2}, ALIGN),
    ({"hidden": A}, ALIAS), ({"out": B + 128}, ALIAS), ({"out": F}, ALIAS),
    ({"hidden": D + 256}, ALIAS), ({"rows": 0, "in_": None, "hidden": None}, OK)])
def test_block_norm_refusals(lib, change, status):
    assert lib.tile_block_norm(ctypes.byref(forward_args(**change)), None) == status


@fake_pointers
def test_block_norm_gate_extent(lib):
    """The gate's last row counts for the overlap check."""
    a = forward_args(rows=9, rows_per_gate=4, hidden=D + 2 * 256)     # gate rows 0..2
    assert lib.tile_block_norm(ctypes.byref(a), None) == ALIAS
    assert lib.tile_block_norm(None, None) == NULL


@fake_pointers
@pytest.mark.parametrize("change,status", [
    ({"in_": None}, NULL), ({"hidden": None}, NULL), ({"dout": None}, NULL), ({"din": None}, NULL),
    ({"dresidual": None}, NULL), ({"norms": 1, "dgamma_pre": None, "dhidden": None}, NULL),
    ({"norms": 1}, OP), ({"norms": 2}, OP), ({"gate": None}, OP), ({"rows": -1}, SHAPE),
    ({"width": 0}, SHAPE), ({"rows_per_gate": 0}, SHAPE), ({"dtype": -1}, DTYPE),
    ({"eps": float("inf")}, EPS), ({"din": H + 1}, ALIGN), ({"dgate": J + 2}, ALIGN),
    ({"din": A}, ALIAS), ({"dresidual": H + 64}, ALIAS), ({"dgate": J}, ALIAS),
    ({"dgamma_pre": L}, ALIAS), ({"din": D + 32}, ALIAS)])
def test_block_norm_backward_refusals(lib, change, status):
    need = tile.tile_block_norm_backward_workspace_bytes(4, 64)
    a = backward_args(**change)
    assert lib.tile_block_norm_backward(ctypes.byref(a), L, need, None) == status


@fake_pointers
def test_block_norm_backward_workspace(lib):
    need = tile.tile_block_norm_backward_workspace_bytes(4, 64)
    a = backward_args()
    f = lib.tile_block_norm_backward
    assert f(ctypes.byref(a), L, need - 1, None) == WORKSPACE
    assert f(ctypes.byref(a), None, need, None) == NULL
    assert f(ctypes.byref(a), L + 8, need, None) == ALIGN
    assert f(None, L, need, None) == NULL
    assert tile.tile_block_norm_backward_workspace_bytes(0, 64) == 0
    assert tile.tile_block_norm_backward_workspace_bytes(4, 131073) == 0
    # bounded in the rows
    w = tile.tile_block_norm_backward_workspace_bytes
    assert w(1 << 20, 4096) == w(1 << 30, 4096)


def ce(lib, need=None, **kw):
    a = dict(dtype=1, x=A, w=B, t=C, loss=D, lse=E, rows=4, width=64, vocab=300, ignore=-100, ws=F)
    a.update(kw)
    if need is None:
        need = 1 << 24
    return lib.tile_linear_cross_entropy(a["dtype"], a["x"], a["w"], a["t"], a["loss"], a["lse"],
                                         a["rows"], a["width"], a["vocab"], a["ignore"], a["ws"],
                                         need, None)


def ce_backward(lib, need=None, **kw):
    a = dict(dtype=1, x=A, w=B, t=C, lse=D, dl=E, dx=F, dw=G, rows=4, width=64, vocab=300,
             ignore=-100, ws=H)
    a.update(kw)
    if need is None:
        need = 1 << 24
    return lib.tile_linear_cross_entropy_backward(
        a["dtype"], a["x"], a["w"], a["t"], a["lse"], a["dl"], a["dx"], a["dw"], a["rows"],
        a["width"], a["vocab"], a["ignore"], a["ws"], need, None)


@fake_pointers
@pytest.mark.parametrize("change,status", [
    ({"dtype": 0}, DTYPE), ({"dtype": 5}, DTYPE), ({"rows": -1}, SHAPE), ({"width": 0}, SHAPE),
    ({"width": 131073}, SHAPE), ({"vocab": 0}, SHAPE), ({"vocab": (1 << 30) + 1}, SHAPE),
    ({"x": None}, NULL), ({"w": None}, NULL), ({"t": None}, NULL), ({"ws": None}, NULL),
    ({"x": A + 2}, ALIGN), ({"w": B + 8}, ALIGN), ({"width": 65, "x": A + 1}, ALIGN),
    ({"t": C + 4}, ALIGN), ({"ws": H + 128}, ALIGN)])
def test_linear_ce_refusals(lib, change, status):
    assert ce(lib, **change) == status
    assert ce_backward(lib, **change) == status


@fake_pointers
def test_linear_ce_more_refusals(lib):
    assert ce(lib, rows=0, x=None, ws=None) == OK
    assert ce(lib, loss=None) == NULL and ce(lib, lse=None) == NULL
    assert ce(lib, loss=A) == ALIAS and ce(lib, loss=E) == ALIAS and ce(lib, ws=B) == ALIAS
    need = tile.tile_linear_cross_entropy_workspace_bytes(4, 64, 300)
    assert need > 0 and ce(lib, need=need - 1) == WORKSPACE
    assert ce_backward(lib, lse=None) == NULL and ce_backward(lib, dl=None) == NULL
    assert ce_backward(lib, dx=None, dw=None) == NULL
    assert ce_backward(lib, dx=F + 1) == ALIGN and ce_backward(lib, dw=G + 1) == ALIGN
    assert ce_backward(lib, dx=A) == ALIAS and ce_backward(lib, dw=F + 2) == ALIAS
    assert ce_backward(lib, ws=G) == ALIAS
    need = tile.tile_linear_cross_entropy_backward_workspace_bytes(4, 64, 300)
    assert need > 0 and ce_backward(lib, need=need - 1) == WORKSPACE
    for f in (tile.tile_linear_cross_entropy_workspace_bytes,
              tile.tile_linear_cross_entropy_backward_workspace_bytes):
        assert f(0, 64, 300) == 0 and f(4, 0, 300) == 0 and f(4, 64, 0) == 0


def test_linear_ce_workspace_grows_with_the_call(lib):
    f = tile.tile_linear_cross_entropy_backward_workspace_bytes
    assert f(4096, 4096, 131072) < 2 << 30        # the logits alone would be 1 GiB in 16 bits
    assert f(65536, 4096, 131072) < 4 << 30       # ... and 16 GiB here
    assert f(64, 65, 1000) > f(64, 64, 1000)      # a copy of the weight in whole vectors


def test_binding_refuses_what_it_cannot_pass():
    import torch
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        tile.block_norm(x, x)
    with pytest.raises(ValueError):
        tile.linear_cross_entropy(x.bfloat16(), x.bfloat16(), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        tile.tile_linear_cross_entropy(x, x, x, x, x, x)
