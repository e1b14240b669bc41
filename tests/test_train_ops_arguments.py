"""What the binding of the block norm and the linear cross entropy does with
arguments that a C int does not hold, without a GPU: tensors that say they are
on a device stand in for real ones, and the C entry point is recorded instead of
called."""

import pytest
import torch

import tile_compiler_row_gb300 as tile

BIG = 1 << 32


class OnDevice(torch.Tensor):
    """A tensor without memory that says it lies on cuda:<index>."""

    index = 0

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 0x10000000


def on_device(*shape, dtype=torch.float32, index=0):
    t = torch.empty(*shape, dtype=dtype, device="meta").as_subclass(OnDevice)
    t.index = index
    return t


@pytest.fixture
def calls(monkeypatch):
    """The arguments of each call that would reach a C entry point."""
    made = []
    monkeypatch.setattr(tile, "_call_on", lambda dev, stream, name, *args: made.append((name, args)))
    return made


def norm(x, calls, gate=None, per=0, **kw):
    tile.tile_block_norm(x, x, x, x, None, gate, None, rows_per_gate=per, **kw)
    return calls[-1][1][0]._obj


def norm_backward(x, calls, gate=None, per=0, **kw):
    ws = on_device(1 << 20, dtype=torch.uint8)
    tile.tile_block_norm_backward(x, x, x, x, x, x, ws, None, gate, None, dgate=gate,
                                  rows_per_gate=per, **kw)
    return calls[-1][1][0]._obj


@pytest.mark.parametrize("call", [norm, norm_backward])
@pytest.mark.parametrize("per", [9, 10, BIG, BIG + 1, BIG + 4, 1 << 40, (1 << 64) + 1])
def test_one_gate_row_reaches_the_call_as_one(calls, call, per):
    """At least as many rows to a gate as there are rows: one gate row, and the
    kernel may not be told fewer."""
    args = call(on_device(9, 64), calls, on_device(1, 64), per)
    assert args.rows_per_gate >= 9
    # its shape is checked by the same number
    with pytest.raises(ValueError):
        call(on_device(9, 64), calls, on_device(2, 64), per)


@pytest.mark.parametrize("call", [norm, norm_backward])
def test_rows_per_gate_as_given(calls, call):
    for per, gates in ((1, 9), (4, 3), (8, 2)):
        assert call(on_device(9, 64), calls, on_device(gates, 64), per).rows_per_gate == per
    assert call(on_device(9, 64), calls, on_device(64), 0).rows_per_gate >= 9
    for per in (-1, 1 - BIG, -BIG):
        with pytest.raises(ValueError):
            call(on_device(9, 64), calls, on_device(1, 64), per)
    assert len(calls) == 4


@pytest.mark.parametrize("call", [norm, norm_backward])
@pytest.mark.parametrize("shape", [(BIG + 1, 8), (1 << 31, 8), (1, BIG + 64), (BIG, 1 << 20)])
def test_block_norm_sizes_past_an_int(calls, call, shape):
    with pytest.raises(ValueError):
        call(on_device(*shape, dtype=torch.bfloat16), calls)
    assert not calls


def loss(rows, width, vocab, ignore=-100):
    bf = torch.bfloat16
    f = on_device(rows)
    tile.tile_linear_cross_entropy(on_device(rows, width, dtype=bf), on_device(vocab, width, dtype=bf),
                                   on_device(rows, dtype=torch.int64), f, f,
                                   on_device(64, dtype=torch.uint8), ignore_index=ignore)


def loss_backward(rows, width, vocab, ignore=-100):
    bf = torch.bfloat16
    f, x, w = on_device(rows), on_device(rows, width, dtype=bf), on_device(vocab, width, dtype=bf)
    tile.tile_linear_cross_entropy_backward(x, w, on_device(rows, dtype=torch.int64), f, f, x, w,
                                            on_device(64, dtype=torch.uint8), ignore_index=ignore)


@pytest.mark.parametrize("call", [loss, loss_backward])
def test_linear_ce_sizes_past_an_int(calls, call):
    call(4, 64, 300)
    assert len(calls) == 1
    for sizes in ((BIG + 4, 64, 300), (1 << 31, 64, 300), (4, BIG + 64, 300), (4, 64, BIG + 300),
                  (4, 64, 1 << 31)):
        with pytest.raises(ValueError):
            call(*sizes)
    assert len(calls) == 1


@pytest.mark.parametrize("call", [loss, loss_backward])
def test_ignore_index_past_64_bits(calls, call):
    """No 64-bit target equals it; its low 64 bits may not stand for it."""
    for ignore in (-100, (1 << 63) - 1, -1 << 63):
        call(4, 64, 300, ignore)
    for ignore in ((1 << 64) - 100, 1 << 63, (-1 << 63) - 1):
        with pytest.raises(ValueError):
            call(4, 64, 300, ignore)
    assert len(calls) == 3


def test_no_workspace_for_sizes_past_an_int():
    """0 bytes, as for other sizes that a call refuses."""
    from tile_compiler_row_gb300 import _build
    _build.build()
    assert tile.tile_block_norm_backward_workspace_bytes(BIG + 4, 64) == 0
    assert tile.tile_block_norm_backward_workspace_bytes(4, BIG + 64) == 0
    for f in (tile.tile_linear_cross_entropy_workspace_bytes,
              tile.tile_linear_cross_entropy_backward_workspace_bytes):
        assert f(4, 64, 300) > 0
        for sizes in ((BIG + 4, 64, 300), (4, BIG + 64, 300), (4, 64, BIG + 300), (4 - BIG, 64, 300)):
            assert f(*sizes) == 0


def test_gradients_of_nothing_are_refused():
    """Neither the hidden rows nor a gradient of them: no shape to go by."""
    x, g = torch.zeros(2, 8), torch.zeros(8)
    for pre in (True, False):
        with pytest.raises(ValueError, match="hidden"):
            tile.block_norm_backward(x, None, g, None, g, None, x, pre=pre)
