"""The stream that the block norm's and the linear cross entropy's calls run on
when it belongs to another device than the current one, without a GPU: tensors
and streams that say which device they are on stand in for real ones."""

import contextlib
import types

import pytest
import torch

import tile_compiler_row_gb300 as tile


class OnDevice(torch.Tensor):
    """A tensor without memory that says it lies on cuda:<index>."""

    index = 0

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.index


def on_device(index, *shape):
    t = torch.empty(*shape, dtype=torch.bfloat16, device="meta").as_subclass(OnDevice)
    t.index = index
    return t


def torch_stream(index, handle=0x5000):
    return types.SimpleNamespace(device=torch.device("cuda", index), cuda_stream=handle)


@pytest.fixture
def current(monkeypatch):
    """The stack of current streams; an integer handle becomes a stream of
    the device it is given, or of the current one (0)."""
    stack = []

    def external(handle, device=None):
        index = 0 if device is None else torch.device("cuda", device).index \
            if isinstance(device, int) else torch.device(device).index
        return torch_stream(index, handle)

    @contextlib.contextmanager
    def stream(s):
        stack.append(s)
        yield
        stack.pop()
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    return stack


# every wrapper that allocates, with tensors of one device (the first argument
# of the block norm's gradients may be None)
def calls(index):
    x, w = on_device(index, 4, 64), on_device(index, 300, 64)
    return [("block_norm", (x, x), {}),
            ("block_norm", (), {"x": x, "residual": x}),
            ("block_norm_backward", (None, x, None, None, None, None, x), {"post": False}),
            ("linear_cross_entropy", (x, w, x), {}),
            ("linear_cross_entropy_backward", (x, w, x, x, x), {})]


@pytest.mark.parametrize("index", [0, 1, 3])
@pytest.mark.parametrize("which", range(5))
def test_a_handle_is_one_of_the_tensors_device(current, index, which):
    name, args, kwargs = calls(index)[which]
    seen = []
    wrapped = tile._on_stream(lambda *a, **k: seen.append(current[-1]))
    assert hasattr(getattr(tile, name), "__wrapped__")       # the same wrapper
    wrapped(*args, stream=0x7700, **kwargs)
    assert len(seen) == 1 and not current
    assert seen[0].cuda_stream == 0x7700 and seen[0].device.index == index


@pytest.mark.parametrize("which", range(5))
def test_a_stream_of_another_device_is_refused(current, which):
    name, args, kwargs = calls(1)[which]
    with pytest.raises(ValueError, match="stream"):
        getattr(tile, name)(*args, stream=torch_stream(0), **kwargs)
    assert not current
    seen = []
    tile._on_stream(lambda *a, **k: seen.append(current[-1]))(*args, stream=torch_stream(1), **kwargs)
    assert seen[0].device.index == 1


def test_calls_below_take_the_stream_they_are_given(monkeypatch):
    """With the tensors' device current, an integer as it is, a stream's
    handle, and no stream of another device."""
    made, devices = [], []

    @contextlib.contextmanager
    def device(index):
        devices.append(index)
        yield
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(tile, "load", lambda: types.SimpleNamespace(
        entry=lambda *a: made.append(a) or 0))
    for dev in (0, 1):
        tile._call_on(dev, 0x7700, "entry", 5)
        tile._call_on(dev, torch_stream(dev), "entry", 5)
        with pytest.raises(ValueError, match="stream"):
            tile._call_on(dev, torch_stream(1 - dev), "entry", 5)
    assert made == [(5, 0x7700), (5, 0x5000)] * 2 and devices.count(0) == 0


def test_tensors_off_the_gpu_are_refused_with_a_stream():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        tile.block_norm(x, x, stream=0x7700)


@pytest.mark.gpu
def test_a_stream_and_its_handle_give_the_same():
    from tile_compiler_row_gb300 import _build
    _build.build()
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, w = (torch.randn(n, 128, device="cuda", generator=gen).bfloat16() for n in (40, 500))
    target = torch.randint(500, (40,), device="cuda", generator=gen)
    side = torch.cuda.Stream()

    def step(stream):
        side.wait_stream(torch.cuda.current_stream())
        hidden, y = tile.block_norm(x, x, stream=stream)
        loss, lse = tile.linear_cross_entropy(y, w, target, stream=stream)
        dy, dw = tile.linear_cross_entropy_backward(y, w, target, lse, lse, stream=stream)
        din = tile.block_norm_backward(x, hidden, None, None, None, None, dy, stream=stream)[0]
        torch.cuda.synchronize()
        return hidden, y, loss, lse, dy, dw, din
    for a, b, c in zip(step(None), step(side), step(side.cuda_stream)):
        assert torch.equal(a, b) and torch.equal(a, c)
