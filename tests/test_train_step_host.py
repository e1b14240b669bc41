"""Host-only checks of the embedding, the policy loss, the gradient norm and the
AdamW step: bad arguments are refused before any CUDA call, and the binding
refuses tensors it cannot pass on."""

import ctypes
import math
import struct
import types

import pytest
import torch

import tile_compiler_row_gb300 as tile
from tile_compiler_row_gb300 import _build

OK, NULL, SHAPE, ALIAS, EPS, OP, ALIGN, WORKSPACE, DTYPE = 0, -1, -2, -3, -4, -6, -7, -10, -11
BIG = 1 << 32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return tile.load()


fake_pointers = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers: CPU-only test")

# fake device addresses, 16 MiB apart, never dereferenced
A, B, C, D, E, F, G, H, I, J = (0x10000000 + 0x1000000 * i for i in range(10))


def embed(lib, **kw):
    a = dict(dtype=1, tokens=A, weight=B, out=C, rows=4, width=64, vocab=300, scale=1.0, ignore=-100)
    a.update(kw)
    return lib.tile_embedding(*a.values(), None)


@fake_pointers
@pytest.mark.parametrize("change,status", [
    ({"dtype": 3}, DTYPE), ({"tokens": None}, NULL), ({"weight": None}, NULL), ({"out": None}, NULL),
    ({"rows": -1}, SHAPE), ({"rows": (1 << 24) + 1}, SHAPE), ({"width": 0}, SHAPE),
    ({"width": 131073}, SHAPE), ({"vocab": 0}, SHAPE), ({"vocab": (1 << 30) + 1}, SHAPE),
    ({"scale": INF}, EPS), ({"scale": NAN}, EPS), ({"tokens": A + 4}, ALIGN), ({"weight": B + 1}, ALIGN),
    ({"dtype": 0, "out": C + 2}, ALIGN), ({"out": B}, ALIAS), ({"out": B + 300 * 128 - 2}, ALIAS),
    ({"out": A - 4 * 128 + 2}, ALIAS), ({"rows": 0, "out": None}, OK)])
def test_embedding_refusals(lib, change, status):
    assert embed(lib, **change) == status


def embed_backward(lib, nbytes=1 << 22, **kw):
    a = dict(dtype=1, into=1, tokens=A, dout=B, dweight=C, rows=3000, width=64, vocab=300, scale=1.0,
             ignore=-100, add=0, ws=D)
    a.update(kw)
    return lib.tile_embedding_backward(*a.values(), nbytes, None)


@fake_pointers
@pytest.mark.parametrize("change,status", [
    ({"dtype": -1}, DTYPE), ({"into": 2}, DTYPE), ({"dtype": 0, "into": 1}, DTYPE), ({"tokens": None}, NULL),
    ({"dout": None}, NULL), ({"dweight": None}, NULL), ({"ws": None}, NULL), ({"rows": -1}, SHAPE),
    ({"rows": (1 << 24) + 1}, SHAPE), ({"width": 0}, SHAPE), ({"vocab": 0}, SHAPE), ({"scale": INF}, EPS),
    ({"tokens": A + 4}, ALIGN), ({"dout": B + 1}, ALIGN), ({"into": 0, "dweight": C + 2}, ALIGN),
    ({"ws": D + 128}, ALIGN), ({"nbytes": 1000}, WORKSPACE), ({"dweight": B}, ALIAS),
    ({"ws": B}, ALIAS), ({"ws": C}, ALIAS), ({"dweight": A}, ALIAS), ({"rows": 0, "add": 1}, OK)])
def test_embedding_backward_refusals(lib, change, status):
    assert embed_backward(lib, **change) == status


def test_embedding_workspace(lib):
    w = tile.tile_embedding_backward_workspace_bytes
    assert w(1, 64, 300) == 0 and w(0, 64, 300) == 0 and w(-1, 64, 300) == 0
    assert w(3000, 64, 300) > 3000 * 16
    assert w(1 << 24, 4096, 1 << 30) > 0 and w((1 << 24) + 1, 64, 300) == 0
    for sizes in ((BIG + 4, 64, 300), (4000, BIG + 64, 300), (4000, 64, BIG + 300)):
        assert w(*sizes) == 0


def policy_args(**kw):
    a = tile.TilePolicyLossArgs()
    a.nll, a.old_nll, a.ref_nll, a.advantage, a.target, a.offsets = A, B, C, D, E, F
    a.ignore_index, a.rows, a.sequences, a.flags = -100, 1000, 10, 0
    a.clip_low, a.clip_high, a.kl_coef = 0.2, 0.2, 0.1
    for k, v in kw.items():
        setattr(a, k, v)
    return a


POLICY = [({"nll": None}, NULL), ({"old_nll": None}, NULL), ({"advantage": None}, NULL),
          ({"ref_nll": None}, NULL), ({"rows": -1}, SHAPE), ({"rows": (1 << 30) + 1}, SHAPE),
          ({"sequences": 0}, SHAPE), ({"offsets": None}, SHAPE), ({"flags": 4}, OP), ({"flags": -1}, OP),
          ({"clip_low": -0.1}, EPS), ({"clip_low": 1.1}, EPS), ({"clip_low": NAN}, EPS),
          ({"clip_high": -0.1}, EPS), ({"clip_high": NAN}, EPS), ({"kl_coef": INF}, EPS),
          ({"nll": A + 2}, ALIGN), ({"advantage": D + 1}, ALIGN), ({"target": E + 4}, ALIGN),
          ({"offsets": F + 4}, ALIGN)]


@fake_pointers
@pytest.mark.parametrize("change,status", POLICY)
def test_policy_refusals(lib, change, status):
    a = policy_args(**change)
    assert lib.tile_policy_loss(ctypes.byref(a), G, H, I, 1 << 20, None) == status
    assert lib.tile_policy_loss_backward(ctypes.byref(a), G, H, I, None) == status


@fake_pointers
def test_policy_outputs(lib):
    a = ctypes.byref(policy_args())
    need = tile.tile_policy_loss_workspace_bytes(1000, 10)
    f, g = lib.tile_policy_loss, lib.tile_policy_loss_backward
    assert f(None, G, H, I, need, None) == NULL and g(None, G, H, I, None) == NULL
    assert f(a, None, H, I, need, None) == NULL and f(a, G, None, I, need, None) == NULL
    assert f(a, G, H, None, need, None) == NULL and f(a, G, H, I, need - 1, None) == WORKSPACE
    assert f(a, G + 2, H, I, need, None) == ALIGN and f(a, G, H, I + 8, need, None) == ALIGN
    assert f(a, A, H, I, need, None) == ALIAS and f(a, G, F, I, need, None) == ALIAS
    assert f(a, G, G + 12, I, need, None) == ALIAS and f(a, G, H, D, need, None) == ALIAS
    assert g(a, None, H, I, None) == NULL and g(a, G, H, None, None) == NULL
    assert g(a, G, H + 2, I, None) == ALIGN and g(a, G, H, A, None) == ALIAS
    assert g(a, G, H, G, None) == ALIAS and g(a, G, I, I, None) == ALIAS
    empty = ctypes.byref(policy_args(rows=0))
    assert g(empty, None, None, None, None) == OK
    w = tile.tile_policy_loss_workspace_bytes
    assert w(0, 1) == 0 and w(5, 0) == 0 and w(BIG + 5, 1) == 0 and w(5, BIG + 1) == 0 and w(1, 1) > 0


def norm(lib, rows=((B, 100, 1), (C, 0, 0), (D, 7, 0)), nbytes=1 << 20, **kw):
    data = b"".join(struct.pack("2qi4x", p or 0, n, t) for p, n, t in rows)
    a = dict(table=data, count=len(rows), scale=1.0, most=1.0, out=A, ws=E)
    a.update(kw)
    return lib.tile_grad_norm(*a.values(), nbytes, None)


@fake_pointers
@pytest.mark.parametrize("change,status", [
    ({"count": -1}, SHAPE), ({"table": None}, NULL), ({"out": None}, NULL), ({"ws": None}, NULL),
    ({"scale": 0.0}, EPS), ({"scale": -1.0}, EPS), ({"scale": INF}, EPS), ({"most": 0.0}, EPS),
    ({"most": NAN}, EPS), ({"out": A + 2}, ALIGN), ({"ws": E + 8}, ALIGN), ({"nbytes": 100}, WORKSPACE),
    ({"out": B}, ALIAS), ({"ws": D}, ALIAS), ({"out": E}, ALIAS)])
def test_norm_refusals(lib, change, status):
    assert norm(lib, **change) == status


@fake_pointers
@pytest.mark.parametrize("row,status", [((None, 5, 0), NULL), ((B, -1, 0), SHAPE), ((B, 1 << 41, 0), SHAPE),
                                        ((B, 5, 3), DTYPE), ((B + 2, 5, 0), ALIGN), ((B + 1, 5, 2), ALIGN)])
def test_norm_tensor_refusals(lib, row, status):
    assert norm(lib, rows=((C, 8, 0), row)) == status


FIELDS = dict(param=A, grad=B, m=C, v=D, ms=0, vs=0, copy=0, n=1000, decay=0.1, grad_type=1, copy_type=0)


def adamw(lib, rows=({},), config=None, **kw):
    data = b"".join(struct.pack("8qf2i4x", *{**FIELDS, **r}.values()) for r in rows)
    c = tile.TileAdamwConfig(1e-3, 0.9, 0.99, 1e-8, 1, None, None, None, 0, 0)
    for k, v in (config or {}).items():
        setattr(c, k, v)
    a = dict(table=data, count=len(rows))
    a.update(kw)
    return lib.tile_adamw(a["table"], a["count"], ctypes.byref(c), None)


EIGHT = dict(ms=E, vs=F)


@fake_pointers
@pytest.mark.parametrize("row,status", [
    ({"param": 0}, NULL), ({"grad": 0}, NULL), ({"m": 0}, NULL), ({"v": 0}, NULL), ({"n": -1}, SHAPE),
    ({"n": 1 << 41}, SHAPE), ({"decay": INF}, EPS), ({"grad_type": 3}, DTYPE),
    ({"copy": G, "copy_type": 0}, DTYPE), ({"copy": G, "copy_type": 3}, DTYPE), ({"param": A + 2}, ALIGN),
    ({"grad": B + 1}, ALIGN), ({"m": C + 1}, ALIGN), ({"copy": G + 1, "copy_type": 1}, ALIGN),
    ({"grad": A}, ALIAS), ({"m": A + 3996}, ALIAS), ({"v": C}, ALIAS), ({"copy": B + 1998, "copy_type": 1}, ALIAS),
    ({"copy": A - 1998, "copy_type": 2}, ALIAS)])
def test_adamw_tensor_refusals(lib, row, status):
    other = dict(param=H, grad=I, m=J, v=J + 65536, n=5)
    assert adamw(lib, (row, other)) == status
    assert adamw(lib, (other, row)) == status


@fake_pointers
def test_adamw_tensors_are_listed_once(lib):
    assert adamw(lib, ({}, {})) == ALIAS
    half = dict(param=A + 2000, grad=G, m=H, v=I, n=5)
    assert adamw(lib, ({}, half)) == ALIAS
    # a gradient may be shared: it is only read
    assert adamw(lib, ({}, dict(param=G, grad=B, m=H, v=I, n=5), dict(n=-1))) == SHAPE
    assert adamw(lib, ({"n": 0, "param": 0, "grad": 0, "m": 0, "v": 0},)) == OK and adamw(lib, ()) == OK


@fake_pointers
@pytest.mark.parametrize("row,status", [
    ({"ms": 0}, NULL), ({"vs": 0}, NULL), ({"ms": E + 2}, ALIGN), ({"vs": E}, ALIAS), ({"ms": C + 996}, ALIAS),
    ({"vs": E + 12}, ALIAS), ({"m": C + 1, "ms": A}, ALIAS)])
def test_adamw_eight_bit_refusals(lib, row, status):
    assert adamw(lib, ({**EIGHT, **row},), {"state": 1}) == status


@fake_pointers
@pytest.mark.parametrize("config,status", [
    ({"beta1": 1.0}, EPS), ({"beta1": -0.1}, EPS), ({"beta2": 1.0}, EPS), ({"beta2": NAN}, EPS),
    ({"eps": 0.0}, EPS), ({"eps": 1e-39}, EPS), ({"eps": INF}, EPS), ({"lr": INF}, EPS), ({"lr": 1e40}, EPS),
    ({"step": 0}, SHAPE), ({"step": -5}, SHAPE), ({"state": 2}, OP), ({"lr_device": G + 2}, ALIGN),
    ({"step_device": G + 4}, ALIGN), ({"factor": G + 1}, ALIGN), ({"factor": A}, ALIAS),
    ({"step_device": D + 8}, ALIAS)])
def test_adamw_config_refusals(lib, config, status):
    assert adamw(lib, config=config) == status
    assert adamw(lib, table=None) == NULL and adamw(lib, count=-1) == SHAPE
    assert lib.tile_adamw(b"", 0, None, None) == NULL


def test_injected_failure(lib):
    """The launch fails on the host: nothing reaches a GPU."""
    if torch.cuda.is_available():
        pytest.skip("fake device pointers: CPU-only test")
    calls = [lambda: embed(lib), lambda: embed_backward(lib),
             lambda: lib.tile_policy_loss(ctypes.byref(policy_args()), G, H, I, 1 << 20, None),
             lambda: lib.tile_policy_loss_backward(ctypes.byref(policy_args()), G, H, I, None),
             lambda: norm(lib), lambda: adamw(lib), lambda: adamw(lib, (EIGHT,), {"state": 1})]
    for call in calls:
        lib.tile_inject_launch_failure(700, 0, 1)
        assert call() == -5 and tile.tile_last_cuda_error() == 700
        lib.tile_inject_launch_failure(0, 0, 0)


# ---- the binding ------------------------------------------------------------------


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
    made = []
    monkeypatch.setattr(tile, "_call_on", lambda dev, stream, name, *args: made.append((name, args)))
    return made


def test_embedding_tensors(calls):
    i64, bf = torch.int64, torch.bfloat16
    t, w, o = on_device(4, dtype=i64), on_device(300, 64, dtype=bf), on_device(4, 64, dtype=bf)
    tile.tile_embedding(t, w, o)
    assert len(calls) == 1
    for args in ((on_device(4, dtype=torch.int32), w, o), (on_device(2, 2, dtype=i64), w, o),
                 (t, on_device(300, 64, dtype=torch.float64), o), (t, on_device(300, dtype=bf), o),
                 (t, w, on_device(4, 64)), (t, w, on_device(5, 64, dtype=bf)), (torch.zeros(4, dtype=i64), w, o),
                 (on_device(4, dtype=i64, index=1), w, o), (t, on_device(64, 300, dtype=bf).t(), o),
                 (on_device(BIG, dtype=i64), w, on_device(BIG, 64, dtype=bf))):
        with pytest.raises(ValueError):
            tile.tile_embedding(*args)
    for ignore in (1 << 63, (1 << 64) - 100):
        with pytest.raises(ValueError):
            tile.tile_embedding(t, w, o, ignore_index=ignore)
    ws = on_device(1 << 20, dtype=torch.uint8)
    tile.tile_embedding_backward(t, o, w, ws)
    tile.tile_embedding_backward(t, o, on_device(300, 64), ws, accumulate=True)
    for args in ((t, o, on_device(300, 63, dtype=bf), ws), (t, o, on_device(300, 64, dtype=torch.int32), ws),
                 (on_device(5, dtype=i64), o, w, ws), (t, o, w, torch.zeros(5)),
                 (t, o, on_device(300, 64, dtype=bf, index=1), ws)):
        with pytest.raises(ValueError):
            tile.tile_embedding_backward(*args)
    assert len(calls) == 3
    with pytest.raises(ValueError):
        tile.embedding_backward(t, o)
    with pytest.raises(ValueError):
        tile.embedding_backward(t, o, 299, dweight=w)
    with pytest.raises(ValueError):
        tile.embedding_backward(t, o, dweight=w, dtype=torch.float32)


def test_policy_tensors(calls):
    i64 = torch.int64
    x, adv, off, tgt = on_device(9), on_device(3), on_device(4, dtype=i64), on_device(9, dtype=i64)
    out = dict(stats=on_device(4), weights=on_device(3), workspace=on_device(4096, dtype=torch.uint8))
    tile.tile_policy_loss(x, x, adv, **out, offsets=off, target=tgt, sequence_advantage=True)
    tile.tile_policy_loss(x, x, x, **out, offsets=off, ref_nll=x)
    assert len(calls) == 2
    for args, kw in (((x, x, adv), {}), ((x, x, adv), dict(offsets=off)), ((x, on_device(8), x), dict(offsets=off)),
                     ((x, x, x), dict(offsets=on_device(4))), ((x, x, x), dict(offsets=on_device(1, dtype=i64))),
                     ((x, x, x), dict(offsets=off, target=x)), ((x, x, x), {}),
                     ((on_device(3, 3), x, x), dict(offsets=off)), ((torch.zeros(9), x, x), dict(offsets=off)),
                     ((x, x, x), dict(offsets=off, ref_nll=on_device(9, dtype=torch.bfloat16))),
                     ((x, x, x), dict(offsets=off, ignore_index=1 << 63))):
        with pytest.raises(ValueError):
            tile.tile_policy_loss(*args, **out, **kw)
    with pytest.raises(ValueError):
        tile.policy_loss(x, x, x, mean="rows")
    w = on_device(3)
    tile.tile_policy_loss_backward(x, x, x, w, x, on_device(1), offsets=off)
    tile.tile_policy_loss_backward(x, x, x, w, x, on_device(1, 1), offsets=off)
    for args in ((x, x, x, on_device(2), x), (x, x, x, w, on_device(8)), (x, x, x, w, x, on_device(2)),
                 (x, x, x, w, x, on_device(1, dtype=torch.float64))):
        with pytest.raises(ValueError):
            tile.tile_policy_loss_backward(*args, offsets=off)
    assert len(calls) == 4


def test_lists_of_tensors(calls):
    f8, bf = torch.float8_e4m3fn, torch.bfloat16
    p = [on_device(3, 4), on_device(700)]
    g = [on_device(12, dtype=bf), on_device(700)]
    c = [on_device(12, dtype=bf), on_device(700, dtype=torch.float16)]
    tile.tile_adamw(p, g, p, p, 1)
    tile.tile_adamw(p, g, p, p, 1, copies=c, weight_decay=[0.1, 0])
    table = calls[-1][1][0]
    assert len(table) == 160 and struct.unpack("8qf2i4x", table[80:])[7:] == (700, 0.0, 0, 2)
    tile.tile_adamw(p, g, p, p, 1, copies=[None, c[1]])
    table = calls.pop()[1][0]
    assert struct.unpack("8qf2i4x", table[:80])[6] == 0 and struct.unpack("8qf2i4x", table[80:])[6] != 0
    e = [on_device(12, dtype=f8), on_device(700, dtype=f8)]
    s = [on_device(1), on_device(3)]
    tile.tile_adamw(p, g, e, e, on_device(1, dtype=torch.int64), on_device(1), exp_avg_scales=s, exp_avg_sq_scales=s)
    tile.tile_adamw([], [], [], [], 1)
    assert len(calls) == 3
    ok = dict(params=p, grads=g, exp_avg=p, exp_avg_sq=p, step=1)
    for change in (dict(grads=g[:1]), dict(exp_avg=[p[1], p[0]]), dict(params=c), dict(exp_avg=e),
                   dict(exp_avg=e, exp_avg_sq=e), dict(exp_avg=e, exp_avg_sq=e, exp_avg_scales=s, exp_avg_sq_scales=p),
                   dict(exp_avg_scales=s), dict(grads=[on_device(12, dtype=torch.int32), g[1]]),
                   dict(grads=[on_device(4, 6).t()[::2], g[1]]), dict(copies=p), dict(copies=c[:1]),
                   dict(weight_decay=[0.1]), dict(step=1 << 63), dict(params=[on_device(3, 4, index=1), p[1]]),
                   dict(grads=[torch.zeros(12), g[1]]), dict(step=on_device(2, dtype=torch.int64)),
                   dict(step=on_device(1)), dict(lr=on_device(1, dtype=torch.float64)), dict(factor=on_device(2)),
                   dict(params=[torch.zeros(3, 4), p[1]]), dict(params=[], exp_avg=[], exp_avg_sq=[])):
        with pytest.raises(ValueError):
            tile.tile_adamw(**{**ok, **change})
    for change in (dict(grads=[None, g[1]]), dict(params=p[0]), dict(exp_avg=[1.0, 2.0])):
        with pytest.raises(TypeError):
            tile.tile_adamw(**{**ok, **change})
    ws, out = on_device(1 << 16, dtype=torch.uint8), on_device(2)
    tile.tile_grad_norm(g, out, ws)
    assert calls[-1][1][3] == math.inf
    for grads in ([on_device(5, dtype=torch.int8)], [on_device(5, index=1)], [torch.zeros(5)],
                  [on_device(4, 6).t()]):
        with pytest.raises(ValueError):
            tile.tile_grad_norm(grads, out, ws)
    with pytest.raises(TypeError):
        tile.tile_grad_norm(on_device(5), out, ws)
    with pytest.raises(ValueError):
        tile.grad_norm([])
    with pytest.raises(ValueError):
        tile.adamw_state(p, bits=16)
    assert len(calls) == 4


def test_streams_of_wrappers_that_take_lists(monkeypatch):
    """The first tensor of a list says whose stream a handle is."""
    seen = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: seen.append(device) or
                        types.SimpleNamespace(device=torch.device("cuda", device), cuda_stream=handle))

    class Current:
        def __init__(self, s):
            pass

        def __enter__(self):
            return self

        def __exit__(self, *a):
            return False
    monkeypatch.setattr(torch.cuda, "stream", Current)
    tile._on_stream(lambda grads: None)([on_device(4, index=2)], stream=0x7700)
    assert seen == [2]
    with pytest.raises(ValueError, match="stream"):
        tile.grad_norm([on_device(4, index=1)], stream=types.SimpleNamespace(device=torch.device("cuda", 0),
                                                                            cuda_stream=5))
    for name in ("embedding", "embedding_backward", "policy_loss", "policy_loss_backward", "grad_norm"):
        assert hasattr(getattr(tile, name), "__wrapped__")
