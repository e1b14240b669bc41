"""Python binding of ``libtile_rows.so``: fused FP32 row normalisation on GB300.

Argument marshalling only.  Every function here checks tensor metadata, takes
device pointers and the current CUDA stream from PyTorch, and calls the C ABI
of the same name (declared in ``include/tile_rows.h``); all arithmetic runs in
the library's CUDA kernels.  There is no CPU path: CPU tensors are rejected,
and importing the binding without the built library raises.

    import torch, tile_compiler_row_gb300 as tile
    y = torch.empty_like(x)
    tile.tile_residual_layernorm_f32(x, r, y, eps=1e-5)
"""

from __future__ import annotations

import ctypes
import itertools
import operator
import os
import struct

from ._build import LIBRARY

__all__ = [
    "TileError", "OPS", "load", "library_path",
    "tile_residual_layernorm_f32", "tile_layernorm_f32", "tile_rmsnorm_f32",
    "tile_softmax_f32", "tile_run_plan_f32", "tile_describe_plan", "tile_plan_info",
    "tile_plan_count", "tile_max_width", "tile_status_string",
    "tile_check_device_status", "tile_last_cuda_error", "tile_run_host_f32",
    "tile_host_workspace_bytes", "tile_host_schedule", "tile_run_host_static_f32", "tile_layernorm_affine_f32",
    "tile_rmsnorm_weighted_f32", "tile_row_sum_f32", "tile_row_minmax_f32",
    "tile_run_plan_args_f32", "tile_sigmoid_pair_f32", "tile_gelu_tanh_pair_f32",
    "tile_residual_layernorm_bf16", "tile_layernorm_bf16", "tile_rmsnorm_bf16",
    "tile_softmax_bf16", "tile_layernorm_affine_bf16", "tile_rmsnorm_weighted_bf16",
    "tile_row_sum_bf16", "tile_row_minmax_bf16", "tile_residual_layernorm_f16",
    "tile_layernorm_f16", "tile_rmsnorm_f16", "tile_softmax_f16", "tile_layernorm_affine_f16",
    "tile_rmsnorm_weighted_f16", "tile_row_sum_f16", "tile_row_minmax_f16",
    "tile_describe_plan_ex", "tile_plan_info_ex",
    "tile_layernorm_backward_f32", "tile_rmsnorm_backward_f32", "tile_softmax_backward_f32",
    "tile_run_backward_plan_f32", "tile_norm_param_grad_workspace_bytes",
    "tile_block_norm", "tile_block_norm_backward", "tile_block_norm_backward_workspace_bytes",
    "tile_block_norm_backward_gated_workspace_bytes",
    "tile_test_block_norm_backward_wait_timeout", "tile_test_linear_cross_entropy_wait_timeout",
    "tile_linear_cross_entropy", "tile_linear_cross_entropy_workspace_bytes",
    "tile_linear_cross_entropy_backward", "tile_linear_cross_entropy_backward_workspace_bytes",
    "block_norm", "block_norm_backward", "linear_cross_entropy", "linear_cross_entropy_backward",
    "tile_embedding", "tile_embedding_backward", "tile_embedding_backward_workspace_bytes",
    "tile_policy_loss", "tile_policy_loss_backward", "tile_policy_loss_workspace_bytes",
    "tile_grad_norm", "tile_grad_norm_workspace_bytes", "tile_adamw",
    "embedding", "embedding_backward", "policy_loss", "policy_loss_backward", "grad_norm",
    "adamw", "adamw_state",
    "tile_norm_param_grad_f32", "tile_run_backward_plan_ex",
    "tile_layernorm_backward_bf16", "tile_rmsnorm_backward_bf16", "tile_softmax_backward_bf16",
    "tile_norm_param_grad_bf16", "tile_layernorm_backward_f16", "tile_rmsnorm_backward_f16",
    "tile_softmax_backward_f16", "tile_norm_param_grad_f16", "tile_test_staged_wait_timeout",
    "tile_inject_launch_failure", "tile_describe_backward_plan", "tile_test_force_general_kernels",
    "residual_layernorm", "layernorm", "rmsnorm", "softmax", "run",
]

#: Library operation codes, by name.
OPS = {"residual_layernorm": 0, "layernorm": 1, "rmsnorm": 2, "softmax": 3, "row_sum": 4,
       "row_minmax": 5, "layernorm_affine": 6, "rmsnorm_weighted": 7}

TILE_OK = 0

#: Element type codes (TILE_DTYPE_*).
DTYPES = {"f32": 0, "bf16": 1, "f16": 2}


class TileError(RuntimeError):
    """A non-zero status returned by the C ABI."""

    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: status {status} ({tile_status_string(status)})"
        if status == -5:
            msg += f", cudaError {tile_last_cuda_error()}"
        super().__init__(msg)


class TilePlan(ctypes.Structure):
    _fields_ = [
        ("op", ctypes.c_int), ("rows", ctypes.c_int), ("width", ctypes.c_int),
        ("id", ctypes.c_int), ("path", ctypes.c_int), ("vec", ctypes.c_int),
        ("warps_per_program", ctypes.c_int), ("programs_per_cta", ctypes.c_int),
        ("chunks", ctypes.c_int), ("cluster", ctypes.c_int), ("threads", ctypes.c_int),
        ("workers", ctypes.c_int), ("stripe_floats", ctypes.c_int),
        ("max_width", ctypes.c_int), ("smem_bytes", ctypes.c_int),
        ("barriers_per_row", ctypes.c_int), ("grid", ctypes.c_longlong),
        ("dtype", ctypes.c_int),
    ]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class TileBlockNormArgs(ctypes.Structure):
    _fields_ = [
        ("in_", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("gamma_post", ctypes.c_void_p),
        ("gate", ctypes.c_void_p), ("gamma_pre", ctypes.c_void_p), ("hidden", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("rows", ctypes.c_int), ("width", ctypes.c_int),
        ("rows_per_gate", ctypes.c_int), ("norms", ctypes.c_int),
        ("residual_scale", ctypes.c_float), ("eps", ctypes.c_float), ("dtype", ctypes.c_int),
    ]


class TileBlockNormBackwardArgs(ctypes.Structure):
    _fields_ = [
        ("in_", ctypes.c_void_p), ("hidden", ctypes.c_void_p), ("dhidden", ctypes.c_void_p),
        ("dout", ctypes.c_void_p), ("gamma_post", ctypes.c_void_p), ("gate", ctypes.c_void_p),
        ("gamma_pre", ctypes.c_void_p), ("din", ctypes.c_void_p), ("dresidual", ctypes.c_void_p),
        ("dgamma_post", ctypes.c_void_p), ("dgate", ctypes.c_void_p),
        ("dgamma_pre", ctypes.c_void_p), ("rows", ctypes.c_int), ("width", ctypes.c_int),
        ("rows_per_gate", ctypes.c_int), ("norms", ctypes.c_int),
        ("residual_scale", ctypes.c_float), ("eps", ctypes.c_float), ("dtype", ctypes.c_int),
    ]


class TilePolicyLossArgs(ctypes.Structure):
    _fields_ = [
        ("nll", ctypes.c_void_p), ("old_nll", ctypes.c_void_p), ("ref_nll", ctypes.c_void_p),
        ("advantage", ctypes.c_void_p), ("target", ctypes.c_void_p),
        ("offsets", ctypes.c_void_p), ("ignore_index", ctypes.c_longlong),
        ("rows", ctypes.c_int), ("sequences", ctypes.c_int), ("flags", ctypes.c_int),
        ("clip_low", ctypes.c_float), ("clip_high", ctypes.c_float), ("kl_coef", ctypes.c_float),
    ]


class TileAdamwConfig(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
        ("eps", ctypes.c_double), ("step", ctypes.c_longlong), ("lr_device", ctypes.c_void_p),
        ("step_device", ctypes.c_void_p), ("factor", ctypes.c_void_p),
        ("seed", ctypes.c_ulonglong), ("state", ctypes.c_int),
    ]


class TileRowArgs(ctypes.Structure):
    _fields_ = [
        ("in_", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("gamma", ctypes.c_void_p),
        ("beta", ctypes.c_void_p), ("out", ctypes.c_void_p), ("out2", ctypes.c_void_p),
        ("rows", ctypes.c_int), ("width", ctypes.c_int), ("eps", ctypes.c_float),
        ("dtype", ctypes.c_int),
    ]


_lib = None


def library_path() -> str:
    return LIBRARY


def load():
    """Load the shared library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIBRARY):
        raise RuntimeError(
            f"{LIBRARY} is not built: run `python -c 'import __graft_entry__ as g; g.build()'` "
            "(the library has no CPU fallback)")
    lib = ctypes.CDLL(LIBRARY)
    P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    sigs = {
        "tile_residual_layernorm_f32": [P, P, P, I, I, F, P],
        "tile_layernorm_f32": [P, P, I, I, F, P],
        "tile_rmsnorm_f32": [P, P, I, I, F, P],
        "tile_softmax_f32": [P, P, I, I, F, P],
        "tile_run_plan_f32": [I, I, P, P, P, I, I, F, P],
        "tile_describe_plan": [I, I, I, ctypes.POINTER(TilePlan)],
        "tile_plan_info": [I, I, I, I, ctypes.POINTER(TilePlan)],
        "tile_plan_count": [],
        "tile_max_width": [],
        "tile_check_device_status": [P],
        "tile_last_cuda_error": [],
        "tile_run_host_f32": [I, P, P, P, I, I, F, P, ctypes.c_size_t, P],
        "tile_host_schedule": [I, I, I, ctypes.c_size_t, I, ctypes.POINTER(ctypes.c_int),
                               ctypes.POINTER(ctypes.c_int)],
        "tile_run_host_static_f32": [I, P, P, P, I, I, F, P],
        "tile_layernorm_affine_f32": [P, P, P, P, P, I, I, F, P],
        "tile_rmsnorm_weighted_f32": [P, P, P, I, I, F, P],
        "tile_row_sum_f32": [P, P, I, I, P],
        "tile_row_minmax_f32": [P, P, P, I, I, P],
        "tile_run_plan_args_f32": [I, I, ctypes.POINTER(TileRowArgs), P],
        "tile_sigmoid_pair_f32": [P, P, P, ctypes.c_longlong, P],
        "tile_gelu_tanh_pair_f32": [P, P, P, ctypes.c_longlong, P],
        "tile_residual_layernorm_bf16": [P, P, P, I, I, F, P],
        "tile_layernorm_bf16": [P, P, I, I, F, P],
        "tile_rmsnorm_bf16": [P, P, I, I, F, P],
        "tile_softmax_bf16": [P, P, I, I, F, P],
        "tile_layernorm_affine_bf16": [P, P, P, P, P, I, I, F, P],
        "tile_rmsnorm_weighted_bf16": [P, P, P, I, I, F, P],
        "tile_row_sum_bf16": [P, P, I, I, P],
        "tile_row_minmax_bf16": [P, P, P, I, I, P],
        "tile_residual_layernorm_f16": [P, P, P, I, I, F, P],
        "tile_layernorm_f16": [P, P, I, I, F, P],
        "tile_rmsnorm_f16": [P, P, I, I, F, P],
        "tile_softmax_f16": [P, P, I, I, F, P],
        "tile_layernorm_affine_f16": [P, P, P, P, P, I, I, F, P],
        "tile_rmsnorm_weighted_f16": [P, P, P, I, I, F, P],
        "tile_row_sum_f16": [P, P, I, I, P],
        "tile_row_minmax_f16": [P, P, P, I, I, P],
        "tile_describe_plan_ex": [I, I, I, I, ctypes.POINTER(TilePlan)],
        "tile_layernorm_backward_f32": [P, P, P, P, P, I, I, F, P],
        "tile_rmsnorm_backward_f32": [P, P, P, P, P, I, I, F, P],
        "tile_softmax_backward_f32": [P, P, P, I, I, P],
        "tile_run_backward_plan_f32": [I, I, P, P, P, P, P, I, I, F, P],
        "tile_norm_param_grad_f32": [P, P, P, P, P, I, I, P, ctypes.c_size_t, P],
        "tile_run_backward_plan_ex": [I, I, I, P, P, P, P, P, I, I, F, P],
        "tile_layernorm_backward_bf16": [P, P, P, P, P, I, I, F, P],
        "tile_rmsnorm_backward_bf16": [P, P, P, P, P, I, I, F, P],
        "tile_softmax_backward_bf16": [P, P, P, I, I, P],
        "tile_norm_param_grad_bf16": [P, P, P, P, P, I, I, P, ctypes.c_size_t, P],
        "tile_layernorm_backward_f16": [P, P, P, P, P, I, I, F, P],
        "tile_rmsnorm_backward_f16": [P, P, P, P, P, I, I, F, P],
        "tile_softmax_backward_f16": [P, P, P, I, I, P],
        "tile_norm_param_grad_f16": [P, P, P, P, P, I, I, P, ctypes.c_size_t, P],
        "tile_plan_info_ex": [I, I, I, I, I, ctypes.POINTER(TilePlan)],
        "tile_test_staged_wait_timeout": [I, I, ctypes.POINTER(TileRowArgs), ctypes.c_uint, P],
        "tile_inject_launch_failure": [I, I, I],
        "tile_test_force_general_kernels": [I],
        "tile_describe_backward_plan": [I, I, I, I, ctypes.POINTER(TilePlan)],
        "tile_block_norm": [ctypes.POINTER(TileBlockNormArgs), P],
        "tile_block_norm_backward": [ctypes.POINTER(TileBlockNormBackwardArgs), P,
                                     ctypes.c_size_t, P],
        "tile_test_block_norm_backward_wait_timeout": [
            ctypes.POINTER(TileBlockNormBackwardArgs), P, ctypes.c_size_t, P],
        "tile_test_linear_cross_entropy_wait_timeout": [I, P, P, P, P, P, I, I, I,
                                                        ctypes.c_longlong, P, ctypes.c_size_t, P],
        "tile_linear_cross_entropy": [I, P, P, P, P, P, I, I, I, ctypes.c_longlong, P,
                                      ctypes.c_size_t, P],
        "tile_linear_cross_entropy_backward": [I, P, P, P, P, P, P, P, I, I, I,
                                               ctypes.c_longlong, P, ctypes.c_size_t, P],
        "tile_embedding": [I, P, P, P, I, I, I, F, ctypes.c_longlong, P],
        "tile_embedding_backward": [I, I, P, P, P, I, I, I, F, ctypes.c_longlong, I, P,
                                    ctypes.c_size_t, P],
        "tile_policy_loss": [ctypes.POINTER(TilePolicyLossArgs), P, P, P, ctypes.c_size_t, P],
        "tile_policy_loss_backward": [ctypes.POINTER(TilePolicyLossArgs), P, P, P, P],
        "tile_grad_norm": [P, I, F, F, P, P, ctypes.c_size_t, P],
        "tile_adamw": [P, I, ctypes.POINTER(TileAdamwConfig), P],
    }
    for name, argtypes in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = argtypes
        fn.restype = ctypes.c_int
    lib.tile_norm_param_grad_workspace_bytes.argtypes = [I, I]
    lib.tile_norm_param_grad_workspace_bytes.restype = ctypes.c_size_t
    lib.tile_block_norm_backward_workspace_bytes.argtypes = [I, I]
    lib.tile_block_norm_backward_workspace_bytes.restype = ctypes.c_size_t
    lib.tile_block_norm_backward_gated_workspace_bytes.argtypes = [I, I, I]
    lib.tile_block_norm_backward_gated_workspace_bytes.restype = ctypes.c_size_t
    for name in ("tile_linear_cross_entropy_workspace_bytes",
                 "tile_linear_cross_entropy_backward_workspace_bytes",
                 "tile_embedding_backward_workspace_bytes"):
        getattr(lib, name).argtypes = [I, I, I]
        getattr(lib, name).restype = ctypes.c_size_t
    lib.tile_policy_loss_workspace_bytes.argtypes = [I, I]
    lib.tile_policy_loss_workspace_bytes.restype = ctypes.c_size_t
    lib.tile_grad_norm_workspace_bytes.argtypes = [I]
    lib.tile_grad_norm_workspace_bytes.restype = ctypes.c_size_t
    lib.tile_host_workspace_bytes.argtypes = [I, I, I]
    lib.tile_host_workspace_bytes.restype = ctypes.c_size_t
    lib.tile_status_string.argtypes = [I]
    lib.tile_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _matrix(t, name, dtype="f32"):
    """(pointer, rows, width) of a CUDA row-major matrix tensor of ``dtype``."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    want = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    if t.dtype != want:
        raise ValueError(f"{name} must be {want}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D [rows, width]")
    rows, width = t.shape
    if rows > 1 and t.stride(0) != width or width > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be row-major with row stride == width")
    return t.data_ptr(), rows, width


def _check(status, where):
    if status != TILE_OK:
        raise TileError(status, where)


def _same_shape(a, b, names):
    if tuple(a.shape) != tuple(b.shape):
        raise ValueError(f"{names}: shapes {tuple(a.shape)} and {tuple(b.shape)} differ")


# ---------------------------------------------------------------------------
# the C ABI, one Python function per entry point
# ---------------------------------------------------------------------------

def tile_residual_layernorm_f32(x, residual, out, eps=1e-5, stream=None):
    px, rows, width = _matrix(x, "x")
    pr, _, _ = _matrix(residual, "residual")
    po, _, _ = _matrix(out, "out")
    _same_shape(x, residual, "x/residual")
    _same_shape(x, out, "x/out")
    _check(load().tile_residual_layernorm_f32(px, pr, po, rows, width, eps, _stream(stream)),
           "tile_residual_layernorm_f32")


def _unary(name):
    def fn(x, out, eps=1e-5, stream=None):
        px, rows, width = _matrix(x, "x")
        po, _, _ = _matrix(out, "out")
        _same_shape(x, out, "x/out")
        _check(getattr(load(), name)(px, po, rows, width, eps, _stream(stream)), name)
    fn.__name__ = name
    fn.__doc__ = f"Calls ``{name}`` (see include/tile_rows.h)."
    return fn


tile_layernorm_f32 = _unary("tile_layernorm_f32")
tile_rmsnorm_f32 = _unary("tile_rmsnorm_f32")
tile_softmax_f32 = _unary("tile_softmax_f32")


def tile_run_plan_f32(op, plan_id, x, residual, out, eps=1e-5, stream=None):
    op = OPS[op] if isinstance(op, str) else op
    px, rows, width = _matrix(x, "x")
    po, _, _ = _matrix(out, "out")
    _same_shape(x, out, "x/out")
    pr = None
    if residual is not None:
        pr, _, _ = _matrix(residual, "residual")
        _same_shape(x, residual, "x/residual")
    _check(load().tile_run_plan_f32(op, plan_id, px, pr, po, rows, width, eps, _stream(stream)),
           "tile_run_plan_f32")


def _vector(t, n, name):
    """Pointer of a CUDA FP32 contiguous tensor of n elements (None -> NULL)."""
    import torch
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32:
        raise ValueError(f"{name} must be a CUDA float32 tensor")
    if not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{name} must be contiguous with {n} elements")
    return t.data_ptr()


def tile_layernorm_affine_f32(x, residual, gamma, beta, out, eps=1e-5, stream=None):
    """LayerNorm(x [+ residual]) * gamma + beta; residual and beta may be None."""
    px, rows, width = _matrix(x, "x")
    po, _, _ = _matrix(out, "out")
    _same_shape(x, out, "x/out")
    pr = None
    if residual is not None:
        pr, _, _ = _matrix(residual, "residual")
        _same_shape(x, residual, "x/residual")
    pg = _vector(gamma, width, "gamma")
    pb = _vector(beta, width, "beta")
    _check(load().tile_layernorm_affine_f32(px, pr, pg, pb, po, rows, width, eps, _stream(stream)),
           "tile_layernorm_affine_f32")


def tile_rmsnorm_weighted_f32(x, gamma, out, eps=1e-5, stream=None):
    px, rows, width = _matrix(x, "x")
    po, _, _ = _matrix(out, "out")
    _same_shape(x, out, "x/out")
    pg = _vector(gamma, width, "gamma")
    _check(load().tile_rmsnorm_weighted_f32(px, pg, po, rows, width, eps, _stream(stream)),
           "tile_rmsnorm_weighted_f32")


def tile_row_sum_f32(x, sums, stream=None):
    px, rows, width = _matrix(x, "x")
    ps = _vector(sums, rows, "sums")
    _check(load().tile_row_sum_f32(px, ps, rows, width, _stream(stream)), "tile_row_sum_f32")


def tile_row_minmax_f32(x, mins, maxs, stream=None):
    px, rows, width = _matrix(x, "x")
    pmn = _vector(mins, rows, "mins")
    pmx = _vector(maxs, rows, "maxs")
    _check(load().tile_row_minmax_f32(px, pmn, pmx, rows, width, _stream(stream)),
           "tile_row_minmax_f32")


def _row_args(x, out, residual, gamma, beta, out2, eps):
    import torch
    dt = {torch.bfloat16: "bf16", torch.float16: "f16"}.get(
        x.dtype if isinstance(x, torch.Tensor) else None, "f32")
    px, rows, width = _matrix(x, "x", dt)
    a = TileRowArgs()
    a.in_ = px
    a.dtype = DTYPES[dt]
    a.residual = _matrix(residual, "residual", dt)[0] if residual is not None else None
    a.gamma = _vector(gamma, width, "gamma")
    a.beta = _vector(beta, width, "beta")
    a.out = out.data_ptr()
    a.out2 = out2.data_ptr() if out2 is not None else None
    a.rows, a.width, a.eps = rows, width, eps
    return a


def tile_run_plan_args_f32(op, plan_id, x, out, residual=None, gamma=None, beta=None, out2=None,
                           eps=1e-5, stream=None):
    """Any row op with a forced plan (``out``: matrix, or [rows] for row_sum/row_minmax).
    ``x`` may be float32, bfloat16 or float16; the element type follows it."""
    op = OPS[op] if isinstance(op, str) else op
    a = _row_args(x, out, residual, gamma, beta, out2, eps)
    _check(load().tile_run_plan_args_f32(op, plan_id, ctypes.byref(a), _stream(stream)),
           "tile_run_plan_args_f32")


def tile_inject_launch_failure(cuda_error, skip=0, count=1):
    """Test hook: after ``skip`` launch attempts, the next ``count`` fail on
    the host with ``cuda_error`` (``count=0`` disarms)."""
    _check(load().tile_inject_launch_failure(int(cuda_error), int(skip), int(count)),
           "tile_inject_launch_failure")


def tile_test_force_general_kernels(on):
    """Test hook: with ``on`` true, 2-byte launches take the general kernel
    forms instead of the whole-vector ones (bitwise the same results)."""
    _check(load().tile_test_force_general_kernels(int(bool(on))),
           "tile_test_force_general_kernels")


def tile_test_staged_wait_timeout(op, plan_id, x, out, spin_limit, residual=None, gamma=None,
                                  beta=None, eps=1e-5, stream=None):
    """Test hook: the staged plan with every CTA's first copy withheld and
    waits limited to ``spin_limit`` polls (the outputs are invalid; the
    device status word reports the timeout)."""
    op = OPS[op] if isinstance(op, str) else op
    a = _row_args(x, out, residual, gamma, beta, None, eps)
    _check(load().tile_test_staged_wait_timeout(op, plan_id, ctypes.byref(a), int(spin_limit),
                                                _stream(stream)),
           "tile_test_staged_wait_timeout")


def _flat(t, name):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32:
        raise ValueError(f"{name} must be a CUDA float32 tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr(), t.numel()


def _pair_fn(name):
    def fn(x, value, derivative, stream=None):
        px, n = _flat(x, "x")
        pv, nv = _flat(value, "value")
        pd, nd = _flat(derivative, "derivative")
        if nv != n or nd != n:
            raise ValueError("value and derivative must have as many elements as x")
        _check(getattr(load(), name)(px, pv, pd, n, _stream(stream)), name)
    fn.__name__ = name
    fn.__doc__ = f"Calls ``{name}`` (see include/tile_rows.h)."
    return fn


tile_sigmoid_pair_f32 = _pair_fn("tile_sigmoid_pair_f32")
tile_gelu_tanh_pair_f32 = _pair_fn("tile_gelu_tanh_pair_f32")


# ---- backward passes ----------------------------------------------------------

def _bwd(name, dtype="f32"):
    def fn(x, gamma, dy, dx, row_stats=None, eps=1e-5, stream=None):
        px, rows, width = _matrix(x, "x", dtype)
        pd, _, _ = _matrix(dy, "dy", dtype)
        po, _, _ = _matrix(dx, "dx", dtype)
        _same_shape(x, dy, "x/dy")
        _same_shape(x, dx, "x/dx")
        ps = _vector(row_stats, 2 * rows, "row_stats") if row_stats is not None else None
        _check(getattr(load(), name)(px, _vector(gamma, width, "gamma"), pd, po, ps, rows, width,
                                     eps, _stream(stream)), name)
    fn.__name__ = name
    fn.__doc__ = f"Calls ``{name}`` (see include/tile_rows.h)."
    return fn


tile_layernorm_backward_f32 = _bwd("tile_layernorm_backward_f32")
tile_rmsnorm_backward_f32 = _bwd("tile_rmsnorm_backward_f32")


def tile_softmax_backward_f32(y, dy, dx, stream=None):
    py, rows, width = _matrix(y, "y")
    pd, _, _ = _matrix(dy, "dy")
    po, _, _ = _matrix(dx, "dx")
    _same_shape(y, dy, "y/dy")
    _same_shape(y, dx, "y/dx")
    _check(load().tile_softmax_backward_f32(py, pd, po, rows, width, _stream(stream)),
           "tile_softmax_backward_f32")


def tile_run_backward_plan_f32(op, plan_id, x, gamma, dy, dx, row_stats=None, eps=1e-5,
                               stream=None):
    op = OPS[op] if isinstance(op, str) else op
    px, rows, width = _matrix(x, "x")
    pd, _, _ = _matrix(dy, "dy")
    po, _, _ = _matrix(dx, "dx")
    ps = _vector(row_stats, 2 * rows, "row_stats") if row_stats is not None else None
    _check(load().tile_run_backward_plan_f32(op, plan_id, px, _vector(gamma, width, "gamma"), pd,
                                             po, ps, rows, width, eps, _stream(stream)),
           "tile_run_backward_plan_f32")


def _softmax_bwd(name, dtype):
    def fn(y, dy, dx, stream=None):
        py, rows, width = _matrix(y, "y", dtype)
        pd, _, _ = _matrix(dy, "dy", dtype)
        po, _, _ = _matrix(dx, "dx", dtype)
        _same_shape(y, dy, "y/dy")
        _same_shape(y, dx, "y/dx")
        _check(getattr(load(), name)(py, pd, po, rows, width, _stream(stream)), name)
    fn.__name__ = name
    fn.__doc__ = f"Calls ``{name}`` (see include/tile_rows.h)."
    return fn


def _param_grad(name, dtype):
    def fn(x, dy, row_stats, dgamma, dbeta, workspace, stream=None):
        px, rows, width = _matrix(x, "x", dtype)
        pd, _, _ = _matrix(dy, "dy", dtype)
        if not workspace.is_cuda:
            raise ValueError("workspace must be a CUDA tensor")
        _check(getattr(load(), name)(
            px, pd, _vector(row_stats, 2 * rows, "row_stats"), _vector(dgamma, width, "dgamma"),
            _vector(dbeta, width, "dbeta"), rows, width, workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _stream(stream)), name)
    fn.__name__ = name
    fn.__doc__ = f"Calls ``{name}`` (see include/tile_rows.h)."
    return fn


tile_layernorm_backward_bf16 = _bwd("tile_layernorm_backward_bf16", "bf16")
tile_rmsnorm_backward_bf16 = _bwd("tile_rmsnorm_backward_bf16", "bf16")
tile_softmax_backward_bf16 = _softmax_bwd("tile_softmax_backward_bf16", "bf16")
tile_norm_param_grad_bf16 = _param_grad("tile_norm_param_grad_bf16", "bf16")
tile_layernorm_backward_f16 = _bwd("tile_layernorm_backward_f16", "f16")
tile_rmsnorm_backward_f16 = _bwd("tile_rmsnorm_backward_f16", "f16")
tile_softmax_backward_f16 = _softmax_bwd("tile_softmax_backward_f16", "f16")
tile_norm_param_grad_f16 = _param_grad("tile_norm_param_grad_f16", "f16")


def tile_run_backward_plan_ex(op, plan_id, x, gamma, dy, dx, row_stats=None, eps=1e-5,
                              stream=None):
    """tile_run_backward_plan_f32 for the element type of ``x`` (float32,
    bfloat16 or float16)."""
    import torch
    op = OPS[op] if isinstance(op, str) else op
    dt = {torch.bfloat16: "bf16", torch.float16: "f16"}.get(x.dtype, "f32")
    px, rows, width = _matrix(x, "x", dt)
    pd, _, _ = _matrix(dy, "dy", dt)
    po, _, _ = _matrix(dx, "dx", dt)
    ps = _vector(row_stats, 2 * rows, "row_stats") if row_stats is not None else None
    _check(load().tile_run_backward_plan_ex(op, plan_id, DTYPES[dt], px,
                                            _vector(gamma, width, "gamma"), pd, po, ps, rows,
                                            width, eps, _stream(stream)),
           "tile_run_backward_plan_ex")


def tile_norm_param_grad_workspace_bytes(rows, width):
    return load().tile_norm_param_grad_workspace_bytes(rows, width)


def tile_norm_param_grad_f32(x, dy, row_stats, dgamma, dbeta, workspace, stream=None):
    px, rows, width = _matrix(x, "x")
    pd, _, _ = _matrix(dy, "dy")
    if not workspace.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    _check(load().tile_norm_param_grad_f32(
        px, pd, _vector(row_stats, 2 * rows, "row_stats"), _vector(dgamma, width, "dgamma"),
        _vector(dbeta, width, "dbeta"), rows, width, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream(stream)), "tile_norm_param_grad_f32")


# ---- BF16 rows ---------------------------------------------------------------

def tile_residual_layernorm_bf16(x, residual, out, eps=1e-5, stream=None):
    px, rows, width = _matrix(x, "x", "bf16")
    pr, _, _ = _matrix(residual, "residual", "bf16")
    po, _, _ = _matrix(out, "out", "bf16")
    _same_shape(x, residual, "x/residual")
    _same_shape(x, out, "x/out")
    _check(load().tile_residual_layernorm_bf16(px, pr, po, rows, width, eps, _stream(stream)),
           "tile_residual_layernorm_bf16")


def _unary_bf16(name):
    def fn(x, out, eps=1e-5, stream=None):
        px, rows, width = _matrix(x, "x", "bf16")
        po, _, _ = _matrix(out, "out", "bf16")
        _same_shape(x, out, "x/out")
        _check(getattr(load(), name)(px, po, rows, width, eps, _stream(stream)), name)
    fn.__name__ = name
    fn.__doc__ = f"Calls ``{name}`` (see include/tile_rows.h)."
    return fn


tile_layernorm_bf16 = _unary_bf16("tile_layernorm_bf16")
tile_rmsnorm_bf16 = _unary_bf16("tile_rmsnorm_bf16")
tile_softmax_bf16 = _unary_bf16("tile_softmax_bf16")


def tile_layernorm_affine_bf16(x, residual, gamma, beta, out, eps=1e-5, stream=None):
    px, rows, width = _matrix(x, "x", "bf16")
    po, _, _ = _matrix(out, "out", "bf16")
    _same_shape(x, out, "x/out")
    pr = None
    if residual is not None:
        pr, _, _ = _matrix(residual, "residual", "bf16")
        _same_shape(x, residual, "x/residual")
    _check(load().tile_layernorm_affine_bf16(px, pr, _vector(gamma, width, "gamma"),
                                             _vector(beta, width, "beta"), po, rows, width, eps,
                                             _stream(stream)), "tile_layernorm_affine_bf16")


def tile_rmsnorm_weighted_bf16(x, gamma, out, eps=1e-5, stream=None):
    px, rows, width = _matrix(x, "x", "bf16")
    po, _, _ = _matrix(out, "out", "bf16")
    _same_shape(x, out, "x/out")
    _check(load().tile_rmsnorm_weighted_bf16(px, _vector(gamma, width, "gamma"), po, rows, width,
                                             eps, _stream(stream)), "tile_rmsnorm_weighted_bf16")


def tile_row_sum_bf16(x, sums, stream=None):
    px, rows, width = _matrix(x, "x", "bf16")
    _check(load().tile_row_sum_bf16(px, _vector(sums, rows, "sums"), rows, width, _stream(stream)),
           "tile_row_sum_bf16")


def tile_row_minmax_bf16(x, mins, maxs, stream=None):
    px, rows, width = _matrix(x, "x", "bf16")
    _check(load().tile_row_minmax_bf16(px, _vector(mins, rows, "mins"), _vector(maxs, rows, "maxs"),
                                       rows, width, _stream(stream)), "tile_row_minmax_bf16")


def tile_residual_layernorm_f16(x, residual, out, eps=1e-5, stream=None):
    px, rows, width = _matrix(x, "x", "f16")
    pr, _, _ = _matrix(residual, "residual", "f16")
    po, _, _ = _matrix(out, "out", "f16")
    _same_shape(x, residual, "x/residual")
    _same_shape(x, out, "x/out")
    _check(load().tile_residual_layernorm_f16(px, pr, po, rows, width, eps, _stream(stream)),
           "tile_residual_layernorm_f16")


def _unary_f16(name):
    def fn(x, out, eps=1e-5, stream=None):
        px, rows, width = _matrix(x, "x", "f16")
        po, _, _ = _matrix(out, "out", "f16")
        _same_shape(x, out, "x/out")
        _check(getattr(load(), name)(px, po, rows, width, eps, _stream(stream)), name)
    fn.__name__ = name
    fn.__doc__ = f"Calls ``{name}`` (see include/tile_rows.h)."
    return fn


tile_layernorm_f16 = _unary_f16("tile_layernorm_f16")
tile_rmsnorm_f16 = _unary_f16("tile_rmsnorm_f16")
tile_softmax_f16 = _unary_f16("tile_softmax_f16")


def tile_layernorm_affine_f16(x, residual, gamma, beta, out, eps=1e-5, stream=None):
    px, rows, width = _matrix(x, "x", "f16")
    po, _, _ = _matrix(out, "out", "f16")
    _same_shape(x, out, "x/out")
    pr = None
    if residual is not None:
        pr, _, _ = _matrix(residual, "residual", "f16")
        _same_shape(x, residual, "x/residual")
    _check(load().tile_layernorm_affine_f16(px, pr, _vector(gamma, width, "gamma"),
                                             _vector(beta, width, "beta"), po, rows, width, eps,
                                             _stream(stream)), "tile_layernorm_affine_f16")


def tile_rmsnorm_weighted_f16(x, gamma, out, eps=1e-5, stream=None):
    px, rows, width = _matrix(x, "x", "f16")
    po, _, _ = _matrix(out, "out", "f16")
    _same_shape(x, out, "x/out")
    _check(load().tile_rmsnorm_weighted_f16(px, _vector(gamma, width, "gamma"), po, rows, width,
                                             eps, _stream(stream)), "tile_rmsnorm_weighted_f16")


def tile_row_sum_f16(x, sums, stream=None):
    px, rows, width = _matrix(x, "x", "f16")
    _check(load().tile_row_sum_f16(px, _vector(sums, rows, "sums"), rows, width, _stream(stream)),
           "tile_row_sum_f16")


def tile_row_minmax_f16(x, mins, maxs, stream=None):
    px, rows, width = _matrix(x, "x", "f16")
    _check(load().tile_row_minmax_f16(px, _vector(mins, rows, "mins"), _vector(maxs, rows, "maxs"),
                                       rows, width, _stream(stream)), "tile_row_minmax_f16")


def _host_matrix(t, name):
    """(pointer, rows, width) of a CPU FP32 row-major matrix tensor."""
    import torch
    if not isinstance(t, torch.Tensor) or t.is_cuda:
        raise ValueError(f"{name} must be a CPU tensor (ideally pinned)")
    if t.dtype != torch.float32 or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D float32 tensor")
    rows, width = t.shape
    if rows > 1 and t.stride(0) != width or width > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be row-major with row stride == width")
    return t.data_ptr(), rows, width


def tile_run_host_f32(op, x, residual, out, workspace, eps=1e-5, stream=None):
    """``op`` on host tensors: in place when every tensor is pinned (one kernel
    reads and writes them over the host link), otherwise through the device
    ``workspace`` (a CUDA tensor) in chunks."""
    op = OPS[op] if isinstance(op, str) else op
    px, rows, width = _host_matrix(x, "x")
    po, _, _ = _host_matrix(out, "out")
    _same_shape(x, out, "x/out")
    pr = None
    if residual is not None:
        pr, _, _ = _host_matrix(residual, "residual")
        _same_shape(x, residual, "x/residual")
    if not workspace.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().tile_run_host_f32(op, px, pr, po, rows, width, eps, workspace.data_ptr(),
                                    nbytes, _stream(stream)), "tile_run_host_f32")


def tile_run_host_static_f32(op, x, residual, out, eps=1e-5, stream=None):
    """``op`` on host tensors through the library's static device staging
    area: for callers that cannot allocate device memory."""
    op = OPS[op] if isinstance(op, str) else op
    px, rows, width = _host_matrix(x, "x")
    po, _, _ = _host_matrix(out, "out")
    _same_shape(x, out, "x/out")
    pr = None
    if residual is not None:
        pr, _, _ = _host_matrix(residual, "residual")
        _same_shape(x, residual, "x/residual")
    _check(load().tile_run_host_static_f32(op, px, pr, po, rows, width, eps, _stream(stream)),
           "tile_run_host_static_f32")


def tile_host_workspace_bytes(op, width, chunk_rows):
    op = OPS[op] if isinstance(op, str) else op
    return load().tile_host_workspace_bytes(op, width, chunk_rows)


def tile_host_schedule(op, rows, width, work_bytes, direct_output=True):
    """(chunk rows, ring slots) that tile_run_host_f32 uses for these
    arguments; `direct_output` describes a pinned output buffer."""
    op = OPS[op] if isinstance(op, str) else op
    chunk, slots = ctypes.c_int(0), ctypes.c_int(0)
    _check(load().tile_host_schedule(op, rows, width, work_bytes, int(bool(direct_output)),
                                     ctypes.byref(chunk), ctypes.byref(slots)),
           "tile_host_schedule")
    return chunk.value, slots.value


def tile_describe_plan(op, rows, width):
    op = OPS[op] if isinstance(op, str) else op
    plan = TilePlan()
    _check(load().tile_describe_plan(op, rows, width, ctypes.byref(plan)), "tile_describe_plan")
    return plan.as_dict()


def tile_describe_plan_ex(op, dtype, rows, width):
    op = OPS[op] if isinstance(op, str) else op
    dtype = DTYPES[dtype] if isinstance(dtype, str) else dtype
    plan = TilePlan()
    _check(load().tile_describe_plan_ex(op, dtype, rows, width, ctypes.byref(plan)),
           "tile_describe_plan_ex")
    return plan.as_dict()


def tile_describe_backward_plan(op, dtype, rows, width):
    """The plan the backward entry points launch for (op, dtype, rows, width)
    on 16-byte co-aligned tensors."""
    op = OPS[op] if isinstance(op, str) else op
    dtype = DTYPES[dtype] if isinstance(dtype, str) else dtype
    plan = TilePlan()
    _check(load().tile_describe_backward_plan(op, dtype, rows, width, ctypes.byref(plan)),
           "tile_describe_backward_plan")
    return plan.as_dict()


def tile_plan_info_ex(plan_id, op, dtype, rows, width):
    """Plan ``plan_id`` for (op, dtype, rows, width), or None if not built, not
    covering, or without a variant for ``op``."""
    op = OPS[op] if isinstance(op, str) else op
    dtype = DTYPES[dtype] if isinstance(dtype, str) else dtype
    plan = TilePlan()
    st = load().tile_plan_info_ex(plan_id, op, dtype, rows, width, ctypes.byref(plan))
    if st in (-2, -8):
        return None
    _check(st, "tile_plan_info_ex")
    return plan.as_dict()


def tile_plan_info(plan_id, op, rows, width):
    """The built plan ``plan_id`` for (op, rows, width), or None if it cannot
    cover ``width`` or has no variant for ``op``."""
    op = OPS[op] if isinstance(op, str) else op
    plan = TilePlan()
    st = load().tile_plan_info(plan_id, op, rows, width, ctypes.byref(plan))
    if st in (-2, -8):
        return None
    _check(st, "tile_plan_info")
    return plan.as_dict()


def tile_plan_count():
    return load().tile_plan_count()


def tile_max_width():
    return load().tile_max_width()


def tile_status_string(status):
    return load().tile_status_string(status).decode()


def tile_check_device_status(stream=None):
    return load().tile_check_device_status(_stream(stream))


def tile_last_cuda_error():
    return load().tile_last_cuda_error()


# ---- block norm and linear cross entropy: marshalling ---------------------------
#
# A decode step calls these for a few rows at a time, where the host's part of
# a call is longer than the kernel's: each tensor is checked by one expression,
# and only a tensor that fails it is looked at again for the message.

_CODES = {}      # torch dtype -> DTYPES code, filled on first use


def _row_code(t, name):
    """The element type code of a row tensor."""
    if not _CODES:
        import torch
        _CODES.update({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2})
    code = _CODES.get(getattr(t, "dtype", None))
    if code is None:
        raise ValueError(f"{name} must be a float32, bfloat16 or float16 tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D [rows, width]")
    return code


def _ptr(t, name, dtype, shape, dev):
    """Pointer of a contiguous CUDA tensor of this type and shape on device
    index ``dev`` (None -> NULL)."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev} like the other tensors")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


_INT_MAX = 0x7fffffff
_INF = float("inf")


def _fit_int(*sizes):
    """Whether the C ABI's int holds every size (ctypes keeps the low 32 bits
    of what it does not hold)."""
    return min(sizes) >= 0 and max(sizes) <= _INT_MAX


def _device_index(t, name):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    return t.get_device()


def _workspace(t, dev):
    """(pointer, bytes) of a workspace tensor on device index ``dev``."""
    if not t.is_cuda or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    return t.data_ptr(), t.numel() * t.element_size()


def _same_device(stream, dev):
    """Refuses a torch stream of another device than index ``dev`` (an integer
    handle does not say whose it is)."""
    device = getattr(stream, "device", None)
    if device is not None and device.index != dev:
        raise ValueError(f"stream must be one of cuda:{dev} like the tensors, not of {device}")


def _call_on(dev, stream, name, *args):
    """Calls a C entry point with device ``dev`` current; ``stream`` None is
    that device's current stream."""
    import torch
    fn = getattr(load(), name)
    if stream is not None:
        _same_device(stream, dev)
    if torch._C._cuda_getDevice() == dev:
        s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)
        _check(fn(*args, s), name)
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, _stream(stream)), name)


# ---- block norm --------------------------------------------------------------

def _gates(t, rows, width, per_gate, dev, name):
    """Pointer of a gate matrix [ceil(rows / per_gate)][width] (a single gate
    row may be a vector), or None."""
    import torch
    if t is None:
        return None
    if per_gate < 1:
        raise ValueError("rows_per_gate must be at least 1 with a gate")
    n = -(-rows // per_gate)
    return _ptr(t, name, torch.float32, (width,) if n == 1 and t.dim() == 1 else (n, width), dev)


def tile_block_norm(x, residual, hidden, out, gamma_post=None, gate=None, gamma_pre=None,
                    post=True, pre=True, rows_per_gate=0, residual_scale=1.0, eps=1e-5,
                    stream=None):
    """hidden = residual_scale * residual + gate * norm(x; gamma_post) and
    out = norm(hidden; gamma_pre), RMSNorms, of float32, bfloat16 or float16
    rows; see ``tile_block_norm`` in include/tile_rows.h.  ``post`` / ``pre``
    switch the norms (without ``pre``, ``out`` is None); ``rows_per_gate``
    0, and any number from ``rows`` on, stands for all rows."""
    import torch
    code, dev = _row_code(x, "x"), _device_index(x, "x")
    shape, dt, f32 = x.shape, x.dtype, torch.float32
    rows, width = shape
    if not _fit_int(rows, width):
        raise ValueError(f"rows and width must be below 2^31, not {rows} x {width}")
    vec, per = (width,), min(rows_per_gate, rows) or rows or 1
    a = TileBlockNormArgs(
        _ptr(x, "x", dt, shape, dev), _ptr(residual, "residual", dt, shape, dev),
        _ptr(gamma_post, "gamma_post", f32, vec, dev), _gates(gate, rows, width, per, dev, "gate"),
        _ptr(gamma_pre, "gamma_pre", f32, vec, dev), _ptr(hidden, "hidden", dt, shape, dev),
        _ptr(out, "out", dt, shape, dev) if pre else None, rows, width, per,
        (1 if post else 0) | (2 if pre else 0), residual_scale, eps, code)
    _call_on(dev, stream, "tile_block_norm", ctypes.byref(a))


def tile_block_norm_backward_workspace_bytes(rows, width):
    """Enough for any number of gate rows."""
    if not _fit_int(rows, width):
        return 0
    return load().tile_block_norm_backward_workspace_bytes(rows, width)


def tile_block_norm_backward_gated_workspace_bytes(rows, width, gate_rows):
    """What a call with this many gate rows (0: no gate) needs."""
    if not _fit_int(rows, width, gate_rows):
        return 0
    return load().tile_block_norm_backward_gated_workspace_bytes(rows, width, gate_rows)


def tile_test_block_norm_backward_wait_timeout(*args, **kwargs):
    """Test hook: ``tile_block_norm_backward`` with a copy withheld, so that
    its waits give up (see include/tile_rows.h)."""
    tile_block_norm_backward(*args, **kwargs,
                             _entry="tile_test_block_norm_backward_wait_timeout")


def tile_block_norm_backward(x, hidden, dhidden, dout, din, dresidual, workspace,
                             gamma_post=None, gate=None, gamma_pre=None, dgamma_post=None,
                             dgate=None, dgamma_pre=None, post=True, pre=True, rows_per_gate=0,
                             residual_scale=1.0, eps=1e-5, stream=None,
                             _entry="tile_block_norm_backward"):
    """The gradients of ``tile_block_norm`` (see include/tile_rows.h).
    ``hidden`` is the forward's; ``dhidden`` may be None (``dout`` is then
    the only gradient), as may any parameter gradient."""
    import torch
    code, dev = _row_code(din, "din"), _device_index(din, "din")
    shape, dt, f32 = din.shape, din.dtype, torch.float32
    rows, width = shape
    if not _fit_int(rows, width):
        raise ValueError(f"rows and width must be below 2^31, not {rows} x {width}")
    vec, per = (width,), min(rows_per_gate, rows) or rows or 1
    a = TileBlockNormBackwardArgs(
        _ptr(x, "x", dt, shape, dev), _ptr(hidden, "hidden", dt, shape, dev),
        _ptr(dhidden, "dhidden", dt, shape, dev), _ptr(dout, "dout", dt, shape, dev),
        _ptr(gamma_post, "gamma_post", f32, vec, dev), _gates(gate, rows, width, per, dev, "gate"),
        _ptr(gamma_pre, "gamma_pre", f32, vec, dev), _ptr(din, "din", dt, shape, dev),
        _ptr(dresidual, "dresidual", dt, shape, dev),
        _ptr(dgamma_post, "dgamma_post", f32, vec, dev),
        _gates(dgate, rows, width, per, dev, "dgate"),
        _ptr(dgamma_pre, "dgamma_pre", f32, vec, dev), rows, width, per,
        (1 if post else 0) | (2 if pre else 0), residual_scale, eps, code)
    ws, nbytes = _workspace(workspace, dev)
    _call_on(dev, stream, _entry, ctypes.byref(a), ws, nbytes)


# ---- linear cross entropy -------------------------------------------------------

def tile_linear_cross_entropy_workspace_bytes(rows, width, vocab):
    if not _fit_int(rows, width, vocab):
        return 0
    return load().tile_linear_cross_entropy_workspace_bytes(rows, width, vocab)


def tile_linear_cross_entropy_backward_workspace_bytes(rows, width, vocab):
    if not _fit_int(rows, width, vocab):
        return 0
    return load().tile_linear_cross_entropy_backward_workspace_bytes(rows, width, vocab)


def _ce_inputs(x, weight, target, ignore_index):
    """(type code, device, x, weight and target pointers, rows, width, vocab)."""
    import torch
    code, dev = _row_code(x, "x"), _device_index(x, "x")
    if code == 0:
        raise ValueError("x must be bfloat16 or float16")
    rows, width = x.shape
    vocab = weight.shape[0]
    if not _fit_int(rows, width, vocab):
        raise ValueError(f"rows, width and vocab must be below 2^31, not {rows}, {width}, {vocab}")
    if not -1 << 63 <= ignore_index < 1 << 63:
        raise ValueError("ignore_index must be a 64-bit integer, as the targets are")
    return (code, dev, _ptr(x, "x", x.dtype, x.shape, dev),
            _ptr(weight, "weight", x.dtype, (vocab, width), dev),
            _ptr(target, "target", torch.int64, (rows,), dev), rows, width, vocab)


def tile_test_linear_cross_entropy_wait_timeout(*args, **kwargs):
    """Test hook: ``tile_linear_cross_entropy`` with a copy withheld, so that
    its waits give up (see include/tile_rows.h)."""
    tile_linear_cross_entropy(*args, **kwargs,
                              _entry="tile_test_linear_cross_entropy_wait_timeout")


def tile_linear_cross_entropy(x, weight, target, loss, lse, workspace, ignore_index=-100,
                              stream=None, _entry="tile_linear_cross_entropy"):
    """loss and log-sum-exp of the rows' logits x weight^T (bfloat16 or
    float16) without keeping them; see include/tile_rows.h."""
    import torch
    code, dev, px, pw, pt, rows, width, vocab = _ce_inputs(x, weight, target, ignore_index)
    ws, nbytes = _workspace(workspace, dev)
    _call_on(dev, stream, _entry, code, px, pw, pt,
             _ptr(loss, "loss", torch.float32, (rows,), dev),
             _ptr(lse, "lse", torch.float32, (rows,), dev), rows, width, vocab, ignore_index, ws,
             nbytes)


def tile_linear_cross_entropy_backward(x, weight, target, lse, dloss, dx, dweight, workspace,
                                       ignore_index=-100, stream=None):
    """Gradients of ``tile_linear_cross_entropy`` for the gradient ``dloss``
    of each row's loss; ``dx`` or ``dweight`` may be None."""
    import torch
    code, dev, px, pw, pt, rows, width, vocab = _ce_inputs(x, weight, target, ignore_index)
    ws, nbytes = _workspace(workspace, dev)
    _call_on(dev, stream, "tile_linear_cross_entropy_backward", code, px, pw, pt,
             _ptr(lse, "lse", torch.float32, (rows,), dev),
             _ptr(dloss, "dloss", torch.float32, (rows,), dev),
             _ptr(dx, "dx", x.dtype, x.shape, dev),
             _ptr(dweight, "dweight", x.dtype, weight.shape, dev), rows, width, vocab,
             ignore_index, ws, nbytes)


# ---- embedding -----------------------------------------------------------------

_F32 = _I64 = _F8 = None     # torch dtypes, filled with _CODES


def _kinds():
    """The torch dtypes above, on first use."""
    global _F32, _I64, _F8
    import torch
    _CODES.update({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2})
    _I64, _F8, _F32 = torch.int64, torch.float8_e4m3fn, torch.float32


def _rows_of(t, name):
    """(type code, device index) of a 2-D row tensor on a device."""
    if _F32 is None:
        _kinds()
    code = _CODES.get(getattr(t, "dtype", None))
    if code is None or t.dim() != 2 or not t.is_cuda:
        _row_code(t, name)
        _device_index(t, name)
    return code, t.get_device()


def _long(value, name):
    if not -0x8000000000000000 <= value <= 0x7fffffffffffffff:
        raise ValueError(f"{name} must be a 64-bit integer")
    return value


def tile_embedding(tokens, weight, out, scale=1.0, ignore_index=-100, stream=None):
    """out[i] = scale * weight[tokens[i]] (float32, bfloat16 or float16); see
    include/tile_rows.h."""
    code, dev = _rows_of(weight, "weight")
    shape, dtype = weight.shape, weight.dtype
    vocab, width = shape
    rows = tokens.shape[0] if tokens.dim() == 1 else -1
    if not _fit_int(rows, width, vocab):
        raise ValueError("tokens must be 1-D, and rows, width and vocab below 2^31")
    _call_on(dev, stream, "tile_embedding", code, _ptr(tokens, "tokens", _I64, (rows,), dev),
             _ptr(weight, "weight", dtype, shape, dev),
             _ptr(out, "out", dtype, (rows, width), dev), rows, width, vocab, scale,
             _long(ignore_index, "ignore_index"))


def tile_embedding_backward_workspace_bytes(rows, width, vocab):
    if not _fit_int(rows, width, vocab):
        return 0
    return load().tile_embedding_backward_workspace_bytes(rows, width, vocab)


def tile_embedding_backward(tokens, dout, dweight, workspace, scale=1.0, ignore_index=-100,
                            accumulate=False, stream=None):
    """dweight = (or, with ``accumulate``, +=) the gradient of
    ``tile_embedding``'s weight; dweight may be float32 for 16-bit rows, and
    workspace None where none is needed (0 bytes)."""
    code, dev = _rows_of(dout, "dout")
    into, _ = _rows_of(dweight, "dweight")
    rows, width = dout.shape
    vocab = dweight.shape[0]
    if not _fit_int(rows, width, vocab):
        raise ValueError(f"rows, width and vocab must be below 2^31, not {rows}, {width}, {vocab}")
    ws, nbytes = (None, 0) if workspace is None else _workspace(workspace, dev)
    _call_on(dev, stream, "tile_embedding_backward", code, into,
             _ptr(tokens, "tokens", _I64, (rows,), dev),
             _ptr(dout, "dout", dout.dtype, dout.shape, dev),
             _ptr(dweight, "dweight", dweight.dtype, (vocab, width), dev), rows, width, vocab,
             scale, _long(ignore_index, "ignore_index"), 1 if accumulate else 0, ws, nbytes)


# ---- policy loss -----------------------------------------------------------------

def tile_policy_loss_workspace_bytes(rows, sequences):
    if not _fit_int(rows, sequences):
        return 0
    return load().tile_policy_loss_workspace_bytes(rows, sequences)


def _policy_args(nll, old_nll, advantage, ref_nll, target, offsets, clip_low, clip_high, kl_coef,
                 sequence_advantage, sequence_mean, ignore_index):
    """(argument struct, device index, shape of nll, sequences)."""
    if _F32 is None:
        _kinds()
    dev, f32 = _device_index(nll, "nll"), _F32
    if nll.dim() != 1:
        raise ValueError("nll must be 1-D")
    shape = nll.shape
    rows = shape[0]
    sequences = 1 if offsets is None else offsets.numel() - 1
    if not _fit_int(rows, sequences) or sequences < 1:
        raise ValueError("offsets must have at least two elements, and rows be below 2^31")
    a = TilePolicyLossArgs(
        _ptr(nll, "nll", f32, shape, dev), _ptr(old_nll, "old_nll", f32, shape, dev),
        _ptr(ref_nll, "ref_nll", f32, shape, dev),
        _ptr(advantage, "advantage", f32, (sequences,) if sequence_advantage else shape, dev),
        _ptr(target, "target", _I64, shape, dev),
        _ptr(offsets, "offsets", _I64, (sequences + 1,), dev),
        _long(ignore_index, "ignore_index"), rows, sequences,
        (1 if sequence_advantage else 0) | (2 if sequence_mean else 0), clip_low, clip_high,
        kl_coef)
    return a, dev, shape, sequences


def tile_policy_loss(nll, old_nll, advantage, stats, weights, workspace, ref_nll=None, target=None,
                     offsets=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0,
                     sequence_advantage=False, sequence_mean=False, ignore_index=-100, stream=None):
    """stats (loss, clipped term, KL term, clipped share) and the token weights
    of each sequence; see ``tile_policy_loss`` in include/tile_rows.h."""
    a, dev, _, sequences = _policy_args(nll, old_nll, advantage, ref_nll, target, offsets, clip_low,
                                        clip_high, kl_coef, sequence_advantage, sequence_mean,
                                        ignore_index)
    ws, nbytes = _workspace(workspace, dev)
    _call_on(dev, stream, "tile_policy_loss", ctypes.byref(a),
             _ptr(stats, "stats", _F32, (4,), dev),
             _ptr(weights, "weights", _F32, (sequences,), dev), ws, nbytes)


def tile_policy_loss_backward(nll, old_nll, advantage, weights, dnll, dloss=None, ref_nll=None,
                              target=None, offsets=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0,
                              sequence_advantage=False, ignore_index=-100, stream=None):
    """dnll of ``tile_policy_loss`` for the gradient ``dloss`` of stats[0] (one
    element on the device; None: 1)."""
    a, dev, shape, sequences = _policy_args(nll, old_nll, advantage, ref_nll, target, offsets,
                                            clip_low, clip_high, kl_coef, sequence_advantage, False,
                                            ignore_index)
    _call_on(dev, stream, "tile_policy_loss_backward", ctypes.byref(a),
             _ptr(weights, "weights", _F32, (sequences,), dev), _one(dloss, "dloss", _F32, dev),
             _ptr(dnll, "dnll", _F32, shape, dev))


def _one(t, name, dtype, dev):
    """Pointer of a CUDA tensor of one element, of any number of dimensions."""
    if t is None:
        return None
    if t.numel() != 1:
        raise ValueError(f"{name} must have one element")
    return _ptr(t, name, dtype, t.shape, dev)


# ---- gradient norm and AdamW step --------------------------------------------------
#
# A small model has hundreds of tensors of which a call takes five lists: each
# list is gone through once by one expression a tensor, and only a tensor that
# fails it is looked at again for the message.

_DTYPE_OF = operator.attrgetter("dtype")


def _columns(tensors, name, types, counts, dev):
    """(pointers, element counts, types) of a list of contiguous CUDA tensors
    on device index ``dev``, of types that ``types`` has codes for and of these
    element counts (None: any)."""
    if hasattr(tensors, "dtype"):
        raise TypeError(f"{name} must be a list of tensors")
    if counts is not None and len(tensors) != len(counts):
        raise ValueError(f"{name} must have {len(counts)} tensors like the other lists, "
                         f"not {len(tensors)}")
    try:
        sizes = [t.numel() for t in tensors] if counts is None else counts
        kind = tensors[0].dtype if len(tensors) else None
        pointers = [t.data_ptr() for t, n in zip(tensors, sizes)
                    if t.dtype is kind and t.numel() == n and t.get_device() == dev
                    and t.is_contiguous()] if kind in types else []
        if len(pointers) == len(sizes):
            return pointers, sizes, [kind] * len(sizes)
        # of several types
        kinds = list(map(_DTYPE_OF, tensors))
        pointers = [t.data_ptr() for t, n in zip(tensors, sizes)
                    if t.numel() == n and t.get_device() == dev and t.is_contiguous()]
        if types.keys() >= set(kinds) and len(pointers) == len(sizes):
            return pointers, sizes, kinds
    except AttributeError:
        pass
    _list_of_tensors(tensors, name)
    for i, t in enumerate(tensors):
        if t.dtype not in types:
            raise ValueError(f"{name}[{i}] must be one of {sorted(map(str, types))}, not {t.dtype}")
        if counts is not None and t.numel() != counts[i]:
            raise ValueError(f"{name}[{i}] must have {counts[i]} elements, not {t.numel()}")
        _ptr(t, f"{name}[{i}]", t.dtype, t.shape, dev)
    raise ValueError(f"{name} must be CUDA tensors of one device")


def _list_of_tensors(tensors, name):
    import torch
    if isinstance(tensors, torch.Tensor):
        raise TypeError(f"{name} must be a list of tensors")
    for i, t in enumerate(tensors):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}[{i}] must be a torch.Tensor")


def _list_device(tensors, name):
    """Device index of the first tensor of a list, None of an empty one."""
    import torch
    if isinstance(tensors, torch.Tensor) or not len(tensors) or \
            not isinstance(tensors[0], torch.Tensor):
        _list_of_tensors(tensors, name)
        return None
    return _device_index(tensors[0], f"{name}[0]")


def _records(form, count, columns):
    """C structs of one format from columns of their fields."""
    return struct.pack(form * count, *itertools.chain.from_iterable(zip(*columns)))


def tile_grad_norm_workspace_bytes(count):
    return load().tile_grad_norm_workspace_bytes(count) if _fit_int(count) else 0


def tile_grad_norm(grads, out, workspace, scale=1.0, max_norm=None, stream=None):
    """out = (norm, clipping factor) of all ``grads`` together (float32,
    bfloat16 or float16, in any mix); see include/tile_rows.h."""
    if _F32 is None:
        _kinds()
    dev = _device_index(out, "out")
    p, n, kinds = _columns(grads, "grads", _CODES, None, dev)
    table = _records("2qi4x", len(p), (p, n, [_CODES[k] for k in kinds]))
    ws, nbytes = _workspace(workspace, dev)
    _call_on(dev, stream, "tile_grad_norm", table, len(p), scale,
             _INF if max_norm is None else max_norm, _ptr(out, "out", _F32, (2,), dev), ws, nbytes)


def tile_adamw(params, grads, exp_avg, exp_avg_sq, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8,
               weight_decay=0.01, factor=None, copies=None, exp_avg_scales=None,
               exp_avg_sq_scales=None, seed=0, stream=None):
    """One AdamW step of every tensor of ``params`` (float32), in place, with
    its state; see ``tile_adamw`` in include/tile_rows.h.  Lists of one length:
    ``grads`` (float32, bfloat16 or float16), the states (float32, or
    float8_e4m3fn with the scales), and, where wanted, ``copies`` (bfloat16 or
    float16, None for a parameter without one).  ``step`` (from 1 on) and ``lr`` are numbers, or tensors of one
    element on the device (int64, float32); ``weight_decay`` a number or one
    for each tensor; ``factor`` ``tile_grad_norm``'s second output."""
    if _F32 is None:
        _kinds()
    dev, count = _list_device(params, "params"), len(params)
    f32 = {_F32: 0}
    p, n, _ = _columns(params, "params", f32, None, dev)
    g, _, kinds = _columns(grads, "grads", _CODES, n, dev)
    eight = count > 0 and len(exp_avg) > 0 and getattr(exp_avg[0], "dtype", None) is _F8
    state = {_F8: 0} if eight else f32
    m, _, _ = _columns(exp_avg, "exp_avg", state, n, dev)
    v, _, _ = _columns(exp_avg_sq, "exp_avg_sq", state, n, dev)
    ms = vs = c = copy_kinds = [0] * count
    if eight:
        if exp_avg_scales is None or exp_avg_sq_scales is None:
            raise ValueError("8-bit states need exp_avg_scales and exp_avg_sq_scales")
        blocks = [-(-k // 256) for k in n]
        ms, _, _ = _columns(exp_avg_scales, "exp_avg_scales", f32, blocks, dev)
        vs, _, _ = _columns(exp_avg_sq_scales, "exp_avg_sq_scales", f32, blocks, dev)
    elif count > 0 and (exp_avg_scales is not None or exp_avg_sq_scales is not None):
        raise ValueError("scales belong to 8-bit states")
    if copies is not None:
        if hasattr(copies, "dtype") or len(copies) != count:
            raise ValueError(f"copies must be a list of {count} tensors or None")
        halves = {k: i for k, i in _CODES.items() if i != 0}
        which = [i for i, t in enumerate(copies) if t is not None]
        at, _, types = _columns([copies[i] for i in which], "copies", halves,
                                [n[i] for i in which], dev)
        c, copy_kinds = [0] * count, [0] * count
        for i, a, k in zip(which, at, types):
            c[i], copy_kinds[i] = a, halves[k]
    decay = [weight_decay] * count if isinstance(weight_decay, (int, float)) else weight_decay
    if len(decay) != count:
        raise ValueError(f"weight_decay must be a number or {count} of them")
    if count == 0:
        return
    table = _records("8qf2i4x", count, (p, g, m, v, ms, vs, c, n, decay,
                                        [_CODES[k] for k in kinds], copy_kinds))
    step_at, lr_at = getattr(step, "is_cuda", None), getattr(lr, "is_cuda", None)
    config = TileAdamwConfig(
        lr if lr_at is None else 0.0, betas[0], betas[1], eps,
        _long(step, "step") if step_at is None else 0,
        None if lr_at is None else _one(lr, "lr", _F32, dev),
        None if step_at is None else _one(step, "step", _I64, dev),
        _one(factor, "factor", _F32, dev), seed & 0xFFFFFFFFFFFFFFFF, 1 if eight else 0)
    _call_on(dev, stream, "tile_adamw", table, count, ctypes.byref(config))


# ---------------------------------------------------------------------------
# convenience wrappers (allocate the output with torch when not given)
# ---------------------------------------------------------------------------

def residual_layernorm(x, residual, out=None, eps=1e-5, stream=None):
    import torch
    out = torch.empty_like(x) if out is None else out
    tile_residual_layernorm_f32(x, residual, out, eps, stream)
    return out


def layernorm(x, out=None, eps=1e-5, stream=None):
    import torch
    out = torch.empty_like(x) if out is None else out
    tile_layernorm_f32(x, out, eps, stream)
    return out


def rmsnorm(x, out=None, eps=1e-5, stream=None):
    import torch
    out = torch.empty_like(x) if out is None else out
    tile_rmsnorm_f32(x, out, eps, stream)
    return out


def softmax(x, out=None, stream=None):
    import torch
    out = torch.empty_like(x) if out is None else out
    tile_softmax_f32(x, out, 0.0, stream)
    return out


def _on_stream(fn):
    """A wrapper that allocates runs with its ``stream`` current, so that what
    it allocates belongs to the stream its kernels run on.  The stream is one
    of the tensors' device, which need not be the current one."""
    import functools

    @functools.wraps(fn)
    def call(*args, stream=None, **kwargs):
        if stream is None:
            return fn(*args, **kwargs)
        import torch
        dev = next((t.get_device() for a in (*args, *kwargs.values())
                    for t in (a if isinstance(a, (list, tuple)) else (a,))
                    if isinstance(t, torch.Tensor) and t.is_cuda), None)
        if dev is None:
            raise ValueError(f"{fn.__name__} takes CUDA tensors (there is no CPU path)")
        _same_device(stream, dev)
        s = torch.cuda.ExternalStream(stream, device=dev) if isinstance(stream, int) else stream
        with torch.cuda.stream(s):
            return fn(*args, **kwargs)
    return call


def _scratch(nbytes, like):
    import torch
    return torch.empty(nbytes or 1, dtype=torch.uint8, device=like.device)


@_on_stream
def block_norm(x, residual, gamma_post=None, gate=None, gamma_pre=None, post=True, pre=True,
               rows_per_gate=0, residual_scale=1.0, eps=1e-5):
    """(hidden, out) of ``tile_block_norm``; out is None without ``pre``."""
    import torch
    hidden = torch.empty_like(x)
    out = torch.empty_like(x) if pre else None
    tile_block_norm(x, residual, hidden, out, gamma_post, gate, gamma_pre, post, pre,
                    rows_per_gate, residual_scale, eps)
    return hidden, out


@_on_stream
def block_norm_backward(x, hidden, gamma_post, gate, gamma_pre, dhidden, dout, post=True,
                        pre=True, rows_per_gate=0, residual_scale=1.0, eps=1e-5):
    """(din, dresidual, dgamma_post, dgate, dgamma_pre) of
    ``tile_block_norm_backward``; the gradients of parameters that are None
    are None."""
    import torch
    like = hidden if hidden is not None else dhidden
    if like is None:
        raise ValueError("hidden (with pre) or dhidden (without) must be a CUDA tensor")
    din, dresidual = torch.empty_like(like), torch.empty_like(like)
    dgamma_post = torch.empty_like(gamma_post) if post and gamma_post is not None else None
    dgate = torch.empty_like(gate) if gate is not None else None
    dgamma_pre = torch.empty_like(gamma_pre) if pre and gamma_pre is not None else None
    gate_rows = 0 if gate is None else 1 if gate.dim() == 1 else gate.shape[0]
    ws = _scratch(tile_block_norm_backward_gated_workspace_bytes(*like.shape, gate_rows), like)
    tile_block_norm_backward(x, hidden, dhidden, dout, din, dresidual, ws, gamma_post, gate,
                             gamma_pre, dgamma_post, dgate, dgamma_pre, post, pre, rows_per_gate,
                             residual_scale, eps)
    return din, dresidual, dgamma_post, dgate, dgamma_pre


@_on_stream
def linear_cross_entropy(x, weight, target, ignore_index=-100):
    """(loss, lse) of ``tile_linear_cross_entropy``, float32, one per row."""
    import torch
    rows, width = x.shape
    loss = torch.empty(rows, dtype=torch.float32, device=x.device)
    lse = torch.empty_like(loss)
    ws = _scratch(tile_linear_cross_entropy_workspace_bytes(rows, width, weight.shape[0]), x)
    tile_linear_cross_entropy(x, weight, target, loss, lse, ws, ignore_index)
    return loss, lse


@_on_stream
def linear_cross_entropy_backward(x, weight, target, lse, dloss, ignore_index=-100,
                                  need_dx=True, need_dweight=True):
    """(dx, dweight) of ``tile_linear_cross_entropy_backward``."""
    import torch
    rows, width = x.shape
    dx = torch.empty_like(x) if need_dx else None
    dweight = torch.empty_like(weight) if need_dweight else None
    ws = _scratch(tile_linear_cross_entropy_backward_workspace_bytes(rows, width,
                                                                     weight.shape[0]), x)
    tile_linear_cross_entropy_backward(x, weight, target, lse, dloss, dx, dweight, ws,
                                       ignore_index)
    return dx, dweight


@_on_stream
def embedding(tokens, weight, scale=1.0, ignore_index=-100):
    """scale * weight[tokens], rows of zeros where a token is ignore_index."""
    import torch
    _rows_of(weight, "weight")
    out = torch.empty((tokens.shape[0], weight.shape[1]), dtype=weight.dtype, device=weight.device)
    tile_embedding(tokens, weight, out, scale, ignore_index)
    return out


@_on_stream
def embedding_backward(tokens, dout, vocab=None, scale=1.0, ignore_index=-100, dtype=None,
                       dweight=None):
    """The gradient of ``embedding``'s weight: a new [vocab, width] tensor (of
    dout's type, or ``dtype`` float32), or added to ``dweight``, which is
    returned (say, what ``linear_cross_entropy_backward`` left for a weight that
    the head shares)."""
    import torch
    add = dweight is not None
    if add:
        if vocab not in (None, dweight.shape[0]) or dtype not in (None, dweight.dtype):
            raise ValueError("vocab and dtype are those of dweight")
    elif vocab is None:
        raise ValueError("vocab or dweight is needed")
    else:
        dweight = torch.empty(vocab, dout.shape[1], dtype=dtype or dout.dtype, device=dout.device)
    need = tile_embedding_backward_workspace_bytes(*dout.shape, dweight.shape[0])
    tile_embedding_backward(tokens, dout, dweight, _scratch(need, dout) if need else None, scale,
                            ignore_index, add)
    return dweight


def _mean_of(mean):
    if mean not in ("token", "sequence"):
        raise ValueError('mean must be "token" or "sequence"')
    return mean == "sequence"


@_on_stream
def policy_loss(nll, old_nll, advantage, ref_nll=None, target=None, offsets=None,
                per_sequence=False, clip_low=0.2, clip_high=0.2, kl_coef=0.0, mean="token",
                ignore_index=-100):
    """(stats, weights) of ``tile_policy_loss``: stats[0] is the loss, and
    ``policy_loss_backward`` takes the weights.  ``per_sequence``: an advantage
    for each sequence; ``mean``: over "token"s or over each "sequence"'s mean."""
    import torch
    sequences = 1 if offsets is None else offsets.numel() - 1
    stats = torch.empty(4, dtype=torch.float32, device=nll.device)
    weights = torch.empty(max(sequences, 0), dtype=torch.float32, device=nll.device)
    ws = _scratch(tile_policy_loss_workspace_bytes(nll.shape[0], sequences), nll)
    tile_policy_loss(nll, old_nll, advantage, stats, weights, ws, ref_nll, target, offsets,
                     clip_low, clip_high, kl_coef, per_sequence, _mean_of(mean), ignore_index)
    return stats, weights


@_on_stream
def policy_loss_backward(nll, old_nll, advantage, weights, dloss=None, ref_nll=None, target=None,
                         offsets=None, per_sequence=False, clip_low=0.2, clip_high=0.2,
                         kl_coef=0.0, ignore_index=-100):
    """dnll of ``tile_policy_loss_backward``: the ``dloss`` of
    ``linear_cross_entropy_backward``."""
    import torch
    dnll = torch.empty_like(nll)
    tile_policy_loss_backward(nll, old_nll, advantage, weights, dnll, dloss, ref_nll, target,
                              offsets, clip_low, clip_high, kl_coef, per_sequence, ignore_index)
    return dnll


@_on_stream
def grad_norm(grads, max_norm=None, scale=1.0):
    """(norm, clipping factor) of all ``grads`` together as a tensor of two;
    ``adamw`` takes its second element as ``factor``."""
    import torch
    if _list_device(grads, "grads") is None:
        raise ValueError("grads is empty")
    out = torch.empty(2, dtype=torch.float32, device=grads[0].device)
    tile_grad_norm(grads, out, _scratch(tile_grad_norm_workspace_bytes(len(grads)), out), scale,
                   max_norm)
    return out


def adamw(params, grads, exp_avg, exp_avg_sq, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8,
          weight_decay=0.01, factor=None, copies=None, exp_avg_scales=None,
          exp_avg_sq_scales=None, seed=0, stream=None):
    """``tile_adamw``; ``adamw_state`` makes the states."""
    tile_adamw(params, grads, exp_avg, exp_avg_sq, step, lr, betas, eps, weight_decay, factor,
               copies, exp_avg_scales, exp_avg_sq_scales, seed, stream)


def adamw_state(params, bits=32):
    """Zero states of ``adamw`` for these parameters: the keyword arguments
    exp_avg and exp_avg_sq, and with ``bits`` 8 their scales."""
    import torch
    if bits not in (8, 32):
        raise ValueError("states have 8 or 32 bits")
    kind = torch.float32 if bits == 32 else torch.float8_e4m3fn

    def zeros(blocks=None):
        return [torch.zeros(p.shape if blocks is None else -(-p.numel() // blocks),
                            dtype=kind if blocks is None else torch.float32, device=p.device)
                for p in params]
    state = {"exp_avg": zeros(), "exp_avg_sq": zeros()}
    if bits == 8:
        state.update(exp_avg_scales=zeros(256), exp_avg_sq_scales=zeros(256))
    return state


def run(op, x, residual=None, out=None, eps=1e-5, stream=None):
    """Dispatch by op name."""
    if op == "residual_layernorm":
        return residual_layernorm(x, residual, out, eps, stream)
    if op == "softmax":
        return softmax(x, out, stream)
    return {"layernorm": layernorm, "rmsnorm": rmsnorm}[op](x, out, eps, stream)
