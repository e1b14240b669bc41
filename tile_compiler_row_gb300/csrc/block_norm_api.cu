// C ABI of the block norm (include/tile_rows.h): argument checks and dispatch.
#include <cmath>

#include "../../include/tile_rows.h"
#include "block_norm.cuh"
#include "host_checks.h"
#include "plans.h"

namespace {

using tile::cuda_status;
using tile::elem_size;
using tile::misaligned_to;
using tile::Range;

bool valid_dtype(int dtype) {
    return dtype == TILE_DTYPE_F32 || dtype == TILE_DTYPE_BF16 || dtype == TILE_DTYPE_F16;
}

tile::BlockAccess access_of(const void *const *mats, int nmats, const void *const *params,
                            int nparams, int width, size_t es) {
    for (int i = 0; i < nmats; ++i)
        if (misaligned_to(mats[i], 16)) return tile::ACCESS_ELEMENTS;
    if (static_cast<size_t>(width) * es % 16 != 0) return tile::ACCESS_SHIFTED;
    // the FP32 parameters of 16 bytes of a row are one load
    for (int i = 0; i < nparams; ++i)
        if (misaligned_to(params[i], 64 / es)) return tile::ACCESS_SHIFTED;
    return tile::ACCESS_VECTORS;
}

bool any_misaligned(const void *const *p, int n, size_t to) {
    for (int i = 0; i < n; ++i)
        if (misaligned_to(p[i], to)) return true;
    return false;
}

// The checks that forward and backward share.
int check_shape(int norms, int dtype, int rows, int width, const float *gate, int rows_per_gate,
                float scale, float eps) {
    if (norms < 1 || norms > (TILE_NORM_POST | TILE_NORM_PRE)) return TILE_ERR_OP;
    if (!valid_dtype(dtype)) return TILE_ERR_DTYPE;
    if (rows < 0 || width < 1 || width > TILE_MAX_WIDTH) return TILE_ERR_SHAPE;
    if (gate != nullptr && rows_per_gate < 1) return TILE_ERR_SHAPE;
    if (!(std::isfinite(eps) && eps >= 0.0f) || !std::isfinite(scale)) return TILE_ERR_EPS;
    return TILE_OK;
}

}  // namespace

extern "C" {

int tile_block_norm(const tile_block_norm_args_t *args, cudaStream_t stream) {
    if (args == nullptr) return TILE_ERR_NULL;
    const tile_block_norm_args_t &c = *args;
    const int st = check_shape(c.norms, c.dtype, c.rows, c.width, c.gate, c.rows_per_gate,
                               c.residual_scale, c.eps);
    if (st != TILE_OK) return st;
    if (c.rows == 0) return TILE_OK;
    const bool post = (c.norms & TILE_NORM_POST) != 0, pre = (c.norms & TILE_NORM_PRE) != 0;
    if (c.in == nullptr || c.residual == nullptr || c.hidden == nullptr ||
        (pre && c.out == nullptr))
        return TILE_ERR_NULL;
    tile::BlockArgs a = {};
    a.x = c.in;
    a.residual = c.residual;
    a.gamma_post = post ? c.gamma_post : nullptr;
    a.gate = c.gate;
    a.gamma_pre = pre ? c.gamma_pre : nullptr;
    a.hidden_out = c.hidden;
    a.out = pre ? c.out : nullptr;
    a.rows = c.rows;
    a.per_gate = c.gate != nullptr ? c.rows_per_gate : c.rows;
    a.width = c.width;
    a.post = post;
    a.pre = pre;
    a.scale = c.residual_scale;
    a.eps = c.eps;
    const size_t es = elem_size(c.dtype);
    const void *mats[] = {a.x, a.residual, a.hidden_out, a.out};
    const void *params[] = {a.gamma_post, a.gate, a.gamma_pre};
    if (any_misaligned(mats, 4, es) || any_misaligned(params, 3, sizeof(float)))
        return TILE_ERR_ALIGN;
    const size_t vec = static_cast<size_t>(c.width) * sizeof(float);
    const size_t mat = static_cast<size_t>(c.rows) * static_cast<size_t>(c.width) * es;
    const size_t gates = static_cast<size_t>((a.rows + a.per_gate - 1) / a.per_gate);
    const Range out[] = {{a.hidden_out, mat}, {a.out, mat}};
    const Range in[] = {{a.x, mat}, {a.residual, mat}, {a.gamma_post, vec},
                        {a.gate, gates * vec}, {a.gamma_pre, vec}};
    if (tile::any_overlap(out, 2, in, 5)) return TILE_ERR_ALIAS;
    const cudaError_t inj = tile::injected_launch_failure();
    if (inj != cudaSuccess) return cuda_status(inj);
    return cuda_status(tile::launch_block_norm(
        c.dtype, access_of(mats, 4, params, 3, c.width, es), a, stream));
}

size_t tile_block_norm_backward_workspace_bytes(int rows, int width) {
    if (rows < 1 || width < 1 || width > TILE_MAX_WIDTH) return 0;
    return tile::block_norm_backward_workspace(rows, width, rows);
}

size_t tile_block_norm_backward_gated_workspace_bytes(int rows, int width, int gate_rows) {
    if (rows < 1 || width < 1 || width > TILE_MAX_WIDTH || gate_rows < 0) return 0;
    const int gates = gate_rows < 1 ? 1 : gate_rows > rows ? rows : gate_rows;
    return tile::block_norm_backward_workspace(rows, width, gates);
}

}  // extern "C"

namespace {

int run_backward(const tile_block_norm_backward_args_t *args, void *workspace,
                 size_t workspace_bytes, bool withheld, cudaStream_t stream) {
    if (args == nullptr) return TILE_ERR_NULL;
    const tile_block_norm_backward_args_t &c = *args;
    const int st = check_shape(c.norms, c.dtype, c.rows, c.width, c.gate, c.rows_per_gate,
                               c.residual_scale, c.eps);
    if (st != TILE_OK) return st;
    const bool post = (c.norms & TILE_NORM_POST) != 0, pre = (c.norms & TILE_NORM_PRE) != 0;
    if ((c.dgamma_post != nullptr && !post) || (c.dgamma_pre != nullptr && !pre) ||
        (c.dgate != nullptr && c.gate == nullptr))
        return TILE_ERR_OP;
    const size_t vec = static_cast<size_t>(c.width) * sizeof(float);
    const void *params[] = {c.gamma_post, c.gate, c.gamma_pre, c.dgamma_post, c.dgate,
                            c.dgamma_pre};
    if (any_misaligned(params, 6, sizeof(float))) return TILE_ERR_ALIGN;
    if (c.rows == 0) {   // no rows: the sums are zero (a gate of no rows has none)
        const cudaError_t inj = tile::injected_launch_failure();
        cudaError_t err = inj;
        for (float *p : {c.dgamma_post, c.dgamma_pre})
            if (p != nullptr && err == cudaSuccess) err = cudaMemsetAsync(p, 0, vec, stream);
        return cuda_status(err);
    }
    const bool uses_x = post || c.gate != nullptr;
    if (c.din == nullptr || c.dresidual == nullptr || (uses_x && c.in == nullptr) ||
        (pre && (c.hidden == nullptr || c.dout == nullptr)) ||
        (!pre && c.dhidden == nullptr) || workspace == nullptr)
        return TILE_ERR_NULL;
    tile::BlockArgs a = {};
    a.x = uses_x ? c.in : nullptr;
    a.hidden = pre ? c.hidden : nullptr;
    a.dhidden = c.dhidden;
    a.dout = pre ? c.dout : nullptr;
    a.gamma_post = post ? c.gamma_post : nullptr;
    a.gate = c.gate;
    a.gamma_pre = pre ? c.gamma_pre : nullptr;
    a.din = c.din;
    a.dresidual = c.dresidual;
    a.dgamma_post = c.dgamma_post;
    a.dgate = c.dgate;
    a.dgamma_pre = c.dgamma_pre;
    a.ws = static_cast<float *>(workspace);
    a.rows = c.rows;
    a.per_gate = c.gate != nullptr ? c.rows_per_gate : c.rows;
    a.width = c.width;
    a.post = post;
    a.pre = pre;
    a.scale = c.residual_scale;
    a.eps = c.eps;
    const size_t es = elem_size(c.dtype);
    const void *mats[] = {a.x, a.hidden, a.dhidden, a.dout, a.din, a.dresidual};
    if (any_misaligned(mats, 6, es) || misaligned_to(workspace, 16)) return TILE_ERR_ALIGN;
    const size_t gates = static_cast<size_t>((a.rows + a.per_gate - 1) / a.per_gate);
    const size_t need = tile::block_norm_backward_workspace(a.rows, a.width, gates);
    if (workspace_bytes < need) return TILE_ERR_WORKSPACE;
    const size_t mat = static_cast<size_t>(c.rows) * static_cast<size_t>(c.width) * es;
    const Range out[] = {{a.din, mat}, {a.dresidual, mat}, {a.dgamma_post, vec},
                         {a.dgate, gates * vec}, {a.dgamma_pre, vec}, {workspace, need}};
    const Range in[] = {{a.x, mat}, {a.hidden, mat}, {a.dhidden, mat}, {a.dout, mat},
                        {a.gamma_post, vec}, {a.gate, gates * vec}, {a.gamma_pre, vec}};
    if (tile::any_overlap(out, 6, in, 7)) return TILE_ERR_ALIAS;
    const cudaError_t inj = tile::injected_launch_failure();
    if (inj != cudaSuccess) return cuda_status(inj);
    a.withheld = withheld;
    const cudaError_t err = tile::launch_block_norm_backward(
        c.dtype, access_of(mats, 6, params, 3, c.width, es), a, stream);
    return withheld && err == cudaErrorNotSupported ? TILE_ERR_PLAN : cuda_status(err);
}

}  // namespace

extern "C" {

int tile_block_norm_backward(const tile_block_norm_backward_args_t *args, void *workspace,
                             size_t workspace_bytes, cudaStream_t stream) {
    return run_backward(args, workspace, workspace_bytes, false, stream);
}

int tile_test_block_norm_backward_wait_timeout(const tile_block_norm_backward_args_t *args,
                                               void *workspace, size_t workspace_bytes,
                                               cudaStream_t stream) {
    return run_backward(args, workspace, workspace_bytes, true, stream);
}

}  // extern "C"
