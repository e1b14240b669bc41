// C ABI of the linear cross entropy (include/tile_rows.h): argument checks
// and dispatch.
#include "../../include/tile_rows.h"
#include "host_checks.h"
#include "launch.h"
#include "linear_ce.h"
#include "plans.h"

namespace {

using tile::cuda_status;
using tile::misaligned_to;
using tile::Range;

int check_shape(int dtype, int rows, int width, int vocab) {
    if (dtype != TILE_DTYPE_BF16 && dtype != TILE_DTYPE_F16) return TILE_ERR_DTYPE;
    if (rows < 0 || width < 1 || width > TILE_MAX_WIDTH || vocab < 1) return TILE_ERR_SHAPE;
    // tile counts and packed positions are ints
    if (rows > (1 << 30) || vocab > (1 << 30)) return TILE_ERR_SHAPE;
    return TILE_OK;
}

// Rows of a multiple of 8 elements are read as they lie (16-byte aligned);
// others are copied first, from any alignment of the element.
size_t row_alignment(int width) { return width % 8 == 0 ? 16 : 2; }

}  // namespace

extern "C" {

size_t tile_linear_cross_entropy_workspace_bytes(int rows, int width, int vocab) {
    if (rows < 1 || check_shape(TILE_DTYPE_BF16, rows, width, vocab) != TILE_OK) return 0;
    return tile::linear_ce_workspace(rows, width, vocab);
}

size_t tile_linear_cross_entropy_backward_workspace_bytes(int rows, int width, int vocab) {
    if (rows < 1 || check_shape(TILE_DTYPE_BF16, rows, width, vocab) != TILE_OK) return 0;
    return tile::linear_ce_backward_workspace(rows, width, vocab);
}

}  // extern "C"

namespace {

int run_forward(int dtype, const void *in, const void *weight, const long long *target, float *loss,
                float *lse, int rows, int width, int vocab, long long ignore_index, void *workspace,
                size_t workspace_bytes, bool withheld, cudaStream_t stream) {
    const int st = check_shape(dtype, rows, width, vocab);
    if (st != TILE_OK) return st;
    if (rows == 0) return TILE_OK;
    if (in == nullptr || weight == nullptr || target == nullptr || loss == nullptr ||
        lse == nullptr || workspace == nullptr)
        return TILE_ERR_NULL;
    if (misaligned_to(in, row_alignment(width)) || misaligned_to(weight, row_alignment(width)) ||
        misaligned_to(target, 8) || misaligned_to(loss, 4) || misaligned_to(lse, 4) ||
        misaligned_to(workspace, 256))
        return TILE_ERR_ALIGN;
    const size_t need = tile::linear_ce_workspace(rows, width, vocab);
    if (workspace_bytes < need) return TILE_ERR_WORKSPACE;
    const size_t r = static_cast<size_t>(rows), row = static_cast<size_t>(width) * 2;
    const Range out[] = {{loss, r * 4}, {lse, r * 4}, {workspace, need}};
    const Range read[] = {{in, r * row}, {weight, static_cast<size_t>(vocab) * row}, {target, r * 8}};
    if (tile::any_overlap(out, 3, read, 3)) return TILE_ERR_ALIAS;
    const cudaError_t inj = tile::injected_launch_failure();
    if (inj != cudaSuccess) return cuda_status(inj);
    tile::LinearCeArgs a = {};
    a.elem = dtype;
    a.x = in;
    a.weight = weight;
    a.target = target;
    a.ignore = ignore_index;
    a.loss = loss;
    a.lse = lse;
    a.rows = rows;
    a.width = width;
    a.vocab = vocab;
    a.ws = workspace;
    a.withheld = withheld;
    const cudaError_t err = tile::launch_linear_ce(a, stream);
    return withheld && err == cudaErrorNotSupported ? TILE_ERR_PLAN : cuda_status(err);
}

}  // namespace

extern "C" {

int tile_linear_cross_entropy(int dtype, const void *in, const void *weight,
                              const long long *target, float *loss, float *lse, int rows,
                              int width, int vocab, long long ignore_index, void *workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
    return run_forward(dtype, in, weight, target, loss, lse, rows, width, vocab, ignore_index,
                       workspace, workspace_bytes, false, stream);
}

int tile_test_linear_cross_entropy_wait_timeout(int dtype, const void *in, const void *weight,
                                                const long long *target, float *loss, float *lse,
                                                int rows, int width, int vocab,
                                                long long ignore_index, void *workspace,
                                                size_t workspace_bytes, cudaStream_t stream) {
    return run_forward(dtype, in, weight, target, loss, lse, rows, width, vocab, ignore_index,
                       workspace, workspace_bytes, true, stream);
}

int tile_linear_cross_entropy_backward(int dtype, const void *in, const void *weight,
                                       const long long *target, const float *lse,
                                       const float *dloss, void *din, void *dweight, int rows,
                                       int width, int vocab, long long ignore_index,
                                       void *workspace, size_t workspace_bytes,
                                       cudaStream_t stream) {
    const int st = check_shape(dtype, rows, width, vocab);
    if (st != TILE_OK) return st;
    const size_t r = static_cast<size_t>(rows), row = static_cast<size_t>(width) * 2;
    const size_t weight_bytes = static_cast<size_t>(vocab) * row;
    if (misaligned_to(din, 2) || misaligned_to(dweight, 2)) return TILE_ERR_ALIGN;
    if (rows == 0) {   // no rows: the weight's gradient is zero
        const cudaError_t inj = tile::injected_launch_failure();
        if (inj != cudaSuccess) return cuda_status(inj);
        if (dweight == nullptr) return TILE_OK;
        return cuda_status(cudaMemsetAsync(dweight, 0, weight_bytes, stream));
    }
    if (in == nullptr || weight == nullptr || target == nullptr || lse == nullptr ||
        dloss == nullptr || workspace == nullptr || (din == nullptr && dweight == nullptr))
        return TILE_ERR_NULL;
    if (misaligned_to(in, row_alignment(width)) || misaligned_to(weight, row_alignment(width)) ||
        misaligned_to(target, 8) || misaligned_to(lse, 4) || misaligned_to(dloss, 4) ||
        misaligned_to(workspace, 256))
        return TILE_ERR_ALIGN;
    const size_t need = tile::linear_ce_backward_workspace(rows, width, vocab);
    if (workspace_bytes < need) return TILE_ERR_WORKSPACE;
    const Range out[] = {{din, r * row}, {dweight, weight_bytes}, {workspace, need}};
    const Range read[] = {{in, r * row}, {weight, weight_bytes}, {target, r * 8}, {lse, r * 4},
                          {dloss, r * 4}};
    if (tile::any_overlap(out, 3, read, 5)) return TILE_ERR_ALIAS;
    const cudaError_t inj = tile::injected_launch_failure();
    if (inj != cudaSuccess) return cuda_status(inj);
    tile::LinearCeArgs a = {};
    a.elem = dtype;
    a.x = in;
    a.weight = weight;
    a.target = target;
    a.ignore = ignore_index;
    a.lse = const_cast<float *>(lse);
    a.dloss = dloss;
    a.dx = din;
    a.dweight = dweight;
    a.rows = rows;
    a.width = width;
    a.vocab = vocab;
    a.ws = workspace;
    return cuda_status(tile::launch_linear_ce_backward(a, stream));
}

}  // extern "C"
