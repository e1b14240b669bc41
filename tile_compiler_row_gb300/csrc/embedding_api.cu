// C ABI of the embedding lookup and its gradient (include/tile_rows.h):
// argument checks and dispatch.
#include <cmath>

#include "../../include/tile_rows.h"
#include "embedding.h"
#include "host_checks.h"
#include "launch.h"
#include "plans.h"

namespace {

using tile::cuda_status;
using tile::elem_size;
using tile::misaligned_to;
using tile::Range;

bool valid_dtype(int dtype) {
    return dtype == TILE_DTYPE_F32 || dtype == TILE_DTYPE_BF16 || dtype == TILE_DTYPE_F16;
}

int check_shape(int rows, int width, int vocab) {
    if (rows < 0 || width < 1 || width > TILE_MAX_WIDTH || vocab < 1 || vocab > (1 << 30))
        return TILE_ERR_SHAPE;
    return rows > (1 << 24) ? TILE_ERR_SHAPE : TILE_OK;   // (the digit counts of a sort)
}

}  // namespace

extern "C" {

int tile_embedding(int dtype, const long long *tokens, const void *weight, void *out, int rows,
                   int width, int vocab, float scale, long long ignore_index,
                   cudaStream_t stream) {
    if (!valid_dtype(dtype)) return TILE_ERR_DTYPE;
    const int st = check_shape(rows, width, vocab);
    if (st != TILE_OK) return st;
    if (!std::isfinite(scale)) return TILE_ERR_EPS;
    if (rows == 0) return TILE_OK;
    if (tokens == nullptr || weight == nullptr || out == nullptr) return TILE_ERR_NULL;
    const size_t es = elem_size(dtype);
    if (misaligned_to(tokens, 8) || misaligned_to(weight, es) || misaligned_to(out, es))
        return TILE_ERR_ALIGN;
    const size_t r = static_cast<size_t>(rows), row = static_cast<size_t>(width) * es;
    const Range written[] = {{out, r * row}};
    const Range read[] = {{tokens, r * 8}, {weight, static_cast<size_t>(vocab) * row}};
    if (tile::any_overlap(written, 1, read, 2)) return TILE_ERR_ALIAS;
    const cudaError_t inj = tile::injected_launch_failure();
    if (inj != cudaSuccess) return cuda_status(inj);
    tile::EmbeddingArgs a = {};
    a.tokens = tokens;
    a.weight = weight;
    a.out = out;
    a.ignore = ignore_index;
    a.rows = rows;
    a.width = width;
    a.vocab = vocab;
    a.scale = scale;
    const bool vectors = !misaligned_to(weight, 16) && !misaligned_to(out, 16) && row % 16 == 0;
    return cuda_status(tile::launch_embedding(dtype, vectors, a, stream));
}

size_t tile_embedding_backward_workspace_bytes(int rows, int width, int vocab) {
    if (rows < 1 || check_shape(rows, width, vocab) != TILE_OK) return 0;
    return tile::embedding_backward_workspace(rows, width, vocab);
}

int tile_embedding_backward(int dtype, int dweight_dtype, const long long *tokens,
                            const void *dout, void *dweight, int rows, int width, int vocab,
                            float scale, long long ignore_index, int accumulate, void *workspace,
                            size_t workspace_bytes, cudaStream_t stream) {
    if (!valid_dtype(dtype) || (dweight_dtype != dtype && dweight_dtype != TILE_DTYPE_F32))
        return TILE_ERR_DTYPE;
    const int st = check_shape(rows, width, vocab);
    if (st != TILE_OK) return st;
    if (!std::isfinite(scale)) return TILE_ERR_EPS;
    if (dweight == nullptr) return TILE_ERR_NULL;
    const size_t es = elem_size(dtype), ds = elem_size(dweight_dtype);
    if (misaligned_to(dweight, ds)) return TILE_ERR_ALIGN;
    const size_t r = static_cast<size_t>(rows), w = static_cast<size_t>(width);
    const size_t grad_bytes = static_cast<size_t>(vocab) * w * ds;
    if (rows == 0) {   // no rows: the gradient is zero, or stays as it is
        const cudaError_t inj = tile::injected_launch_failure();
        if (inj != cudaSuccess) return cuda_status(inj);
        if (accumulate) return TILE_OK;
        return cuda_status(cudaMemsetAsync(dweight, 0, grad_bytes, stream));
    }
    const size_t need = tile::embedding_backward_workspace(rows, width, vocab);
    if (tokens == nullptr || dout == nullptr || (need > 0 && workspace == nullptr))
        return TILE_ERR_NULL;
    if (misaligned_to(tokens, 8) || misaligned_to(dout, es) ||
        (need > 0 && misaligned_to(workspace, 256)))
        return TILE_ERR_ALIGN;
    if (workspace_bytes < need) return TILE_ERR_WORKSPACE;
    const Range written[] = {{dweight, grad_bytes}, {need > 0 ? workspace : nullptr, need}};
    const Range read[] = {{tokens, r * 8}, {dout, r * w * es}};
    if (tile::any_overlap(written, 2, read, 2)) return TILE_ERR_ALIAS;
    const cudaError_t inj = tile::injected_launch_failure();
    if (inj != cudaSuccess) return cuda_status(inj);
    tile::EmbeddingArgs a = {};
    a.tokens = tokens;
    a.dout = dout;
    a.dweight = dweight;
    a.ignore = ignore_index;
    a.rows = rows;
    a.width = width;
    a.vocab = vocab;
    a.scale = scale;
    a.add = accumulate != 0;
    a.ws = workspace;
    const bool vectors = !misaligned_to(dout, 16) && !misaligned_to(dweight, 16) && w * es % 16 == 0;
    return cuda_status(tile::launch_embedding_backward(dtype, dweight_dtype, vectors, a, stream));
}

}  // extern "C"
