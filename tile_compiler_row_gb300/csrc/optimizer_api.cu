// C ABI of the gradients' norm and the AdamW step (include/tile_rows.h):
// argument checks and dispatch.
#include <float.h>
#include <stdlib.h>

#include <algorithm>
#include <cmath>
#include <memory>

#include "../../include/tile_rows.h"
#include "host_checks.h"
#include "launch.h"
#include "optimizer.h"

namespace {

using tile::cuda_status;
using tile::elem_size;
using tile::misaligned_to;

bool valid_dtype(int dtype) {
    return dtype == TILE_DTYPE_F32 || dtype == TILE_DTYPE_BF16 || dtype == TILE_DTYPE_F16;
}

constexpr long long kMostElements = 1ll << 40;   // chunk numbers are ints

// Host memory for `n` of T without an exception where there is none.
template <class T>
std::unique_ptr<T, decltype(&free)> host_array(size_t n) {
    return {static_cast<T *>(malloc((n > 0 ? n : 1) * sizeof(T))), &free};
}

// A device range of a call with many of them.
struct Span {
    uintptr_t begin, end;
    bool written;
};

struct Spans {
    Span *at;
    size_t n;
    void add(const void *p, size_t bytes, bool written) {
        if (p == nullptr || bytes == 0) return;
        const uintptr_t b = reinterpret_cast<uintptr_t>(p);
        at[n++] = Span{b, b + bytes, written};
    }
    // Whether a written range shares a byte with another one.
    bool any_overlap() {
        auto before = [](const Span &a, const Span &b) { return a.begin < b.begin; };
        if (!std::is_sorted(at, at + n, before)) std::sort(at, at + n, before);
        uintptr_t end = 0, written_end = 0;   // of the ranges so far
        for (size_t i = 0; i < n; ++i) {
            if (at[i].begin < (at[i].written ? end : written_end)) return true;
            end = std::max(end, at[i].end);
            if (at[i].written) written_end = std::max(written_end, at[i].end);
        }
        return false;
    }
};

}  // namespace

extern "C" {

size_t tile_grad_norm_workspace_bytes(int count) {
    return count < 1 ? 0 : tile::grad_norm_workspace(count);
}

int tile_grad_norm(const tile_tensor_t *tensors, int count, float scale, float max_norm,
                   float *out, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (count < 0) return TILE_ERR_SHAPE;
    if (out == nullptr || (count > 0 && tensors == nullptr)) return TILE_ERR_NULL;
    if (!(std::isfinite(scale) && scale > 0.0f) || !(max_norm > 0.0f)) return TILE_ERR_EPS;
    if (misaligned_to(out, 4)) return TILE_ERR_ALIGN;
    const auto list = host_array<tile::NormTensor>(static_cast<size_t>(count));
    const auto spans = host_array<Span>(static_cast<size_t>(count) + 2);
    if (list == nullptr || spans == nullptr) return cuda_status(cudaErrorMemoryAllocation);
    Spans used = {spans.get(), 0};
    int n = 0;
    for (int i = 0; i < count; ++i) {
        const tile_tensor_t &t = tensors[i];
        if (!valid_dtype(t.dtype)) return TILE_ERR_DTYPE;
        if (t.n < 0 || t.n > kMostElements) return TILE_ERR_SHAPE;
        if (t.n == 0) continue;
        if (t.data == nullptr) return TILE_ERR_NULL;
        if (misaligned_to(t.data, elem_size(t.dtype))) return TILE_ERR_ALIGN;
        used.add(t.data, static_cast<size_t>(t.n) * elem_size(t.dtype), false);
        list.get()[n++] = tile::NormTensor{t.data, t.n, t.dtype};
    }
    const size_t need = tile_grad_norm_workspace_bytes(count);
    if (count > 0) {
        if (workspace == nullptr) return TILE_ERR_NULL;
        if (misaligned_to(workspace, 16)) return TILE_ERR_ALIGN;
        if (workspace_bytes < need) return TILE_ERR_WORKSPACE;
        used.add(workspace, need, true);
    }
    used.add(out, 8, true);
    if (used.any_overlap()) return TILE_ERR_ALIAS;
    const cudaError_t inj = tile::injected_launch_failure();
    if (inj != cudaSuccess) return cuda_status(inj);
    return cuda_status(tile::launch_grad_norm(list.get(), n, scale, max_norm, out, workspace, stream));
}

int tile_adamw(const tile_adamw_tensor_t *tensors, int count, const tile_adamw_config_t *config,
               cudaStream_t stream) {
    if (config == nullptr) return TILE_ERR_NULL;
    const tile_adamw_config_t &c = *config;
    if (c.state != TILE_STATE_F32 && c.state != TILE_STATE_E4M3) return TILE_ERR_OP;
    if (count < 0 || (c.step_device == nullptr && c.step < 1)) return TILE_ERR_SHAPE;
    if (count > 0 && tensors == nullptr) return TILE_ERR_NULL;
    if (!(c.beta1 >= 0.0 && c.beta1 < 1.0) || !(c.beta2 >= 0.0 && c.beta2 < 1.0) ||
        !(std::isfinite(c.eps) && static_cast<float>(c.eps) >= FLT_MIN) ||
        (c.lr_device == nullptr && !std::isfinite(static_cast<float>(c.lr))))
        return TILE_ERR_EPS;
    if (misaligned_to(c.lr_device, 4) || misaligned_to(c.step_device, 8) || misaligned_to(c.factor, 4))
        return TILE_ERR_ALIGN;
    const bool eight = c.state == TILE_STATE_E4M3;
    const auto list = host_array<tile::AdamwTensor>(static_cast<size_t>(count));
    const auto spans = host_array<Span>(static_cast<size_t>(count) * 7 + 3);
    if (list == nullptr || spans == nullptr) return cuda_status(cudaErrorMemoryAllocation);
    Spans used = {spans.get(), 0};
    bool any = false;
    for (int i = 0; i < count; ++i) {
        const tile_adamw_tensor_t &t = tensors[i];
        if (!valid_dtype(t.grad_dtype) ||
            (t.copy != nullptr && t.copy_dtype != TILE_DTYPE_BF16 && t.copy_dtype != TILE_DTYPE_F16))
            return TILE_ERR_DTYPE;
        if (t.n < 0 || t.n > kMostElements) return TILE_ERR_SHAPE;
        if (!std::isfinite(t.weight_decay)) return TILE_ERR_EPS;
        // (a place of its own for tensors of no elements: the place in the list counts)
        list.get()[i] = tile::AdamwTensor{t.param, t.grad, t.exp_avg, t.exp_avg_sq,
                                          eight ? t.exp_avg_scale : nullptr,
                                          eight ? t.exp_avg_sq_scale : nullptr, t.copy, t.n,
                                          t.weight_decay, static_cast<short>(t.grad_dtype),
                                          static_cast<short>(t.copy != nullptr ? t.copy_dtype : -1)};
        if (t.n == 0) continue;
        any = true;
        if (t.param == nullptr || t.grad == nullptr || t.exp_avg == nullptr || t.exp_avg_sq == nullptr ||
            (eight && (t.exp_avg_scale == nullptr || t.exp_avg_sq_scale == nullptr)))
            return TILE_ERR_NULL;
        const size_t state = eight ? 1 : 4, gs = elem_size(t.grad_dtype), n = static_cast<size_t>(t.n);
        if (misaligned_to(t.param, 4) || misaligned_to(t.grad, gs) || misaligned_to(t.exp_avg, state) ||
            misaligned_to(t.exp_avg_sq, state) || misaligned_to(t.copy, 2) ||
            (eight && (misaligned_to(t.exp_avg_scale, 4) || misaligned_to(t.exp_avg_sq_scale, 4))))
            return TILE_ERR_ALIGN;
        used.add(t.param, n * 4, true);
        used.add(t.grad, n * gs, false);
        used.add(t.exp_avg, n * state, true);
        used.add(t.exp_avg_sq, n * state, true);
        used.add(t.copy, n * 2, true);
        if (eight) {
            const size_t scales = (n + tile::kStateBlock - 1) / tile::kStateBlock * 4;
            used.add(t.exp_avg_scale, scales, true);
            used.add(t.exp_avg_sq_scale, scales, true);
        }
    }
    used.add(c.lr_device, 4, false);
    used.add(c.step_device, 8, false);
    used.add(c.factor, 4, false);
    if (used.any_overlap()) return TILE_ERR_ALIAS;
    if (!any) return TILE_OK;
    const cudaError_t inj = tile::injected_launch_failure();
    if (inj != cudaSuccess) return cuda_status(inj);
    const tile::AdamwConfig a = {c.lr, c.beta1, c.beta2, c.eps, c.step, c.lr_device, c.step_device,
                                 c.factor, c.seed, eight};
    return cuda_status(tile::launch_adamw(list.get(), count, a, stream));
}

}  // extern "C"
