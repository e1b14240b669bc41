// Launchers of the gradients' norm and the AdamW step (optimizer.cu), both
// over many tensors at once.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace tile {

constexpr int kStateBlock = 256;   // elements that share a scale of an 8-bit state

struct NormTensor {
    const void *p;
    long long n;
    int elem;
};

// The norm's CTAs leave this many partial sums for each launch at most: 8 for each of
// 152 SMs, a whole GPU of this kind.  The same on every device: it decides the order
// of additions, so the bits, and the workspace.
constexpr int kNormPrograms = 152 * 8;
constexpr int kNormTensors = 1024;   // tensors of one launch
size_t grad_norm_workspace(int count);
// out: [2] norm and factor; ws: grad_norm_workspace(count) bytes.  Tensors of no
// elements are left out by the caller.
cudaError_t launch_grad_norm(const NormTensor *t, int count, float scale, float max_norm,
                             float *out, void *ws, cudaStream_t stream);

struct AdamwTensor {
    float *param;
    const void *grad;
    void *m, *v;
    float *m_scale, *v_scale;   // 8-bit states
    void *copy;
    long long n;
    float decay;
    short grad_elem, copy_elem;   // copy_elem -1: none
};

struct AdamwConfig {
    double lr, beta1, beta2, eps;
    long long step;
    const float *lr_device;
    const long long *step_device;
    const float *factor;
    unsigned long long seed;
    bool eight;
};

constexpr int kAdamwTensors = 384;   // tensors of one launch
cudaError_t launch_adamw(const AdamwTensor *t, int count, const AdamwConfig &c, cudaStream_t stream);

}  // namespace tile
