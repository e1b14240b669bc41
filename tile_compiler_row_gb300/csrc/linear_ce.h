// Linear softmax cross entropy: host-side launchers (linear_ce.cu) and the
// workspace layout they share with the entry points (linear_ce_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace tile {

struct LinearCeArgs {
    int elem;                   // ELEM_BF16 or ELEM_F16
    const void *x, *weight;     // [rows][width], [vocab][width]
    const long long *target;    // [rows]
    long long ignore;
    float *loss, *lse;          // forward outputs (lse: backward input)
    const float *dloss;         // backward
    void *dx, *dweight;         // backward outputs, either may be NULL
    int rows, width, vocab;
    void *ws;
    bool withheld;              // forward, tests only (tile_test_linear_cross_entropy_wait_timeout)
};

size_t linear_ce_workspace(int rows, int width, int vocab);
size_t linear_ce_backward_workspace(int rows, int width, int vocab);
cudaError_t launch_linear_ce(const LinearCeArgs &a, cudaStream_t stream);
cudaError_t launch_linear_ce_backward(const LinearCeArgs &a, cudaStream_t stream);

}  // namespace tile
