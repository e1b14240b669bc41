// Launchers of the clipped policy loss and its gradient (policy_loss.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace tile {

struct PolicyArgs {
    const float *nll, *old_nll, *ref_nll;   // [rows]; ref_nll may be NULL
    const float *advantage;                 // [rows] or [sequences]
    const long long *target;                // [rows] or NULL
    const long long *offsets;               // [sequences + 1] or NULL: one of all rows
    long long ignore;
    int rows, sequences;
    bool sequence_advantage, sequence_mean;
    float clip_low, clip_high, kl_coef;
    // bounds of the log ratio, log(1 - clip_low) and log(1 + clip_high): the
    // nearest FP32 value and what it leaves
    float low, low_rest, high, high_rest;
    float *stats;       // [4]
    float *weights;     // [sequences]; the gradient reads it
    const float *dloss; // [1] or NULL: 1
    float *dnll;        // [rows]
    void *ws;
    unsigned int *status;
};

size_t policy_loss_workspace(int rows, int sequences);
cudaError_t launch_policy_loss(PolicyArgs a, cudaStream_t stream);
cudaError_t launch_policy_loss_backward(PolicyArgs a, cudaStream_t stream);

}  // namespace tile
