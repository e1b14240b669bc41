// C ABI of the clipped policy loss and its gradient (include/tile_rows.h):
// argument checks and dispatch.
#include <cmath>

#include "../../include/tile_rows.h"
#include "host_checks.h"
#include "launch.h"
#include "policy_loss.h"

namespace {

using tile::cuda_status;
using tile::misaligned_to;
using tile::Range;

constexpr int kMostRows = 1 << 30;

// The nearest FP32 value of a bound and what it leaves of it.
void split(double bound, float *near, float *rest) {
    *near = static_cast<float>(bound);
    *rest = std::isfinite(*near) ? static_cast<float>(bound - *near) : 0.0f;
}

// The checks that forward and backward share, and the kernels' arguments.
int check(const tile_policy_loss_args_t &c, tile::PolicyArgs *a) {
    if (c.flags < 0 || c.flags > (TILE_POLICY_SEQUENCE_ADVANTAGE | TILE_POLICY_SEQUENCE_MEAN))
        return TILE_ERR_OP;
    if (c.rows < 0 || c.rows > kMostRows || c.sequences < 1 || c.sequences > kMostRows ||
        (c.offsets == nullptr && c.sequences != 1))
        return TILE_ERR_SHAPE;
    if (!(c.clip_low >= 0.0f && c.clip_low <= 1.0f) || !(c.clip_high >= 0.0f) ||
        !std::isfinite(c.kl_coef))
        return TILE_ERR_EPS;
    if (c.rows > 0 && (c.nll == nullptr || c.old_nll == nullptr || c.advantage == nullptr ||
                       (c.kl_coef != 0.0f && c.ref_nll == nullptr)))
        return TILE_ERR_NULL;
    if (misaligned_to(c.nll, 4) || misaligned_to(c.old_nll, 4) || misaligned_to(c.ref_nll, 4) ||
        misaligned_to(c.advantage, 4) || misaligned_to(c.target, 8) || misaligned_to(c.offsets, 8))
        return TILE_ERR_ALIGN;
    a->nll = c.nll;
    a->old_nll = c.old_nll;
    a->ref_nll = c.ref_nll;
    a->advantage = c.advantage;
    a->target = c.target;
    a->offsets = c.offsets;
    a->ignore = c.ignore_index;
    a->rows = c.rows;
    a->sequences = c.sequences;
    a->sequence_advantage = (c.flags & TILE_POLICY_SEQUENCE_ADVANTAGE) != 0;
    a->sequence_mean = (c.flags & TILE_POLICY_SEQUENCE_MEAN) != 0;
    a->clip_low = c.clip_low;
    a->clip_high = c.clip_high;
    a->kl_coef = c.kl_coef;
    split(std::log1p(-static_cast<double>(c.clip_low)), &a->low, &a->low_rest);
    split(std::log1p(static_cast<double>(c.clip_high)), &a->high, &a->high_rest);
    return TILE_OK;
}

// The ranges that a call reads.
constexpr int kReads = 6;
void reads(const tile_policy_loss_args_t &c, Range (&r)[kReads]) {
    const size_t rows = static_cast<size_t>(c.rows), seqs = static_cast<size_t>(c.sequences);
    const bool per_sequence = (c.flags & TILE_POLICY_SEQUENCE_ADVANTAGE) != 0;
    r[0] = {c.nll, rows * 4};
    r[1] = {c.old_nll, rows * 4};
    r[2] = {c.ref_nll, rows * 4};
    r[3] = {c.advantage, (per_sequence ? seqs : rows) * 4};
    r[4] = {c.target, rows * 8};
    r[5] = {c.offsets, (seqs + 1) * 8};
}

}  // namespace

extern "C" {

size_t tile_policy_loss_workspace_bytes(int rows, int sequences) {
    if (rows < 1 || rows > kMostRows || sequences < 1 || sequences > kMostRows) return 0;
    return tile::policy_loss_workspace(rows, sequences);
}

int tile_policy_loss(const tile_policy_loss_args_t *args, float *stats, float *weights,
                     void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (args == nullptr) return TILE_ERR_NULL;
    const tile_policy_loss_args_t &c = *args;
    tile::PolicyArgs a = {};
    const int st = check(c, &a);
    if (st != TILE_OK) return st;
    if (stats == nullptr || weights == nullptr || (c.rows > 0 && workspace == nullptr))
        return TILE_ERR_NULL;
    if (misaligned_to(stats, 4) || misaligned_to(weights, 4) ||
        (c.rows > 0 && misaligned_to(workspace, 16)))
        return TILE_ERR_ALIGN;
    const size_t wbytes = static_cast<size_t>(c.sequences) * 4;
    const size_t need = c.rows > 0 ? tile::policy_loss_workspace(c.rows, c.sequences) : 0;
    if (workspace_bytes < need) return TILE_ERR_WORKSPACE;
    const Range written[] = {{stats, 16}, {weights, wbytes}, {c.rows > 0 ? workspace : nullptr, need}};
    Range read[kReads];
    reads(c, read);
    if (tile::any_overlap(written, 3, read, kReads)) return TILE_ERR_ALIAS;
    const cudaError_t inj = tile::injected_launch_failure();
    if (inj != cudaSuccess) return cuda_status(inj);
    if (c.rows == 0) {   // nothing counts
        cudaError_t err = cudaMemsetAsync(stats, 0, 16, stream);
        if (err == cudaSuccess) err = cudaMemsetAsync(weights, 0, wbytes, stream);
        return cuda_status(err);
    }
    a.stats = stats;
    a.weights = weights;
    a.ws = workspace;
    return cuda_status(tile::launch_policy_loss(a, stream));
}

int tile_policy_loss_backward(const tile_policy_loss_args_t *args, const float *weights,
                              const float *dloss, float *dnll, cudaStream_t stream) {
    if (args == nullptr) return TILE_ERR_NULL;
    const tile_policy_loss_args_t &c = *args;
    tile::PolicyArgs a = {};
    const int st = check(c, &a);
    if (st != TILE_OK) return st;
    if (c.rows == 0) return TILE_OK;
    if (weights == nullptr || dnll == nullptr) return TILE_ERR_NULL;
    if (misaligned_to(weights, 4) || misaligned_to(dloss, 4) || misaligned_to(dnll, 4))
        return TILE_ERR_ALIGN;
    const Range written[] = {{dnll, static_cast<size_t>(c.rows) * 4}};
    Range read[kReads + 2];
    Range inputs[kReads];
    reads(c, inputs);
    for (int i = 0; i < kReads; ++i) read[i] = inputs[i];
    read[kReads] = {weights, static_cast<size_t>(c.sequences) * 4};
    read[kReads + 1] = {dloss, 4};
    if (tile::any_overlap(written, 1, read, kReads + 2)) return TILE_ERR_ALIAS;
    const cudaError_t inj = tile::injected_launch_failure();
    if (inj != cudaSuccess) return cuda_status(inj);
    if (c.kl_coef == 0.0f) a.ref_nll = nullptr;   // no term, whatever e^q would be
    a.weights = const_cast<float *>(weights);
    a.dloss = dloss;
    a.dnll = dnll;
    return cuda_status(tile::launch_policy_loss_backward(a, stream));
}

}  // extern "C"
