// Argument checks and statuses shared by the entry points (host only).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/tile_rows.h"
#include "launch.h"

namespace tile {

// The status of an entry point whose CUDA calls ended with err, which is kept
// for tile_last_cuda_error.
inline int cuda_status(cudaError_t err) {
    if (err == cudaSuccess) return TILE_OK;
    set_last_cuda_error(static_cast<int>(err));
    return TILE_ERR_CUDA;
}

inline size_t elem_size(int dtype) {
    return dtype == TILE_DTYPE_BF16 || dtype == TILE_DTYPE_F16 ? 2 : 4;
}

// Whether [a, a + abytes) and [b, b + bbytes) share a byte; NULL overlaps
// nothing.
inline bool overlaps(const void *a, size_t abytes, const void *b, size_t bbytes) {
    if (a == nullptr || b == nullptr) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bbytes && y < x + abytes;
}

// Whether p is not aligned to `bytes` (a power of two).
inline bool misaligned_to(const void *p, size_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

// One device range of a call, for the pairwise overlap check.
struct Range {
    const void *p;
    size_t bytes;
};

// Whether any of the `nout` written ranges overlaps another of them or any
// of the `nin` read ranges.
inline bool any_overlap(const Range *out, int nout, const Range *in, int nin) {
    for (int i = 0; i < nout; ++i) {
        for (int j = i + 1; j < nout; ++j)
            if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return true;
        for (int j = 0; j < nin; ++j)
            if (overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return true;
    }
    return false;
}

}  // namespace tile
