// Rows that begin anywhere, in windows of V = 16 / sizeof(T) elements that lie
// on the 16-byte grid of the row that is written: its first and last window
// may be cut.  The row that is read has a grid of its own; a window of it is
// put together from the two vectors that hold it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "block_norm.cuh"

namespace tile {

// Elements by which the grid's window lies before the element at p.
template <class D>
__device__ __forceinline__ int window_phase(const D *p) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(p) / sizeof(D) % (16 / sizeof(D)));
}

__device__ __forceinline__ uint4 load_vec(const void *p) {
    return __ldg(static_cast<const uint4 *>(p));
}

// Elements [at, at + V) of the row [row, row + width) of T, 0 outside it.
// Reads nothing outside the row.
template <class T, bool VEC>
__device__ __forceinline__ uint4 load_window(const T *row, int at, int width) {
    constexpr int V = 16 / sizeof(T);
    if constexpr (VEC) return load_vec(row + at);
    const uintptr_t p = reinterpret_cast<uintptr_t>(row) + static_cast<long long>(at) * sizeof(T);
    const uintptr_t begin = reinterpret_cast<uintptr_t>(row);
    const uintptr_t end = begin + static_cast<size_t>(width) * sizeof(T);
    const uintptr_t low = p & ~static_cast<uintptr_t>(15);
    const unsigned int shift = static_cast<unsigned int>(p & 15);
    if (low >= begin && low + (shift != 0 ? 32 : 16) <= end) {
        const uint4 a = load_vec(reinterpret_cast<const void *>(low));
        if (shift == 0) return a;
        const uint4 b = load_vec(reinterpret_cast<const void *>(low + 16));
        unsigned int w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        if (shift & 8) {
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        }
        if (shift & 4) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
        }
        if constexpr (sizeof(T) == 2) {
            if (shift & 2) {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    unsigned int w[4] = {};
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (at + j >= 0 && at + j < width) {
            if constexpr (sizeof(T) == 4)
                w[j] = __ldg(reinterpret_cast<const unsigned int *>(row + at + j));
            else
                w[j / 2] |= static_cast<unsigned int>(
                                __ldg(reinterpret_cast<const unsigned short *>(row + at + j)))
                            << (16 * (j & 1));
        }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <class T>
__device__ __forceinline__ void widen_vec(uint4 t, float (&v)[16 / sizeof(T)]) {
    Access<T, 16 / sizeof(T)>::widen(t, v);
}

template <class D>
__device__ __forceinline__ void store_one(D *p, float v) {
    if constexpr (sizeof(D) == 4)
        *reinterpret_cast<float *>(p) = v;
    else if constexpr (std::is_same<D, __half>::value)
        *p = __float2half_rn(v);
    else
        *p = __float2bfloat16_rn(v);
}

// v, rounded to D, to elements [at, at + V) of the row; those outside it are
// left.  The window is on the grid of D.
template <class D, int V, bool VEC>
__device__ __forceinline__ void store_window(D *row, int at, int width, const float (&v)[V]) {
    constexpr int N = 16 / sizeof(D);
    if (VEC || (at >= 0 && at + V <= width)) {
#pragma unroll
        for (int i = 0; i < V; i += N) {
            uint4 t;
            if constexpr (sizeof(D) == 4)
                t = make_uint4(__float_as_uint(v[i]), __float_as_uint(v[i + 1]),
                               __float_as_uint(v[i + 2]), __float_as_uint(v[i + 3]));
            else
                t = make_uint4(Elem<D>::narrow2(v[i], v[i + 1]), Elem<D>::narrow2(v[i + 2], v[i + 3]),
                               Elem<D>::narrow2(v[i + 4], v[i + 5]),
                               Elem<D>::narrow2(v[i + 6], v[i + 7]));
            *reinterpret_cast<uint4 *>(row + at + i) = t;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (at + j >= 0 && at + j < width) store_one(row + at + j, v[j]);
}

// What the window holds now, widened; 0 outside the row.
template <class D, int V, bool VEC>
__device__ __forceinline__ void read_window(const D *row, int at, int width, float (&v)[V]) {
    constexpr int N = 16 / sizeof(D);
    if (VEC || (at >= 0 && at + V <= width)) {
#pragma unroll
        for (int i = 0; i < V; i += N) {
            float p[N];
            widen_vec<D>(*reinterpret_cast<const uint4 *>(row + at + i), p);
#pragma unroll
            for (int j = 0; j < N; ++j) v[i + j] = p[j];
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        v[j] = 0.0f;
        if (at + j >= 0 && at + j < width) v[j] = static_cast<float>(row[at + j]);
    }
}

}  // namespace tile
