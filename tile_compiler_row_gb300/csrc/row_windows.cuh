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

// The matrix that windows are read from: nothing outside it is.
struct Bounds {
    uintptr_t begin;
    long long last;   // bytes from the begin at which two vectors still fit
};
template <class T>
__device__ __forceinline__ Bounds bounds_of(const void *p, long long rows, int width) {
    return Bounds{reinterpret_cast<uintptr_t>(p), rows * width * static_cast<long long>(sizeof(T)) - 32};
}

// The vectors that hold elements [at, at + V) of a row, read without a branch
// so that many windows are in flight; then the window put together.  A
// window's elements outside the row hold what lies there: they are not stored.
template <bool VEC>
struct RawWindow;
template <>
struct RawWindow<true> {
    uint4 a;
};
template <>
struct RawWindow<false> {
    uint4 a, b;
    bool whole;   // both vectors lie in the matrix
};

template <class T, bool VEC>
__device__ __forceinline__ RawWindow<VEC> fetch_window(const T *row, int at, const Bounds &m, bool wanted) {
    RawWindow<VEC> w = {};
    if constexpr (VEC) {
        if (wanted) w.a = load_vec(row + at);
    } else {
        const uintptr_t p = reinterpret_cast<uintptr_t>(row) + static_cast<long long>(at) * sizeof(T);
        const uintptr_t low = p & ~static_cast<uintptr_t>(15);
        // (ends of the matrix, where a vector would pass them: element by element, below)
        const long long off = static_cast<long long>(low - m.begin);
        w.whole = off >= 0 && off <= m.last;
        if (wanted && w.whole) {
            w.a = load_vec(reinterpret_cast<const void *>(low));
            w.b = load_vec(reinterpret_cast<const void *>(low + 16));
        }
    }
    return w;
}

template <class T, bool VEC>
__device__ __forceinline__ uint4 join_window(const RawWindow<VEC> &r, const T *row, int at, int width) {
    if constexpr (VEC) return r.a;
    else {
        constexpr int V = 16 / sizeof(T);
        unsigned int w[4] = {};
        if (!r.whole) {
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
        // bytes by which the window lies behind the first vector: the same for
        // all windows of a row, so these branches do not diverge
        const unsigned int shift = static_cast<unsigned int>(
            (reinterpret_cast<uintptr_t>(row) + static_cast<long long>(at) * sizeof(T)) & 15);
        const unsigned int bits = sizeof(T) == 4 ? 0 : 8 * (shift & 2);
        auto from = [&](unsigned int a, unsigned int b, unsigned int c, unsigned int d, unsigned int e) {
            if constexpr (sizeof(T) == 4) return make_uint4(a, b, c, d);
            else
                return make_uint4(__funnelshift_r(a, b, bits), __funnelshift_r(b, c, bits),
                                  __funnelshift_r(c, d, bits), __funnelshift_r(d, e, bits));
        };
        switch (shift >> 2) {
            case 0: return from(r.a.x, r.a.y, r.a.z, r.a.w, r.b.x);
            case 1: return from(r.a.y, r.a.z, r.a.w, r.b.x, r.b.y);
            case 2: return from(r.a.z, r.a.w, r.b.x, r.b.y, r.b.z);
            default: return from(r.a.w, r.b.x, r.b.y, r.b.z, r.b.w);
        }
    }
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
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (at + j >= 0 && at + j < width) store_one(row + at + j, v[j]);
    }
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
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            v[j] = 0.0f;
            if (at + j >= 0 && at + j < width) v[j] = static_cast<float>(row[at + j]);
        }
    }
}

}  // namespace tile
