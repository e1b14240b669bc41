// Shared parts of the block-norm kernels: the thread layout of a row, vector
// access, and the reduction of a row's partial sums over its threads.
//
// A row program is W = 32 * S threads of each of C CTAs (a thread-block
// cluster when C > 1).  Thread w of CTA rank c owns, of every row it
// handles, the columns ((k * C + c) * W + w) * V + v, k < K, v < V: the same
// columns in every row, so that per-column parameters and column sums stay
// in registers while the program walks over rows.  V is a 16-byte vector
// (4 FP32 or 8 two-byte elements) or 1 (odd widths, pointers that are not
// 16-byte aligned).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"
#include "row_kernel.cuh"

namespace tile {

// How one row is spread over threads.
struct BlockPlan {
    int elems;     // E = K * V elements a thread owns (8, 16 or 32)
    int threads;   // W per CTA
    int cluster;   // C
};

// 8 elements a thread keep the parameters, the column sums and a prefetched
// row in registers at 512 threads (4096 columns); wider rows take 16, then a
// cluster of CTAs, and the widest 32.
inline BlockPlan block_plan(int width) {
    auto warps = [](int n) { return (n + 31) / 32 * 32; };
    if (width <= 8 * 512) return {8, warps((width + 7) / 8), 1};
    if (width <= 16 * 512) return {16, warps((width + 15) / 16), 1};
    for (int c = 2; c <= 8; c *= 2)
        if (width <= 16 * 512 * c) return {16, 512, c};
    return {32, 512, 8};
}

template <class T, int V>
struct Access;

template <class T>
struct Access<T, 1> {
    using Raw = typename std::conditional<sizeof(T) == 4, unsigned int, unsigned short>::type;
    __device__ static Raw load(const T *p) { return __ldcs(reinterpret_cast<const Raw *>(p)); }
    __device__ static void widen(Raw r, float (&v)[1]) {
        if constexpr (sizeof(T) == 4)
            v[0] = __uint_as_float(r);
        else if constexpr (std::is_same<T, __half>::value)
            v[0] = __half2float(__ushort_as_half(r));
        else
            v[0] = __uint_as_float(static_cast<unsigned int>(r) << 16);
    }
    __device__ static void store(T *p, const float (&v)[1]) { Elem<T>::store(p, v[0]); }
};

template <class T, int V>
struct Access {
    static_assert(V == 16 / sizeof(T), "16-byte vectors");
    using Raw = uint4;
    __device__ static Raw load(const T *p) { return __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ static void widen(Raw t, float (&v)[V]) {
        const unsigned int w[4] = {t.x, t.y, t.z, t.w};
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (std::is_same<T, __half>::value) {
                    const float2 f = Elem<__half>::widen2(w[i]);
                    v[2 * i] = f.x;
                    v[2 * i + 1] = f.y;
                } else {
                    v[2 * i] = __uint_as_float(w[i] << 16);
                    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                }
            }
        }
    }
    __device__ static void store(T *p, const float (&v)[V]) { Elem<T>::store_vec(p, v); }
};

// V parameters of a column group (FP32, any 4-byte alignment; 1 when p is
// NULL).
template <int V>
__device__ __forceinline__ void load_params(const float *p, int col, float (&v)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = p != nullptr ? __ldg(p + col + j) : 1.0f;
}

__device__ __forceinline__ void cluster_barrier() {
    cluster_arrive();
    cluster_wait();
}

// Shared memory of the row reductions: two buffers used in turn, so one
// barrier a reduction is enough (a buffer is rewritten only after the next
// reduction's barrier, which every thread reaches after its reads).
template <int N>
struct ReduceMem {
    float warp[2][32 * N];
    float cta[2][N];
};

// Sums of s over the row's threads, in a fixed order, for all of them.
template <int N, bool CL>
__device__ __forceinline__ void row_sum(float (&s)[N], ReduceMem<N> &mem, int &turn, int warps,
                                        int cluster) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], d);
    if (warps > 1) {
        float *buf = mem.warp[turn];
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) buf[i * 32 + (threadIdx.x >> 5)] = s[i];
        __syncthreads();
        // every warp adds the warps' partials (at most 32) in the same tree
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = lane < warps ? buf[i * 32 + lane] : 0.0f;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], d);
    }
    if constexpr (CL) {
        if (threadIdx.x == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) mem.cta[turn][i] = s[i];
        cluster_barrier();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = 0.0f;
            for (int c = 0; c < cluster; ++c) t += load_dsmem(&mem.cta[turn][i], c);
            s[i] = t;
        }
    }
    turn ^= 1;
}

// The unit (of `units`, each with the rows [rows u / units, rows (u + 1) /
// units)) that holds row r.
__host__ __device__ inline long long unit_of_row(long long r, long long rows, long long units) {
    long long u = r * units / rows;
    while (rows * (u + 1) / units <= r) ++u;
    while (u > 0 && rows * u / units > r) --u;
    return u;
}

// One block-norm call (forward and backward); see include/tile_rows.h.
struct BlockArgs {
    const void *x, *residual, *hidden, *dhidden, *dout;
    const float *gamma_post, *gate, *gamma_pre;
    void *hidden_out, *out, *din, *dresidual;
    float *dgamma_post, *dgate, *dgamma_pre;
    float *ws;
    long long rows;
    long long per_gate;   // rows that share a gate row
    int width;
    int post, pre;
    float scale, eps;
    unsigned int *status;
};

cudaError_t launch_block_norm(int elem, bool vec, const BlockArgs &a, cudaStream_t stream);
cudaError_t launch_block_norm_backward(int elem, bool vec, const BlockArgs &a,
                                       cudaStream_t stream);
size_t block_norm_backward_workspace(long long rows, int width);

}  // namespace tile
