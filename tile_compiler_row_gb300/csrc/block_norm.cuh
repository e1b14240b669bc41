// Shared parts of the block-norm kernels: the thread layout of a row, vector
// access, and the reduction of a row's partial sums over its threads.
//
// A row program is W = 32 * S threads of each of C CTAs (a thread-block
// cluster when C > 1); a thread owns E = K * V columns, in K groups of V.  V
// is a 16-byte vector (4 FP32 or 8 two-byte elements) or 1 (odd widths,
// pointers that are not 16-byte aligned).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "launch.h"
#include "row_kernel.cuh"

namespace tile {

// Two FP32 values in one 64-bit register pair, for the packed instructions
// (PTX mul / fma .rn.f32x2, sm_100 and later), each half rounded as by the
// scalar one: these kernels issued 50 to 66 instructions per element
// without, and the issue slots bind.
typedef unsigned long long F2;
__device__ __forceinline__ F2 pack(float lo, float hi) {
    F2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void unpack(F2 v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ F2 both(float v) { return pack(v, v); }
__device__ __forceinline__ float total(F2 v) {
    float lo, hi;
    unpack(v, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// One 16-byte vector of T as FP32 pairs, and back (rounded to nearest even).
template <class T>
struct Vec {
    static constexpr int N = 16 / sizeof(T), P = N / 2;
    __device__ static void widen(uint4 t, F2 (&v)[P]) {
        const unsigned int w[4] = {t.x, t.y, t.z, t.w};
        if constexpr (sizeof(T) == 4) {
            v[0] = pack(__uint_as_float(w[0]), __uint_as_float(w[1]));
            v[1] = pack(__uint_as_float(w[2]), __uint_as_float(w[3]));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (std::is_same<T, __half>::value) {
                    const float2 f = Elem<__half>::widen2(w[i]);
                    v[i] = pack(f.x, f.y);
                } else {
                    v[i] = pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
                }
            }
        }
    }
    __device__ static uint4 narrow(const F2 (&v)[P]) {
        unsigned int w[4];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float lo, hi;
            unpack(v[i], lo, hi);
            if constexpr (sizeof(T) == 4) {
                w[2 * i] = __float_as_uint(lo);
                w[2 * i + 1] = __float_as_uint(hi);
            } else {
                w[i] = Elem<T>::narrow2(lo, hi);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// The vectors that hold a row which lies off the 16-byte grid: its first
// begins `shift` elements before the row, and its last may reach past its end.
// The masks of those two lie in shared memory (a thread's own test of eight
// elements for each vector, row and input made the threads at a row's ends
// the last of their CTA: 16384 x 4097 BF16 backward 345 us).
struct EdgeMasks {
    uint4 first, last;
};
enum { EDGE_FIRST = 1, EDGE_LAST = 2 };

template <class T>
__device__ __forceinline__ uint4 mask_of(int from, int to) {   // elements [from, to) of a vector
    constexpr int N = 16 / sizeof(T);
    unsigned int w[4] = {};
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j >= from && j < to)
            w[j * static_cast<int>(sizeof(T)) / 4] |=
                sizeof(T) == 4 ? 0xffffffffu : 0xffffu << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <class T>
__device__ __forceinline__ void edge_masks(EdgeMasks &m, int shift, int width) {
    constexpr int N = 16 / sizeof(T);
    m.first = mask_of<T>(shift, N);
    m.last = mask_of<T>(0, (width + shift - 1) % N + 1);
}
// Which ends vector v of `vecs` is.
__device__ __forceinline__ int edge_of(int v, int vecs) {
    return (v == 0 ? EDGE_FIRST : 0) | (v == vecs - 1 ? EDGE_LAST : 0);
}
__device__ __forceinline__ uint4 and4(uint4 a, uint4 b) {
    return make_uint4(a.x & b.x, a.y & b.y, a.z & b.z, a.w & b.w);
}
__device__ __forceinline__ uint4 mask_vec(uint4 t, int edge, const EdgeMasks &m) {
    if (edge & EDGE_FIRST) t = and4(t, m.first);
    if (edge & EDGE_LAST) t = and4(t, m.last);
    return t;
}
// Its store: whole, or the elements that are the row's.
template <class T>
__device__ __forceinline__ void store_vec_at(T *p, uint4 t, int first, int width) {
    constexpr int N = 16 / sizeof(T);
    if (first >= 0 && first + N <= width) {
        __stcs(reinterpret_cast<uint4 *>(p), t);
        return;
    }
    const unsigned int w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (first + j >= 0 && first + j < width) {
            if constexpr (sizeof(T) == 4)
                reinterpret_cast<unsigned int *>(p)[j] = w[j];
            else
                reinterpret_cast<unsigned short *>(p)[j] =
                    static_cast<unsigned short>((j & 1) ? w[j / 2] >> 16 : w[j / 2]);
        }
}
// N parameters from column `first` on, as pairs; 0 outside the row, 1 when p
// is NULL.
template <int N>
__device__ __forceinline__ void params_at(const float *p, int first, int width, F2 (&v)[N / 2]) {
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
        const int c = first + 2 * j;
        const float lo = c < 0 || c >= width ? 0.0f : p == nullptr ? 1.0f : __ldg(p + c);
        const float hi = c + 1 < 0 || c + 1 >= width ? 0.0f : p == nullptr ? 1.0f : __ldg(p + c + 1);
        v[j] = pack(lo, hi);
    }
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

// V FP32 parameters of a column group, 1 when p is NULL.  Vector accesses
// (V > 1) take parameters whose rows are aligned to V of them: one load of
// 16 or 32 bytes, so that a warp reads one contiguous run.
template <int V>
__device__ __forceinline__ void load_params(const float *p, int col, float (&v)[V]) {
    if (p == nullptr) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = 1.0f;
    } else if constexpr (V == 8) {
        asm("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
            : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
              "=f"(v[7])
            : "l"(p + col));
    } else if constexpr (V == 4) {
        const float4 t = __ldg(reinterpret_cast<const float4 *>(p + col));
        v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
    } else {
        v[0] = __ldg(p + col);
    }
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

// Sums of s over the row's threads, in a fixed order, for all of them: the
// threads of `warps` warps of each CTA of the cluster, or `lanes` neighbours
// of a warp (a power of two).
template <int N, bool CL>
__device__ __forceinline__ void row_sum(float (&s)[N], ReduceMem<N> &mem, int &turn, int warps,
                                        int cluster, int lanes = 32) {
    if (lanes < 32) {
        for (int d = lanes >> 1; d > 0; d >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], d);
        return;
    }
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
        // every warp adds the warps' partials (at most 16) in the same tree:
        // half the power of two that holds them, down to neighbours
        const int half = warps > 8 ? 8 : warps > 4 ? 4 : warps > 2 ? 2 : 1;
        const int lane = threadIdx.x & (2 * half - 1);
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = lane < warps ? buf[i * 32 + lane] : 0.0f;
        for (int d = half; d > 0; d >>= 1)
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

// The layout of a program that walks over rows.
struct RingPlan {
    int workers;    // W: threads of a program in a CTA (below 32: neighbours in a warp)
    int cluster;    // C
    int slots;      // ring kernel: slots, and bytes of a slot's part for one input
    int pitch;
    int smem;
    int classes;    // row classes by where rows start in a 16-byte block
    int parts;      // above one class: programs that share a class of a group of rows
};

// The rows of a program: first, first + step, ...
struct RowWalk {
    long long first, count;
    int step;
};
// With one class, contiguous ranges of all rows; with more, programs keep to
// one group of `group` rows, and to one class there.
__device__ __forceinline__ RowWalk row_walk(long long rows, long long group, const RingPlan &p,
                                            long long unit, long long units) {
    RowWalk w;
    if (p.classes == 1) {
        w.first = rows * unit / units;
        w.count = rows * (unit + 1) / units - w.first;
        w.step = 1;
        return w;
    }
    const int part = static_cast<int>(unit % p.parts);
    const int cls = static_cast<int>(unit / p.parts % p.classes);
    const long long begin = unit / (p.classes * p.parts) * group;
    const long long end = begin + group < rows ? begin + group : rows;
    // classes is a power of two
    const long long first = begin + ((cls - begin) & (p.classes - 1));
    const long long n = first < end ? (end - 1 - first) / p.classes + 1 : 0;
    w.first = first + p.classes * (n * part / p.parts);
    w.count = n * (part + 1) / p.parts - n * part / p.parts;
    w.step = p.classes;
    return w;
}

// CTAs of a kernel to an SM of the current device for a launch shape, its
// shared memory limit raised to the shape's.  The last answer for a kernel is
// kept per device: calls of one shape follow one another, and the two CUDA
// calls take longer than a launch.
struct OccupancyCache {
    std::atomic<unsigned long long> last[kMaxDevices];   // threads, smem, CTAs
};

template <class Kernel>
cudaError_t occupancy(Kernel kernel, OccupancyCache &cache, int threads, int smem, int *per_sm) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    const unsigned long long key = (static_cast<unsigned long long>(threads) << 32 |
                                    static_cast<unsigned int>(smem)) << 8;
    const unsigned long long known = cache.last[dev].load(std::memory_order_acquire);
    if (known >> 8 == key >> 8 && (known & 0xff) != 0) {
        *per_sm = static_cast<int>(known & 0xff);
        return cudaSuccess;
    }
    // the limit only ever grows, so that a call of another thread that is
    // between this and its launch keeps what it needs
    if (smem > 40 << 10)   // with the static part above 48 KiB
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 << 10);
    if (err != cudaSuccess) return err;
    err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(per_sm, kernel, threads, smem);
    if (err != cudaSuccess) return err;
    if (*per_sm < 1) *per_sm = 1;
    cache.last[dev].store(key | static_cast<unsigned long long>(*per_sm), std::memory_order_release);
    return cudaSuccess;
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
    unsigned int *status;   // backward
    bool withheld;          // backward, tests only (tile_test_block_norm_backward_wait_timeout)
};

// What the pointers of a call allow: every row and parameter row on vectors;
// row matrices that start on 16 bytes (rows of any width, parameters of any
// alignment); neither.
enum BlockAccess { ACCESS_VECTORS, ACCESS_SHIFTED, ACCESS_ELEMENTS };

cudaError_t launch_block_norm(int elem, BlockAccess access, const BlockArgs &a,
                              cudaStream_t stream);
cudaError_t launch_block_norm_backward(int elem, BlockAccess access, const BlockArgs &a,
                                       cudaStream_t stream);
size_t block_norm_backward_workspace(long long rows, int width, long long gates);

}  // namespace tile
