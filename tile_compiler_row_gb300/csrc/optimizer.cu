// The norm of many gradients with the factor that clips it, and the AdamW step
// over many tensors.
//
//   norm = scale sqrt(sum of g^2),  factor = scale min(1, max / norm)
//
//   g = factor grad
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = (1 - lr decay) p - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Bound by DRAM: the norm reads each gradient once; a step reads and writes
// parameter and states, reads the gradient and writes the 16-bit copy.  The
// tensors' table (pointers, sizes, and where each begins in the list of all
// chunks) is a kernel argument of up to 32 KB: no copy to the device, nothing
// to keep alive, and a captured call holds it.  A chunk finds its tensor by
// bisection.
//
// (One GB300, a copy moves 6.68 TB/s.  1.2e9 parameters: norm of BF16 gradients
// 350 us, 1.03 of that rate; step with a BF16 copy 4.74 ms, 1.07.  1.9e8
// parameters with 8-bit states, FP16 gradients and copies: 478 us, 0.96.  11
// tensors of 1.3e5 elements: 5.7 and 2.8 us, of a call, which is the host's, 23 to
// 30 and 30 to 34.  Tensors of unlike starts are taken one element at a time: 1.3e8
// parameters, BF16 gradients and copies, 884 us where the grid takes 536, with 8-bit
// states 542 and 331.)
//
// 8-bit states are e4m3 values with a power of two for each 256 elements, m
// itself and the root of v (whose range an 8-bit v would not hold).  A step
// moves v by some 1e-3 of itself, far below e4m3's steps of 1/8 to 1/16, so
// values are rounded up with the probability of what is cut off: rounded to
// nearest, v could never shrink.  Scaling by powers of two is exact and costs
// a bit of range, none of precision.
#include <cuda_fp8.h>

#include <cmath>

#include "device_status.h"
#include "optimizer.h"
#include "row_windows.cuh"

namespace tile {
namespace {

// ---- tables ---------------------------------------------------------------------

struct NormEntry {
    const void *p;
    long long n;
    int elem, pad;
};
struct AdamwEntry {
    float *param;
    const void *grad;
    void *m, *v;
    float *m_scale, *v_scale;
    void *copy;
    long long n;
    float decay;
    int index;        // in the caller's list
    short grad_elem, copy_elem;
    short vectors;    // every pointer on the grid of the vector accesses
    short head;       // FP32 states: elements in front of the pointers, up to the grid
};

template <class Entry, int N>
struct Table {
    int count, first[N + 1];   // first chunk of each tensor
    Entry entry[N];
};

template <class Entry, int N>
__device__ __forceinline__ int tensor_of(const Table<Entry, N> &t, int chunk) {
    int low = 0, high = t.count - 1;
    while (low < high) {
        const int mid = (low + high + 1) / 2;
        if (t.first[mid] <= chunk)
            low = mid;
        else
            high = mid - 1;
    }
    return low;
}

// ---- gradient norm ----------------------------------------------------------------

constexpr int kNormThreads = 256, kNormLoads = 8, kNormWindows = kNormThreads * kNormLoads;

// Sum of the squares of this thread's windows of a chunk.
template <class T>
__device__ __forceinline__ float chunk_squares(const NormEntry &e, long long chunk) {
    constexpr int V = 16 / sizeof(T);
    const T *p = static_cast<const T *>(e.p);
    const int phase = window_phase(p);
    uint4 raw[kNormLoads];
#pragma unroll
    for (int u = 0; u < kNormLoads; ++u) {
        const long long at = (chunk * kNormWindows + u * kNormThreads + threadIdx.x) * V - phase;
        raw[u] = make_uint4(0, 0, 0, 0);
        if (at >= 0 && at + V <= e.n) {
            raw[u] = __ldcs(reinterpret_cast<const uint4 *>(p + at));
        } else if (at < e.n) {
            unsigned int w[4] = {};
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (at + j >= 0 && at + j < e.n) {
                    if constexpr (sizeof(T) == 4)
                        w[j] = __float_as_uint(p[at + j]);
                    else
                        w[j / 2] |= static_cast<unsigned int>(
                                        reinterpret_cast<const unsigned short *>(p)[at + j]) << (16 * (j & 1));
                }
            raw[u] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < kNormLoads; ++u) {
        float v[V];
        widen_vec<T>(raw[u], v);
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) s = fmaf(v[j], v[j], s);
        sum += s;
    }
    return sum;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// Thread 0's sum over the CTA.
template <int THREADS>
__device__ __forceinline__ double cta_sum(double v, double *part) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    double total = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < THREADS / 32; ++w) total += part[w];
    return total;
}

// The norm and the factor.
__device__ __forceinline__ void finish_norm(double total, float scale, float most, float *out) {
    const double norm = scale * sqrt(total);
    out[0] = static_cast<float>(norm);
    // a norm that is not finite: no factor, and a step that takes it is skipped
    out[1] = !isfinite(out[0]) ? __int_as_float(0x7fffffff)
             : norm > most     ? static_cast<float>(scale * (most / norm))
                               : scale;
}

// FUSED: the grid is one cluster, whose first CTA joins the partial sums.
template <int N, bool FUSED>
__global__ void __launch_bounds__(kNormThreads)
    norm_kernel(const __grid_constant__ Table<NormEntry, N> t, double *partial, float scale, float most, float *out) {
    __shared__ double part[kNormThreads / 32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    float sum = 0.0f, cut = 0.0f;   // a thread's sum over its chunks, and what its roundings cut off
    for (int chunk = blockIdx.x; chunk < t.first[t.count]; chunk += gridDim.x) {
        const int i = tensor_of(t, chunk);
        const NormEntry &e = t.entry[i];
        const long long c = chunk - t.first[i];
        const float s = e.elem == ELEM_F32 ? chunk_squares<float>(e, c)
                        : e.elem == ELEM_BF16 ? chunk_squares<__nv_bfloat16>(e, c)
                                              : chunk_squares<__half>(e, c);
        const float to = __fadd_rn(sum, s), back = __fsub_rn(to, sum);
        cut += __fadd_rn(__fsub_rn(sum, __fsub_rn(to, back)), __fsub_rn(s, back));
        sum = to;
    }
    // an infinite sum has no rest
    const double v = static_cast<double>(sum) + (isfinite(sum) ? static_cast<double>(cut) : 0.0);
    const double total = cta_sum<kNormThreads>(v, part);
    if (threadIdx.x == 0) partial[blockIdx.x] = total;
    if constexpr (FUSED) {
        __syncthreads();
        __threadfence();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (blockIdx.x != 0 || threadIdx.x != 0) return;
        double all = 0.0;
        for (unsigned int i = 0; i < gridDim.x; ++i) all += __ldcg(partial + i);
        finish_norm(all, scale, most, out);
    }
}

constexpr int kNormJoin = 512;
__global__ void __launch_bounds__(kNormJoin)
    norm_join_kernel(const double *partial, int count, float scale, float most, float *out) {
    __shared__ double part[kNormJoin / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the partial sums are written
    double v = 0.0;
    for (int i = threadIdx.x; i < count; i += kNormJoin) v += __ldcg(partial + i);
    const double total = cta_sum<kNormJoin>(v, part);
    if (threadIdx.x == 0) finish_norm(total, scale, most, out);
}

// ---- AdamW --------------------------------------------------------------------------

struct Scalars {
    float lr, beta1, rest1, beta2, rest2, eps;   // rest: 1 - beta
    float log1, log2;           // of the betas
    float rate, root;           // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
    long long step;
    const float *lr_device;
    const long long *step_device;
    const float *factor;
    unsigned long long seed;
};

// What a step takes from the device, if anything.
__device__ __forceinline__ void load_scalars(Scalars &s) {
    if (s.lr_device == nullptr && s.step_device == nullptr) return;
    if (s.lr_device != nullptr) s.lr = __ldg(s.lr_device);
    if (s.step_device != nullptr) s.step = max(__ldg(s.step_device), 1ll);
    const float t = static_cast<float>(s.step);
    s.rate = s.lr / -expm1f(t * s.log1);
    s.root = rsqrtf(-expm1f(t * s.log2));
}

__device__ __forceinline__ float moment1(const Scalars &s, float m, float g) {
    return __fadd_rn(__fmul_rn(m, s.beta1), __fmul_rn(g, s.rest1));
}
__device__ __forceinline__ float moment2(const Scalars &s, float v, float g) {
    return __fadd_rn(__fmul_rn(v, s.beta2), __fmul_rn(__fmul_rn(g, g), s.rest2));
}
// 1 / x to 1 ulp, x from 2^-126 (the least eps) to 2^126: a root of v below 2^64 times
// 1 / sqrt(1 - b2^t) below 2^27 comes to 2^91, and an eps above 2^126 gives 0, no update.
__device__ __forceinline__ float reciprocal(float x) {
    float d;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
    return d;
}
__device__ __forceinline__ float updated(const Scalars &s, float p, float keep, float m, float root_v) {
    return fmaf(m * reciprocal(fmaf(root_v, s.root, s.eps)), -s.rate, p * keep);
}

// Four gradients from element `at` on.
__device__ __forceinline__ uint4 load_grads(const void *p, int elem, long long at) {
    if (elem == ELEM_F32) return __ldcs(reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + at));
    const uint2 t = __ldcs(reinterpret_cast<const uint2 *>(static_cast<const unsigned short *>(p) + at));
    return make_uint4(t.x, t.y, 0, 0);
}
__device__ __forceinline__ void widen_grads(uint4 t, int elem, float (&g)[4]) {
    if (elem == ELEM_F32) {
        g[0] = __uint_as_float(t.x);
        g[1] = __uint_as_float(t.y);
        g[2] = __uint_as_float(t.z);
        g[3] = __uint_as_float(t.w);
    } else if (elem == ELEM_BF16) {
        g[0] = __uint_as_float(t.x << 16);
        g[1] = __uint_as_float(t.x & 0xffff0000u);
        g[2] = __uint_as_float(t.y << 16);
        g[3] = __uint_as_float(t.y & 0xffff0000u);
    } else {
        const float2 a = Elem<__half>::widen2(t.x), b = Elem<__half>::widen2(t.y);
        g[0] = a.x;
        g[1] = a.y;
        g[2] = b.x;
        g[3] = b.y;
    }
}
__device__ __forceinline__ float load_grad(const void *p, int elem, long long at) {
    if (elem == ELEM_F32) return __ldcs(static_cast<const float *>(p) + at);
    const unsigned short t = __ldcs(static_cast<const unsigned short *>(p) + at);
    return elem == ELEM_BF16 ? __uint_as_float(static_cast<unsigned int>(t) << 16)
                             : __half2float(__ushort_as_half(t));
}
__device__ __forceinline__ unsigned int narrow_pair(int elem, float lo, float hi) {
    return elem == ELEM_BF16 ? Elem<__nv_bfloat16>::narrow2(lo, hi) : Elem<__half>::narrow2(lo, hi);
}
__device__ __forceinline__ void store_copy(void *p, int elem, long long at, float v) {
    if (elem == ELEM_BF16)
        store_one(static_cast<__nv_bfloat16 *>(p) + at, v);
    else
        store_one(static_cast<__half *>(p) + at, v);
}

constexpr int kAdamwThreads = 256, kAdamwGroup = kAdamwThreads * 4;

template <int N>
__global__ void __launch_bounds__(kAdamwThreads)
    adamw_kernel(const __grid_constant__ Table<AdamwEntry, N> t, Scalars s, int groups) {
    constexpr int U = 2;
    const int i = tensor_of(t, blockIdx.x);
    const AdamwEntry &e = t.entry[i];
    const float f = s.factor != nullptr ? __ldg(s.factor) : 1.0f;
    if (!isfinite(f)) return;   // a step that is skipped
    load_scalars(s);
    const float keep = fmaf(-s.lr, e.decay, 1.0f);
    const int chunk = groups * kAdamwGroup;   // groups: 1 or even
    const long long base = static_cast<long long>(blockIdx.x - t.first[i]) * chunk;
    float *param = e.param, *m = static_cast<float *>(e.m), *v = static_cast<float *>(e.v);
    auto vectors = [&](auto width, int k) {
        constexpr int W = decltype(width)::value;
        float4 pv[W], mv[W], vv[W];
        uint4 gv[W];
        long long at[W];
#pragma unroll
        for (int u = 0; u < W; ++u) {
            at[u] = base + ((k + u) * kAdamwThreads + threadIdx.x) * 4;
            gv[u] = load_grads(e.grad, e.grad_elem, at[u]);
            mv[u] = __ldcs(reinterpret_cast<const float4 *>(m + at[u]));
            vv[u] = __ldcs(reinterpret_cast<const float4 *>(v + at[u]));
            pv[u] = __ldcs(reinterpret_cast<const float4 *>(param + at[u]));
        }
#pragma unroll
        for (int u = 0; u < W; ++u) {
            float g[4], a[4] = {mv[u].x, mv[u].y, mv[u].z, mv[u].w}, b[4] = {vv[u].x, vv[u].y, vv[u].z, vv[u].w},
                        p[4] = {pv[u].x, pv[u].y, pv[u].z, pv[u].w};
            widen_grads(gv[u], e.grad_elem, g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                g[j] = __fmul_rn(g[j], f);
                a[j] = moment1(s, a[j], g[j]);
                b[j] = moment2(s, b[j], g[j]);
                p[j] = updated(s, p[j], keep, a[j], __fsqrt_rn(b[j]));
            }
            __stcs(reinterpret_cast<float4 *>(m + at[u]), make_float4(a[0], a[1], a[2], a[3]));
            __stcs(reinterpret_cast<float4 *>(v + at[u]), make_float4(b[0], b[1], b[2], b[3]));
            __stcs(reinterpret_cast<float4 *>(param + at[u]), make_float4(p[0], p[1], p[2], p[3]));
            if (e.copy_elem >= 0)
                __stcs(reinterpret_cast<uint2 *>(static_cast<unsigned short *>(e.copy) + at[u]),
                       make_uint2(narrow_pair(e.copy_elem, p[0], p[1]), narrow_pair(e.copy_elem, p[2], p[3])));
        }
    };
    long long at0 = base == 0 ? -static_cast<long long>(e.head) : base, end = min(base + chunk, e.n);
    if (e.vectors && base + chunk <= e.n) {
        if (groups == 1) {
            vectors(std::integral_constant<int, 1>(), 0);
        } else {
#pragma unroll 1
            for (int k = 0; k < groups; k += U) vectors(std::integral_constant<int, U>(), k);
        }
        end = base == 0 ? 0 : at0;   // what lies in front of the grid is left
    }
#pragma unroll 1
    for (; at0 < end; at0 += kAdamwGroup) {
        float g[4], a[4], b[4], p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const long long at = at0 + j * kAdamwThreads + threadIdx.x;
            g[j] = a[j] = b[j] = p[j] = 0.0f;
            if (at >= end) continue;
            g[j] = load_grad(e.grad, e.grad_elem, at);
            a[j] = __ldcs(m + at);
            b[j] = __ldcs(v + at);
            p[j] = __ldcs(param + at);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const long long at = at0 + j * kAdamwThreads + threadIdx.x;
            if (at >= end) continue;
            g[j] = __fmul_rn(g[j], f);
            a[j] = moment1(s, a[j], g[j]);
            b[j] = moment2(s, b[j], g[j]);
            p[j] = updated(s, p[j], keep, a[j], __fsqrt_rn(b[j]));
            __stcs(m + at, a[j]);
            __stcs(v + at, b[j]);
            __stcs(param + at, p[j]);
            if (e.copy_elem >= 0) store_copy(e.copy, e.copy_elem, at, p[j]);
        }
    }
}

// ---- AdamW with 8-bit states -----------------------------------------------------------

// SplitMix64's finalizer (Steele, Lea and Flood, "Fast splittable pseudorandom
// number generators", 2014).
__host__ __device__ __forceinline__ unsigned long long mix64(unsigned long long z) {
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}
constexpr unsigned long long kGolden = 0x9E3779B97F4A7C15ull;

// (32 random bits for each element: the two elements of a pair share a word of
// 64, of mix64(key + (pair + 1) kGolden).)

// The power of two that a block's values are divided by, its inverse: the
// largest of them comes to 128 to 256.  Blocks under 2^-100 are held as they
// are (as zeros); one that is not finite stays so.
struct BlockScale {
    float scale, inverse;
};
__device__ __forceinline__ BlockScale block_scale(unsigned int top) {   // bits of the largest magnitude
    const unsigned int e = top >> 23;
    if (e == 255) return BlockScale{__int_as_float(0x7fffffff), __int_as_float(0x7fffffff)};
    if (e < 27) return BlockScale{1.0f, 1.0f};
    return BlockScale{__uint_as_float((e - 7) << 23), __uint_as_float((261 - e) << 23)};
}

// A magnitude below 256 in e4m3's steps: 16 random bits (bits / 16, of which
// the low four are 0) are added below the three bits of the mantissa that
// stay.  Under 2^-6, where the type's steps no longer shrink, it is moved up to
// where three bits are such a step.  (Issue slots bind: written in C it was one
// instruction more.)
__device__ __forceinline__ float round_at_random(float size, unsigned int bits) {
    float d;
    asm("{\n\t.reg .pred small;\n\t.reg .f32 x;\n\t.reg .b32 w;\n\t"
        "setp.lt.f32 small, %1, 0f3C800000;\n\t"
        "mov.f32 x, %1;\n\t"
        "@small add.rn.f32 x, x, 0f3C800000;\n\t"
        "mov.b32 w, x;\n\t"
        "add.u32 w, w, %2;\n\t"
        "and.b32 w, w, 0xfff00000;\n\t"
        "mov.b32 x, w;\n\t"
        "@small add.rn.f32 x, x, 0fBC800000;\n\t"
        "mov.f32 %0, x;\n\t}" : "=f"(d) : "f"(size), "r"(bits));
    return d;
}

__device__ __forceinline__ unsigned int narrow_codes(float lo, float hi) {   // exact
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 widen_codes(unsigned int two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
// The largest magnitude, NaN where one is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Sums of two packed products.  Scalar: the packed addition of packed products
// came out as one rounding less (a fused multiply-add), against its ".rn".
__device__ __forceinline__ void add_halves(F2 a, F2 b, float &lo, float &hi) {
    float a0, a1, b0, b1;
    unpack(a, a0, a1);
    unpack(b, b0, b1);
    lo = __fadd_rn(a0, b0);
    hi = __fadd_rn(a1, b1);
}
__device__ __forceinline__ void copy_async(void *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 :: "r"(static_cast<unsigned int>(__cvta_generic_to_shared(to))), "l"(from) : "memory");
}

constexpr int kEightWarps = kAdamwThreads / 32;
// Shared memory of a warp: stages of a block of 256 each, its parameters, its
// codes of m and v, its gradients (16-bit: three stages, FP32: two).
constexpr int kEightRoom = 6144;
constexpr int kEightMost = 4;   // blocks of a warp

struct None {};   // no copy

template <class G>
__device__ __forceinline__ void widen_eight(const uint4 *t, float (&g)[8]) {
    if constexpr (sizeof(G) == 4) {
        widen_vec<float>(t[0], *reinterpret_cast<float (*)[4]>(&g[0]));
        widen_vec<float>(t[1], *reinterpret_cast<float (*)[4]>(&g[4]));
    } else {
        widen_vec<G>(t[0], g);
    }
}

// The blocks of one CTA.  Places are counted from the chunk's first element, in
// 32 bits.
template <class G, class C>
__device__ __forceinline__ void eight_chunk(const AdamwEntry &e, const Scalars &s, float f, float keep,
                                            unsigned long long key, long long start, int blocks, char *mine) {
    constexpr bool WIDE = sizeof(G) == 4;
    constexpr int STAGES = WIDE ? 2 : 3, SIZE = WIDE ? 2560 : 2048;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long chunk = static_cast<long long>(blocks) * kEightWarps * kStateBlock;
    const int left = static_cast<int>(min(e.n - start, chunk));        // elements of this CTA
    const int whole_to = e.vectors != 0 ? left & -kStateBlock : 0;   // ... that whole blocks on the grid have
    float *param = e.param + start;
    const G *grad = static_cast<const G *>(e.grad) + start;
    unsigned char *mc = static_cast<unsigned char *>(e.m) + start, *vc = static_cast<unsigned char *>(e.v) + start;
    float *m_scale = e.m_scale + start / kStateBlock, *v_scale = e.v_scale + start / kStateBlock;
    key += (static_cast<unsigned long long>(start) / 2 + 1) * kGolden;
    // a group of copies for each block of this warp, empty where there is none
    auto fetch = [&](int base, int stage) {
        if (base < whole_to) {
            char *to = mine + stage * SIZE + lane * 16;
            const char *p = reinterpret_cast<const char *>(param + base) + lane * 16;
            copy_async(to, p);
            copy_async(to + 512, p + 512);
            copy_async(to + 1024, (lane < 16 ? mc : vc) + base + (lane & 15) * 16);
            const char *g = reinterpret_cast<const char *>(grad + base) + lane * 16;
            copy_async(to + 1536, g);
            if constexpr (WIDE) copy_async(to + 2048, g + 512);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    constexpr int STEP = kEightWarps * kStateBlock;
    int base = warp * kStateBlock;
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) fetch(base + k * STEP, k);
    // the scales of this warp's blocks: lanes 0 .. 3 those of m, 4 .. 7 of v
    float scales = 0.0f;
    {
        const int of = base + (lane & 3) * STEP;
        if (lane < 8 && of < min(left, base + blocks * STEP))
            scales = __ldcs((lane < 4 ? m_scale : v_scale) + of / kStateBlock);
    }
    int stage = 0;
    for (int k = 0; base < left; base += STEP, ++k) {
        const bool whole = base < whole_to;
        fetch(base + (STAGES - 1) * STEP, stage == 0 ? STAGES - 1 : stage - 1);   // the stage read last
        asm volatile("cp.async.wait_group %0;" :: "n"(STAGES - 1) : "memory");
        __syncwarp();
        float p[8], g[8];
        unsigned int mw[2], vw[2];
        const int at = base + lane * 8;
        if (whole) {
            const char *from = mine + stage * SIZE;
            const float4 p0 = *reinterpret_cast<const float4 *>(from + lane * 32);
            const float4 p1 = *reinterpret_cast<const float4 *>(from + lane * 32 + 16);
            const uint2 a = *reinterpret_cast<const uint2 *>(from + 1024 + lane * 8);
            const uint2 b = *reinterpret_cast<const uint2 *>(from + 1280 + lane * 8);
            uint4 raw[2];
            raw[0] = *reinterpret_cast<const uint4 *>(from + 1536 + lane * (WIDE ? 32 : 16));
            if constexpr (WIDE) raw[1] = *reinterpret_cast<const uint4 *>(from + 1536 + lane * 32 + 16);
            widen_eight<G>(raw, g);
            const float q[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] = q[j];
            mw[0] = a.x;
            mw[1] = a.y;
            vw[0] = b.x;
            vw[1] = b.y;
        } else {   // a lane has each 32nd element of the block
            mw[0] = mw[1] = vw[0] = vw[1] = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int w = base + j * 32 + lane;
                p[j] = g[j] = 0.0f;
                if (w < left) {
                    g[j] = static_cast<float>(grad[w]);
                    p[j] = __ldcs(param + w);
                    mw[j / 4] |= static_cast<unsigned int>(mc[w]) << (8 * (j & 3));
                    vw[j / 4] |= static_cast<unsigned int>(vc[w]) << (8 * (j & 3));
                }
            }
        }
        __syncwarp();   // read, before the stage is written again
        stage = stage + 1 == STAGES ? 0 : stage + 1;
        const F2 m_old = both(__shfl_sync(0xffffffffu, scales, k));
        const F2 v_old = both(__shfl_sync(0xffffffffu, scales, 4 + k));
        // two elements at a time
        float m[8], v[8], mtop = 0.0f, vtop = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float2 mcode = widen_codes(mw[j / 4] >> (8 * (j & 3)) & 0xffff);
            const float2 vcode = widen_codes(vw[j / 4] >> (8 * (j & 3)) & 0xffff);
            const F2 g2 = mul2(pack(g[j], g[j + 1]), both(f));
            const F2 root = mul2(pack(vcode.x, vcode.y), v_old);
            add_halves(mul2(mul2(pack(mcode.x, mcode.y), m_old), both(s.beta1)), mul2(g2, both(s.rest1)), m[j],
                       m[j + 1]);
            add_halves(mul2(mul2(root, root), both(s.beta2)), mul2(mul2(g2, g2), both(s.rest2)), v[j], v[j + 1]);
            v[j] = __fsqrt_rn(v[j]);
            v[j + 1] = __fsqrt_rn(v[j + 1]);
            const F2 below = fma2(pack(v[j], v[j + 1]), both(s.root), both(s.eps));
            float d0, d1;
            unpack(below, d0, d1);
            const F2 step = mul2(pack(m[j], m[j + 1]), pack(reciprocal(d0), reciprocal(d1)));
            unpack(fma2(step, both(-s.rate), mul2(pack(p[j], p[j + 1]), both(keep))), p[j], p[j + 1]);
            mtop = max_abs(mtop, m[j], m[j + 1]);
            vtop = max_abs(vtop, v[j], v[j + 1]);
        }
        const BlockScale mscale = block_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(mtop)));
        const BlockScale vscale = block_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(vtop)));
        if (lane == 0) {
            m_scale[base / kStateBlock] = mscale.scale;
            v_scale[base / kStateBlock] = vscale.scale;
        }
        // low half of the bits: m, high half: v
        auto quantise = [&](int j, unsigned int bits) {
            const float size = round_at_random(fabsf(m[j]), (bits & 0xffff) << 4);
            m[j] = copysignf(size, m[j]);
            const float q = round_at_random(v[j], (bits >> 16) << 4);
            v[j] = v[j] > 0.0f ? fmaxf(q, 0.001953125f) : q;   // a root that is not zero stays so
        };
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            unpack(mul2(pack(m[j], m[j + 1]), both(mscale.inverse)), m[j], m[j + 1]);
            unpack(mul2(pack(v[j], v[j + 1]), both(vscale.inverse)), v[j], v[j + 1]);
        }
        if (whole) {   // the two elements of a pair are one lane's
            const unsigned long long at_pair = key + static_cast<unsigned long long>(static_cast<unsigned int>(at) / 2) * kGolden;
            unsigned int m4[4], v4[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const unsigned long long two = mix64(at_pair + static_cast<unsigned long long>(j) * kGolden);
                quantise(2 * j, static_cast<unsigned int>(two));
                quantise(2 * j + 1, static_cast<unsigned int>(two >> 32));
                m4[j] = narrow_codes(m[2 * j], m[2 * j + 1]);
                v4[j] = narrow_codes(v[2 * j], v[2 * j + 1]);
            }
            __stcs(reinterpret_cast<uint2 *>(mc + at), make_uint2(m4[0] | m4[1] << 16, m4[2] | m4[3] << 16));
            __stcs(reinterpret_cast<uint2 *>(vc + at), make_uint2(v4[0] | v4[1] << 16, v4[2] | v4[3] << 16));
            __stcs(reinterpret_cast<float4 *>(param + at), make_float4(p[0], p[1], p[2], p[3]));
            __stcs(reinterpret_cast<float4 *>(param + at) + 1, make_float4(p[4], p[5], p[6], p[7]));
            if constexpr (!std::is_same<C, None>::value)
                __stcs(reinterpret_cast<uint4 *>(static_cast<C *>(e.copy) + start + at),
                       make_uint4(Elem<C>::narrow2(p[0], p[1]), Elem<C>::narrow2(p[2], p[3]),
                                  Elem<C>::narrow2(p[4], p[5]), Elem<C>::narrow2(p[6], p[7])));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int w = base + j * 32 + lane;
                const unsigned long long two = mix64(key + static_cast<unsigned long long>(static_cast<unsigned int>(w) / 2) * kGolden);
                quantise(j, static_cast<unsigned int>((w & 1) != 0 ? two >> 32 : two));
                if (w >= left) continue;
                mc[w] = static_cast<unsigned char>(narrow_codes(m[j], 0.0f) & 0xff);
                vc[w] = static_cast<unsigned char>(narrow_codes(v[j], 0.0f) & 0xff);
                __stcs(param + w, p[j]);
                if constexpr (!std::is_same<C, None>::value) store_one(static_cast<C *>(e.copy) + start + w, p[j]);
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <class G>
__device__ __forceinline__ void eight_chunk_of(const AdamwEntry &e, const Scalars &s, float f, float keep,
                                               unsigned long long key, long long start, int blocks, char *mine) {
    if (e.copy_elem == ELEM_BF16)
        eight_chunk<G, __nv_bfloat16>(e, s, f, keep, key, start, blocks, mine);
    else if (e.copy_elem == ELEM_F16)
        eight_chunk<G, __half>(e, s, f, keep, key, start, blocks, mine);
    else
        eight_chunk<G, None>(e, s, f, keep, key, start, blocks, mine);
}

// A warp for each block of 256, `blocks` of them one after the other, whose
// vectors asynchronous copies bring to shared memory two blocks ahead: issue
// slots (82 % in use) and DRAM bind about alike.  1.9e8 parameters, FP16
// gradients and copies, 458 us of DRAM: 735 us with a block's loads in registers,
// 661 with the next block's too, 558 with the copies, 522 with the types known
// when compiled and shorter chunks, 480 with the scales of all of a warp's
// blocks in one load.  (With the moments fused and an approximate root 450; but
// then codes now and then differ from the definition's.)
template <int N>
__global__ void __launch_bounds__(kAdamwThreads, 4)
    adamw8_kernel(const __grid_constant__ Table<AdamwEntry, N> t, Scalars s, int blocks) {
    __shared__ __align__(16) char room[kEightWarps][kEightRoom];
    const int i = tensor_of(t, blockIdx.x);
    const AdamwEntry &e = t.entry[i];
    const float f = s.factor != nullptr ? __ldg(s.factor) : 1.0f;
    if (!isfinite(f)) return;   // a step that is skipped
    load_scalars(s);
    const float keep = fmaf(-s.lr, e.decay, 1.0f);
    const unsigned long long key =
        mix64(mix64(s.seed + static_cast<unsigned long long>(s.step) * kGolden) +
              static_cast<unsigned long long>(e.index + 1) * kGolden);
    const long long start = static_cast<long long>(blockIdx.x - t.first[i]) * blocks * (kEightWarps * kStateBlock);
    char *mine = room[threadIdx.x >> 5];
    if (e.grad_elem == ELEM_F32)
        eight_chunk_of<float>(e, s, f, keep, key, start, blocks, mine);
    else if (e.grad_elem == ELEM_BF16)
        eight_chunk_of<__nv_bfloat16>(e, s, f, keep, key, start, blocks, mine);
    else
        eight_chunk_of<__half>(e, s, f, keep, key, start, blocks, mine);
}

// ---- launches ---------------------------------------------------------------------------

constexpr int kFewTensors = 32;   // a table this short is a kernel argument of 3 KB

bool on_grid(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

constexpr int kNormCluster = 8, kNormFew = 32;   // CTAs of a cluster, and chunks that one takes

// out != NULL: the norm too, where there are few chunks (*programs is 0 then).
template <int N>
cudaError_t launch_norm_table(const NormTensor *t, int count, double *partial, int *programs, float scale,
                              float most, float *out, cudaStream_t stream) {
    Table<NormEntry, N> table;
    table.count = count;
    long long chunks = 0;
    for (int i = 0; i < count; ++i) {
        table.entry[i] = NormEntry{t[i].p, t[i].n, t[i].elem, 0};
        table.first[i] = static_cast<int>(chunks);
        const long long v = t[i].elem == ELEM_F32 ? 4 : 8;   // windows, with one more for the grid
        chunks += ((t[i].n + v - 1) / v + 1 + kNormWindows - 1) / kNormWindows;
        if (chunks > 0x7fffffff) return cudaErrorInvalidValue;
    }
    table.first[count] = static_cast<int>(chunks);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.blockDim = dim3(kNormThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    if (out != nullptr && chunks <= kNormFew) {
        cfg.gridDim = dim3(static_cast<unsigned int>(chunks < kNormCluster ? chunks : kNormCluster));
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = cfg.gridDim.x;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.numAttrs = 1;
        *programs = 0;
        return cudaLaunchKernelEx(&cfg, norm_kernel<N, true>, table, partial, scale, most, out);
    }
    *programs = chunks < kNormPrograms ? static_cast<int>(chunks) : kNormPrograms;
    cfg.gridDim = dim3(*programs);
    return cudaLaunchKernelEx(&cfg, norm_kernel<N, false>, table, partial, scale, most, out);
}

// Elements of a chunk: as many as leave kChunksPerSm of them for each SM, in 1, 2, 4 .. `most`
// steps of the smallest (few elements: latency counts).  At most 2048 in FP32
// and 8192 with 8-bit states: short CTAs that follow one another keep the
// accesses in the order of the memory (1.2e9 parameters in FP32: 4.93 ms with
// 1024, 4.75 with 2048, 4.81 with 4096, 4.93 with 8192; 1.9e8 with 8 bits: 625
// us with 2048, 522 with 8192, 533 with 16384, 550 with 32768).
constexpr long long kChunksPerSm = 16;
long long chunk_of(long long elements, long long smallest, int most, int *steps) {
    const long long wanted = sm_count_of_device() * kChunksPerSm;
    *steps = 1;
    while (*steps < most && elements / (smallest * *steps * 2) >= wanted) *steps *= 2;
    return smallest * *steps;
}

template <int N>
cudaError_t launch_adamw_table(const AdamwTensor *t, int count, int index, const AdamwConfig &c,
                               const Scalars &s, cudaStream_t stream) {
    Table<AdamwEntry, N> table;
    int used = 0, steps = 0;
    long long chunks = 0, elements = 0;
    for (int i = 0; i < count; ++i) elements += t[i].n;
    const long long chunk = c.eight ? chunk_of(elements, kEightWarps * kStateBlock, kEightMost, &steps)
                                    : chunk_of(elements, kAdamwGroup, 2, &steps);
    for (int i = 0; i < count; ++i) {
        const AdamwTensor &a = t[i];
        if (a.n == 0) continue;
        const size_t four = c.eight ? 8 : 4;   // elements of a vector access
        const size_t grad = a.grad_elem == ELEM_F32 ? 16 : 2 * four;
        auto grid = [&](int head) {   // whether all lie on the grid that many elements on
            auto on = [&](const void *p, size_t elem, size_t to) {
                return p == nullptr || on_grid(static_cast<const char *>(p) + head * elem, to);
            };
            const size_t gs = a.grad_elem == ELEM_F32 ? 4 : 2, ss = c.eight ? 1 : 4;
            return on(a.param, 4, 16) && on(a.grad, gs, grad) && on(a.m, ss, 16) && on(a.v, ss, 16) &&
                   on(a.copy, 2, 2 * four);
        };
        // tensors that lie one behind the other in buffers alike are off the grid
        // by the same elements (1.3e8 parameters, BF16 gradients and copies: 543 us,
        // on the grid 536, of unlike starts 884)
        int head = 0;
        while (!c.eight && head < 3 && head + 1 < a.n && !grid(head)) ++head;
        const bool vectors = grid(head);
        if (!vectors) head = 0;
        const size_t gs = a.grad_elem == ELEM_F32 ? 4 : 2;
        auto on = [&](void *p, size_t elem) { return p == nullptr ? p : static_cast<char *>(p) + head * elem; };
        AdamwEntry e = {a.param + head, static_cast<const char *>(a.grad) + head * gs, a.m, a.v, a.m_scale, a.v_scale,
                        on(a.copy, 2), a.n - head, a.decay, index + i, a.grad_elem, a.copy_elem,
                        static_cast<short>(vectors), static_cast<short>(head)};
        if (!c.eight) {
            e.m = on(a.m, 4);
            e.v = on(a.v, 4);
        }
        table.entry[used] = e;
        table.first[used++] = static_cast<int>(chunks);
        chunks += (e.n + chunk - 1) / chunk;
        if (chunks > 0x7fffffff) return cudaErrorInvalidValue;
    }
    if (used == 0) return cudaSuccess;
    table.count = used;
    table.first[used] = static_cast<int>(chunks);
    const unsigned int grid = static_cast<unsigned int>(chunks);
    if (c.eight)
        adamw8_kernel<N><<<grid, kAdamwThreads, 0, stream>>>(table, s, steps);
    else
        adamw_kernel<N><<<grid, kAdamwThreads, 0, stream>>>(table, s, steps);
    return cudaGetLastError();
}

}  // namespace

size_t grad_norm_workspace(int count) {
    const size_t launches = (static_cast<size_t>(count) + kNormTensors - 1) / kNormTensors;
    return launches * kNormPrograms * sizeof(double);
}

cudaError_t launch_grad_norm(const NormTensor *t, int count, float scale, float max_norm,
                             float *out, void *ws, cudaStream_t stream) {
    double *partial = static_cast<double *>(ws);
    int total = 0;
    float *whole = count > 0 && count <= kNormTensors ? out : nullptr;   // one launch of sums at most
    for (int i = 0; i < count; i += kNormTensors) {
        const int n = count - i < kNormTensors ? count - i : kNormTensors;
        int programs = 0;
        const cudaError_t err = n <= kFewTensors
            ? launch_norm_table<kFewTensors>(t + i, n, partial + total, &programs, scale, max_norm, whole, stream)
            : launch_norm_table<kNormTensors>(t + i, n, partial + total, &programs, scale, max_norm, whole, stream);
        if (err != cudaSuccess || (whole != nullptr && programs == 0)) return err;
        total += programs;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kNormJoin);
    cfg.stream = stream;
    cfg.attrs = attr;
    // with one launch of sums before it, the join comes up while they run
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = count > 0 && count <= kNormTensors ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, norm_join_kernel, static_cast<const double *>(partial), total, scale,
                              max_norm, out);
}

cudaError_t launch_adamw(const AdamwTensor *t, int count, const AdamwConfig &c, cudaStream_t stream) {
    Scalars s = {};
    s.lr = static_cast<float>(c.lr);
    s.beta1 = static_cast<float>(c.beta1);
    s.rest1 = static_cast<float>(1.0 - c.beta1);
    s.beta2 = static_cast<float>(c.beta2);
    s.rest2 = static_cast<float>(1.0 - c.beta2);
    s.eps = static_cast<float>(c.eps);
    s.log1 = static_cast<float>(std::log(c.beta1));
    s.log2 = static_cast<float>(std::log(c.beta2));
    if (c.step_device == nullptr) {
        s.rate = static_cast<float>(c.lr / (1.0 - std::pow(c.beta1, static_cast<double>(c.step))));
        s.root = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(c.beta2, static_cast<double>(c.step))));
    }
    s.step = c.step;
    s.lr_device = c.lr_device;
    s.step_device = c.step_device;
    s.factor = c.factor;
    s.seed = c.seed;
    for (int i = 0; i < count; i += kAdamwTensors) {
        const int n = count - i < kAdamwTensors ? count - i : kAdamwTensors;
        const cudaError_t err = n <= kFewTensors ? launch_adamw_table<kFewTensors>(t + i, n, i, c, s, stream)
                                                 : launch_adamw_table<kAdamwTensors>(t + i, n, i, c, s, stream);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

}  // namespace tile
