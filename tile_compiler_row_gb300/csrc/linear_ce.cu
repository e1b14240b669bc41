// Softmax cross entropy of a linear head, without keeping the logits.
//
//   l = x W^T,  lse = log sum_v exp(l_v),  loss = lse - l_target
//   g = (exp(l - lse) - onehot(target)) dloss,  dx = g W,  dW = g^T x
//
// Every product is a matrix product on the fifth-generation tensor cores
// with FP32 accumulators in tensor memory; what becomes of a 128 x 256 tile
// of it is the epilogue:
//
//   forward    a tile of l is reduced to each row's maximum and sum of
//              exponentials, two numbers per tile and row; a second kernel
//              joins them and takes the target's logit as a dot product of
//              its own, in FP32 FMAs: the tensor cores truncate as they add
//              (at 4096 columns a logit was off by 1e-5), which an lse mostly
//              averages out and one logit does not (the loss of 4096 tokens
//              over 131072 entries was 1.5e-6 off in the 2-norm with the
//              tile's logit).
//   backward   in pieces of the vocabulary: l is computed again, turned into
//              g and kept in 16 bits for this piece only; then dW of the
//              piece's rows is g^T x, and g W is added to an FP32 dx.
//
// Backward first packs the rows whose target counts (and whose dloss is not
// 0) to the front of a copy of x, so rows that are ignored cost nothing and
// a NaN in one of them reaches no gradient.
#include "linear_ce.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "device_status.h"
#include "tcgen05.cuh"

TILE_DEVICE_STATUS(linear_ce)

namespace tile {
namespace {

enum { CE_WAIT_TIMEOUT = 2u, CE_BAD_TARGET = 8u };

constexpr int BM = 128, BN = 256, BK = 64, STAGES = 4;
constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int GEMM_SMEM = STAGES * STAGE_BYTES + 1024;   // + slack to align to 1024
constexpr int GEMM_THREADS = 192;                        // 4 epilogue warps, TMA, MMA
constexpr float kLog2e = 1.4426950408889634f;

enum { EPI_LSE, EPI_GRAD, EPI_DWEIGHT, EPI_DX };

// What a backward call learns on the device before its products.
struct CeState {
    int valid;        // packed rows
    float unscale;    // what the scaled gradients are multiplied by at the end
};

struct GemmArgs {
    int m, n, k;                // extents (rows of A, rows of B, reduction)
    const CeState *state;       // limits m (GRAD, DX) or k (DWEIGHT) to the packed rows
    int bf16;
    // EPI_LSE
    float2 *partial;            // [m][n tiles]
    // EPI_GRAD: packed rows' target, lse log2(e) and scaled dloss
    const int *ptarget;
    const float *plse2, *pdloss;
    void *grad;                 // [m padded][ld]
    int n0;                     // first vocabulary entry of the piece
    // EPI_DWEIGHT / EPI_DX
    void *out;
    long long ld;               // elements per row of grad / out
    int accumulate;             // EPI_DX: add to what is there
    int splits;                 // EPI_DX: parts of k, each with its own slice
    long long slice;            // elements of a slice
    unsigned int *status;
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t pack2(int bf16, float lo, float hi) {
    if (bf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// C[m][n] = sum_k A[m][k] B[n][k], tile by tile on a persistent grid.
// A_MN / B_MN: the operand lies in memory as [k][m] / [k][n].
template <bool A_MN, bool B_MN, int EPI>
__global__ void __launch_bounds__(GEMM_THREADS, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const GemmArgs g) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * STAGES + 4];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto acc_full = [&](int s) { return bar0 + 8u * (2 * STAGES + s); };
    auto acc_empty = [&](int s) { return bar0 + 8u * (2 * STAGES + 2 + s); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < STAGES; ++s) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            bar_init(acc_full(s), 1);
            bar_init(acc_empty(s), 128);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 5) tmem_alloc(smem_u32(&tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *const_cast<volatile uint32_t *>(&tmem_slot);
    volatile int *aborted = &abort_flag;

    int m_ext = g.m, k_ext = g.k;
    if (EPI == EPI_GRAD || EPI == EPI_DX) m_ext = g.state->valid;
    if (EPI == EPI_DWEIGHT) k_ext = g.state->valid;
    const int m_tiles = (m_ext + BM - 1) / BM, n_tiles = (g.n + BN - 1) / BN;
    const int k_blocks = (k_ext + BK - 1) / BK;
    const int splits = EPI == EPI_DX ? g.splits : 1;
    const long long tiles = static_cast<long long>(m_tiles) * n_tiles * splits;
    auto kb_begin = [&](int split) { return k_blocks * split / splits; };

    if (warp == 4 && lane == 0) {   // TMA producer
        int stage = 0;
        unsigned int phase = 0;
        long long issued = 0;
        bool ok = true;
        for (long long t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            const int mt = static_cast<int>(t % m_tiles);
            const int nt = static_cast<int>(t / m_tiles % n_tiles);
            const int sp = static_cast<int>(t / m_tiles / n_tiles);
            for (int kb = kb_begin(sp); kb < kb_begin(sp + 1); ++kb) {
                if (!(ok = bar_wait(empty(stage), phase ^ 1u, aborted, g.status, CE_WAIT_TIMEOUT)))
                    break;
                const uint32_t a = base + stage * STAGE_BYTES, b = a + A_BYTES;
                bar_expect_tx(full(stage), STAGE_BYTES);
                if (A_MN) {
                    for (int i = 0; i < BM / 64; ++i)
                        tma_load(a + i * 8192, &map_a, mt * BM + i * 64, kb * BK, full(stage));
                } else {
                    tma_load(a, &map_a, kb * BK, mt * BM, full(stage));
                }
                if (B_MN) {
                    for (int i = 0; i < BN / 64; ++i)
                        tma_load(b + i * 8192, &map_b, nt * BN + i * 64, kb * BK, full(stage));
                } else {
                    tma_load(b, &map_b, kb * BK, nt * BN, full(stage));
                }
                ++issued;
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        // An aborted CTA waits (bounded) for the copies it issued: none may
        // land in shared memory that it no longer owns.
        if (*aborted)
            for (long long i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
                for (unsigned int n = 0; n < kBarSpins; ++n)
                    if (bar_test(full(static_cast<int>(i % STAGES)), (i / STAGES) & 1)) break;
    } else if (warp == 5 && lane == 0) {   // MMA issuer
        const uint32_t idesc = mma_idesc(g.bf16 != 0, A_MN, B_MN, BM, BN);
        int stage = 0, acc = 0;
        unsigned int phase = 0, acc_phase = 0;
        bool ok = true;
        for (long long t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            const int sp = static_cast<int>(t / m_tiles / n_tiles);
            if (!(ok = bar_wait(acc_empty(acc), acc_phase ^ 1u, aborted, g.status, CE_WAIT_TIMEOUT)))
                break;
            tc_fence_after();
            const uint32_t d = tmem + acc * BN;
            bool first = true;
            for (int kb = kb_begin(sp); kb < kb_begin(sp + 1); ++kb) {
                if (!(ok = bar_wait(full(stage), phase, aborted, g.status, CE_WAIT_TIMEOUT))) break;
                tc_fence_after();
                const uint32_t a = base + stage * STAGE_BYTES, b = a + A_BYTES;
                const uint64_t da = smem_desc(a, A_MN ? 8192 : 16, 1024);
                const uint64_t db = smem_desc(b, B_MN ? 8192 : 16, 1024);
#pragma unroll
                for (int k = 0; k < BK / 16; ++k) {
                    // 16 elements along K: 32 bytes of a K-major row, or 16
                    // rows of 128 bytes
                    tc_mma(d, da + k * (A_MN ? 2048 >> 4 : 32 >> 4),
                           db + k * (B_MN ? 2048 >> 4 : 32 >> 4), idesc, !first);
                    first = false;
                }
                tc_commit(empty(stage));
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            tc_commit(acc_full(acc));
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
        if (*aborted) {   // wait (bounded) until no MMA touches this CTA's memory
            tc_commit(acc_full(acc));
            for (unsigned int n = 0; n < kBarSpins; ++n)
                if (bar_test(acc_full(acc), acc_phase)) break;
        }
    } else if (warp < 4) {   // epilogue: thread = row of the tile
        int acc = 0;
        unsigned int acc_phase = 0;
        for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
            const int mt = static_cast<int>(t % m_tiles);
            const int nt = static_cast<int>(t / m_tiles % n_tiles);
            const int sp = static_cast<int>(t / m_tiles / n_tiles);
            const bool ok = bar_wait(acc_full(acc), acc_phase, aborted, g.status, CE_WAIT_TIMEOUT);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const int row = mt * BM + warp * 32 + lane, col0 = nt * BN;
            const uint32_t d = tmem + acc * BN + (static_cast<uint32_t>(warp * 32) << 16);
            const bool none = kb_begin(sp) == kb_begin(sp + 1);   // no product was made: zero
            if (EPI == EPI_LSE) {
                float m = -INFINITY, s = 0.0f;
                for (int c = 0; c < BN && col0 + c < g.n; c += 32) {
                    float v[32];
                    tmem_load32(d + c, v);
                    if (col0 + c + 32 > g.n)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (col0 + c + j >= g.n) v[j] = -INFINITY;
                    float top = m;
#pragma unroll
                    for (int j = 0; j < 32; ++j) top = fmaxf(top, v[j]);
                    const float ref = top == -INFINITY ? 0.0f : top * kLog2e;
                    s *= ex2(m * kLog2e - ref);
#pragma unroll
                    for (int j = 0; j < 32; ++j) s += ex2(fmaf(v[j], kLog2e, -ref));
                    m = top;
                }
                if (row < m_ext)
                    g.partial[static_cast<long long>(row) * n_tiles + nt] = make_float2(m, s);
            } else if (EPI == EPI_GRAD) {
                const bool in = row < m_ext;
                const long long want = in ? g.ptarget[row] - g.n0 - col0 : -1;
                const float lse2 = in ? g.plse2[row] : 0.0f, dl = in ? g.pdloss[row] : 0.0f;
                uint32_t *to = reinterpret_cast<uint32_t *>(
                    static_cast<unsigned short *>(g.grad) + static_cast<long long>(row) * g.ld + col0);
                for (int c = 0; c < BN; c += 32) {
                    float v[32];
                    tmem_load32(d + c, v);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float p = ex2(fmaf(v[j], kLog2e, -lse2));
                        const float q = (want == c + j ? p - 1.0f : p) * dl;
                        v[j] = in && col0 + c + j < g.n ? q : 0.0f;
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 8)
                        *reinterpret_cast<uint4 *>(to + (c + j) / 2) = make_uint4(
                            pack2(g.bf16, v[j], v[j + 1]), pack2(g.bf16, v[j + 2], v[j + 3]),
                            pack2(g.bf16, v[j + 4], v[j + 5]), pack2(g.bf16, v[j + 6], v[j + 7]));
                }
            } else if (EPI == EPI_DWEIGHT) {
                const float f = g.state->unscale;
                unsigned short *to = static_cast<unsigned short *>(g.out) +
                                     static_cast<long long>(row) * g.ld + col0;
                const bool vec = (g.ld % 8 == 0) && (reinterpret_cast<uintptr_t>(g.out) % 16 == 0);
                for (int c = 0; c < BN && col0 + c < g.n; c += 32) {
                    float v[32];
                    tmem_load32(d + c, v);
                    if (row >= g.m) continue;
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = none ? 0.0f : v[j] * f;
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        const uint4 q = make_uint4(
                            pack2(g.bf16, v[j], v[j + 1]), pack2(g.bf16, v[j + 2], v[j + 3]),
                            pack2(g.bf16, v[j + 4], v[j + 5]), pack2(g.bf16, v[j + 6], v[j + 7]));
                        if (vec && col0 + c + j < g.n) {
                            *reinterpret_cast<uint4 *>(to + c + j) = q;
                        } else {
                            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (col0 + c + j + e < g.n)
                                    to[c + j + e] = static_cast<unsigned short>(
                                        w[e / 2] >> (16 * (e & 1)));
                        }
                    }
                }
            } else {   // EPI_DX: FP32, ld a multiple of 4, rows of whole vectors
                float *to = static_cast<float *>(g.out) + sp * g.slice +
                            static_cast<long long>(row) * g.ld + col0;
                for (int c = 0; c < BN && col0 + c < g.ld; c += 32) {
                    float v[32];
                    tmem_load32(d + c, v);
                    if (row >= m_ext) continue;
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        if (col0 + c + j >= g.ld) break;
                        float4 q = none ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                                        : make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                        float4 *p = reinterpret_cast<float4 *>(to + c + j);
                        if (g.accumulate) {
                            const float4 o = *p;
                            q = make_float4(q.x + o.x, q.y + o.y, q.z + o.z, q.w + o.w);
                        }
                        *p = q;
                    }
                }
            }
            tc_fence_before();
            bar_arrive(acc_empty(acc));
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) tmem_free(tmem, 512);
}

// ---- forward: joining the tiles --------------------------------------------------

template <class T>
__device__ __forceinline__ float widen16(unsigned int bits) {
    if constexpr (std::is_same<T, __half>::value)
        return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
    else
        return __uint_as_float(bits << 16);
}

// sum_h x[h] w[h] over the lanes of a warp (every lane gets it).
template <class T>
__device__ __forceinline__ float warp_dot(const unsigned short *x, const unsigned short *w, int n,
                                          int lane) {
    float t = 0.0f;
    if (((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w)) & 15) == 0) {
        const int vectors = n / 8;
#pragma unroll 4
        for (int i = lane; i < vectors; i += 32) {
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(x) + i);
            const uint4 b = __ldg(reinterpret_cast<const uint4 *>(w) + i);
            const unsigned int p[4] = {a.x, a.y, a.z, a.w}, q[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                t = fmaf(widen16<T>(p[j] & 0xffffu), widen16<T>(q[j] & 0xffffu), t);
                t = fmaf(widen16<T>(p[j] >> 16), widen16<T>(q[j] >> 16), t);
            }
        }
        x += vectors * 8;
        w += vectors * 8;
        n -= vectors * 8;
    }
    for (int i = lane; i < n; i += 32) t = fmaf(widen16<T>(x[i]), widen16<T>(w[i]), t);
    for (int d = 16; d > 0; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
    return t;
}

struct JoinArgs {
    const float2 *partial;
    const unsigned short *x, *weight;
    const long long *target;
    long long ignore;
    int rows, width, vocab, n_tiles;
    float *loss, *lse;
    unsigned int *status;
};

// One warp a row: lanes over the n tiles, joined in a fixed tree.
template <class T>
__global__ void __launch_bounds__(256) join_lse_kernel(const JoinArgs a) {
    const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (row >= a.rows) return;
    const long long t = a.target[row];
    if (t == a.ignore) {
        if (lane == 0) a.loss[row] = a.lse[row] = 0.0f;
        return;
    }
    const float2 *p = a.partial + static_cast<long long>(row) * a.n_tiles;
    float m = -INFINITY;
    for (int i = lane; i < a.n_tiles; i += 32) m = fmaxf(m, p[i].x);
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float ref = m == -INFINITY ? 0.0f : m;
    float s = 0.0f;
    for (int i = lane; i < a.n_tiles; i += 32) {
        const float2 q = p[i];
        s += q.y * expf(q.x - ref);
    }
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float log_s = logf(s);
    const bool in = t >= 0 && t < a.vocab;
    const float l = in ? warp_dot<T>(a.x + static_cast<long long>(row) * a.width,
                                     a.weight + t * a.width, a.width, lane)
                       : NAN;
    if (lane != 0) return;
    a.lse[row] = m + log_s;
    a.loss[row] = (m - l) + log_s;   // m - l is exact where they are close
    if (!in) atomicOr(a.status, CE_BAD_TARGET);
}

// ---- backward: packing rows ----------------------------------------------------------

__device__ __forceinline__ bool counts(long long t, long long ignore, int vocab, float dl) {
    return t != ignore && t >= 0 && t < vocab && dl != 0.0f;
}

// One CTA: place[i] = position of row i among the rows that count, or -1;
// row_of, target, lse and dloss of the packed rows.  dloss is held over its
// largest magnitude: the equal weights of a mean become 1, so that the
// 16-bit gradients round p - onehot and not its product with, say, 1 / 48,
// which is off by the same 2^-9 in every row's largest entry (dx of 48 rows
// was 2.6e-3 off in the 2-norm with dloss in it, 2.0e-3 without; the output's
// own rounding is 1.7e-3).  FP16 gradients are scaled by 2^15 too: |p -
// onehot| <= 1, so nothing overflows, and what underflows is below 2^-40 of
// the largest.
__global__ void __launch_bounds__(1024)
    place_rows_kernel(const long long *target, const float *lse, const float *dloss,
                      long long ignore, int rows, int vocab, int scaled, CeState *state,
                      int *place, int *row_of, int *ptarget, float *plse2, float *pdloss,
                      unsigned int *status) {
    __shared__ int warp_count[32];
    __shared__ float warp_top[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (rows + 1023) / 1024;
    const int begin = min(rows, tid * per), end = min(rows, begin + per);
    int n = 0;
    float top = 0.0f;
    for (int i = begin; i < end; ++i) {
        const long long t = target[i];
        const float dl = dloss[i];
        if (t != ignore && (t < 0 || t >= vocab)) atomicOr(status, CE_BAD_TARGET);
        if (counts(t, ignore, vocab, dl)) {
            ++n;
            if (isfinite(dl)) top = fmaxf(top, fabsf(dl));
        }
    }
    int before = n;
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += o;
    }
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (lane == 31) warp_count[warp] = before;
    if (lane == 0) warp_top[warp] = top;
    __syncthreads();
    int at = before - n, total = 0;
    top = 0.0f;
    for (int i = 0; i < 32; ++i) {
        if (i < warp) at += warp_count[i];
        total += warp_count[i];
        top = fmaxf(top, warp_top[i]);
    }
    // 32768 / top and top / 32768 are finite and not 0 for any normal top
    top = fminf(fmaxf(top, 1e-30f), 1e30f);
    const float full = scaled ? 32768.0f : 1.0f;
    for (int i = begin; i < end; ++i) {
        const long long t = target[i];
        const float dl = dloss[i];
        if (counts(t, ignore, vocab, dl)) {
            place[i] = at;
            row_of[at] = i;
            ptarget[at] = static_cast<int>(t);
            plse2[at] = lse[i] * kLog2e;
            pdloss[at] = full * (dl / top);
            ++at;
        } else {
            place[i] = -1;
        }
    }
    if (tid == 0) {
        state->valid = total;
        state->unscale = top / full;
    }
}

// to[i] = from[row_of[i]] (i itself without row_of), rows of `width`
// two-byte elements into rows of `ld` (a multiple of 8), padded with zeros;
// rows from state->valid on are zero.
__global__ void __launch_bounds__(256)
    pack_rows_kernel(const unsigned short *from, unsigned short *to, long long rows, int width, int ld,
                     const int *row_of, const CeState *state) {
    const int per_row = ld / 8;
    const long long n = rows * per_row;
    const long long valid = state != nullptr ? state->valid : rows;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        const long long r = i / per_row;
        const int c = static_cast<int>(i % per_row) * 8;
        uint4 q = make_uint4(0, 0, 0, 0);
        if (r < valid) {
            const unsigned short *p = from + (row_of != nullptr ? row_of[r] : r) * width + c;
            if (width == ld) {
                q = *reinterpret_cast<const uint4 *>(p);
            } else {
                unsigned int w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = c + j < width ? p[j] : 0u;
                q = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16,
                               w[6] | w[7] << 16);
            }
        }
        *reinterpret_cast<uint4 *>(to + r * ld + c) = q;
    }
}

// dx[i] = the sum of the slices' rows place[i], scaled back and rounded; 0
// for rows that do not count.
__global__ void __launch_bounds__(256)
    finish_dx_kernel(const float *acc, int splits, long long slice, int acc_ld, const int *place,
                     const CeState *state, int bf16, unsigned short *dx, int rows, int width) {
    const long long n = static_cast<long long>(rows) * width;
    const float f = state->unscale;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        const long long r = i / width;
        const int c = static_cast<int>(i % width);
        const int p = place[r];
        float t = 0.0f;
        if (p >= 0)
            for (int s = 0; s < splits; ++s)
                t += acc[s * slice + static_cast<long long>(p) * acc_ld + c];
        dx[i] = static_cast<unsigned short>(pack2(bf16, t * f, 0.0f));
    }
}

// ---- host ---------------------------------------------------------------------------

long long up(long long v, long long to) { return (v + to - 1) / to * to; }

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static std::atomic<void *> cached{nullptr};
    void *p = cached.load(std::memory_order_acquire);
    if (p == nullptr) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        cached.store(p, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(p);
}

// Map of a [rows][cols] matrix of two-byte elements, ld elements a row, in
// 128-byte-swizzled boxes of 64 columns and box_rows rows.
cudaError_t make_map(CUtensorMap *map, int bf16, const void *p, long long rows, long long cols,
                     long long ld, int box_rows) {
    const EncodeTiled encode = encode_tiled();
    if (encode == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t ones[2] = {1, 1};
    const CUresult r =
        encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
               const_cast<void *>(p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <bool A_MN, bool B_MN, int EPI>
cudaError_t launch_gemm(const CUtensorMap &a, const CUtensorMap &b, const GemmArgs &g,
                        cudaStream_t stream) {
    static std::atomic<int> ready[kMaxDevices];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (ready[dev].load(std::memory_order_acquire) == 0) {
        err = cudaFuncSetAttribute(gemm_kernel<A_MN, B_MN, EPI>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, GEMM_SMEM);
        if (err != cudaSuccess) return err;
        ready[dev].store(1, std::memory_order_release);
    }
    const long long tiles = (up(g.m, BM) / BM) * (up(g.n, BN) / BN) * (EPI == EPI_DX ? g.splits : 1);
    long long grid = sm_count_of_device();
    if (grid > tiles) grid = tiles;
    gemm_kernel<A_MN, B_MN, EPI>
        <<<static_cast<unsigned>(grid), GEMM_THREADS, GEMM_SMEM, stream>>>(a, b, g);
    return cudaGetLastError();
}

// Parts of a workspace, in order, each on 256 bytes.
struct Carver {
    unsigned char *p;
    size_t at;
    template <class T>
    T *take(long long n) {
        T *r = reinterpret_cast<T *>(p + at);
        at += static_cast<size_t>(up(n * static_cast<long long>(sizeof(T)), 256));
        return r;
    }
};

// Rows of an odd width are copied to rows of a multiple of 8 elements (TMA
// wants strides of 16 bytes).
bool odd_rows(int width) { return width % 8 != 0; }

struct ForwardSpace {
    unsigned short *x, *w;
    float2 *partial;
    size_t bytes;
};

ForwardSpace forward_space(void *ws, int rows, int width, int vocab) {
    Carver c{static_cast<unsigned char *>(ws), 0};
    ForwardSpace s;
    const long long ld = up(width, 8);
    s.x = s.w = nullptr;
    if (odd_rows(width)) {
        s.x = c.take<unsigned short>(rows * ld);
        s.w = c.take<unsigned short>(vocab * ld);
    }
    s.partial = c.take<float2>(rows * (up(vocab, BN) / BN));
    s.bytes = c.at;
    return s;
}

// A piece of the vocabulary: as many columns as keep its 16-bit gradients
// within 512 MiB, at least 4096 (each piece adds to the FP32 dx once more).
long long piece_of(int rows, int vocab) {
    long long n = (512ll << 20) / (2 * up(rows, BM)) / BN * BN;
    if (n < 4096) n = 4096;
    return n < up(vocab, BN) ? n : up(vocab, BN);
}

// Parts of a dx product's reduction: where its tiles alone would leave SMs
// idle, the vocabulary is split, in parts of at least 512 columns.
int splits_of(int rows, int width, int vocab) {
    const long long tiles = up(rows, BM) / BM * (up(width, BN) / BN);
    long long s = 152 / tiles;
    const long long most = piece_of(rows, vocab) / 512;
    if (s > most) s = most;
    return s < 1 ? 1 : static_cast<int>(s);
}

struct BackwardSpace {
    CeState *state;
    int *place, *row_of, *ptarget;
    float *plse2, *pdloss;
    unsigned short *x, *w, *grad;
    float *acc;
    size_t bytes;
};

BackwardSpace backward_space(void *ws, int rows, int width, int vocab) {
    Carver c{static_cast<unsigned char *>(ws), 0};
    BackwardSpace s;
    const long long ld = up(width, 8);
    s.state = c.take<CeState>(1);
    s.place = c.take<int>(rows);
    s.row_of = c.take<int>(rows);
    s.ptarget = c.take<int>(rows);
    s.plse2 = c.take<float>(rows);
    s.pdloss = c.take<float>(rows);
    s.x = c.take<unsigned short>(rows * ld);
    s.w = odd_rows(width) ? c.take<unsigned short>(vocab * ld) : nullptr;
    s.grad = c.take<unsigned short>(up(rows, BM) * piece_of(rows, vocab));
    s.acc = c.take<float>(splits_of(rows, width, vocab) * up(rows, BM) * up(width, 4));
    s.bytes = c.at;
    return s;
}

unsigned grid_for(long long items) {
    long long b = (items + 255) / 256;
    const long long cap = 152 * 16;
    return static_cast<unsigned>(b < 1 ? 1 : b > cap ? cap : b);
}

}  // namespace

size_t linear_ce_workspace(int rows, int width, int vocab) {
    return forward_space(nullptr, rows, width, vocab).bytes;
}

size_t linear_ce_backward_workspace(int rows, int width, int vocab) {
    return backward_space(nullptr, rows, width, vocab).bytes;
}

#define CE_TRY(call)                            \
    do {                                        \
        const cudaError_t err_ = (call);        \
        if (err_ != cudaSuccess) return err_;   \
    } while (0)

cudaError_t launch_linear_ce(const LinearCeArgs &args, cudaStream_t stream) {
    cudaError_t err = cudaSuccess;
    unsigned int *status = status_address(&err);
    if (status == nullptr) return err;
    const int rows = args.rows, width = args.width, vocab = args.vocab;
    const int bf16 = args.elem == ELEM_BF16;
    const ForwardSpace s = forward_space(args.ws, rows, width, vocab);
    const long long ld = up(width, 8);
    const void *x = args.x, *w = args.weight;
    if (odd_rows(width)) {
        pack_rows_kernel<<<grid_for(rows * ld / 8), 256, 0, stream>>>(
            static_cast<const unsigned short *>(x), s.x, rows, width, static_cast<int>(ld), nullptr,
            nullptr);
        pack_rows_kernel<<<grid_for(vocab * ld / 8), 256, 0, stream>>>(
            static_cast<const unsigned short *>(w), s.w, vocab, width, static_cast<int>(ld), nullptr,
            nullptr);
        CE_TRY(cudaGetLastError());
        x = s.x;
        w = s.w;
    }
    CUtensorMap ma, mb;
    CE_TRY(make_map(&ma, bf16, x, rows, width, ld, BM));
    CE_TRY(make_map(&mb, bf16, w, vocab, width, ld, BN));
    GemmArgs g = {};
    g.m = rows;
    g.n = vocab;
    g.k = width;
    g.bf16 = bf16;
    g.partial = s.partial;
    g.status = status;
    CE_TRY((launch_gemm<false, false, EPI_LSE>(ma, mb, g, stream)));
    const JoinArgs j = {s.partial, static_cast<const unsigned short *>(args.x),
                        static_cast<const unsigned short *>(args.weight), args.target, args.ignore,
                        rows, width, vocab, static_cast<int>(up(vocab, BN) / BN), args.loss,
                        args.lse, status};
    if (bf16)
        join_lse_kernel<__nv_bfloat16><<<(rows + 7) / 8, 256, 0, stream>>>(j);
    else
        join_lse_kernel<__half><<<(rows + 7) / 8, 256, 0, stream>>>(j);
    return cudaGetLastError();
}

cudaError_t launch_linear_ce_backward(const LinearCeArgs &args, cudaStream_t stream) {
    cudaError_t err = cudaSuccess;
    unsigned int *status = status_address(&err);
    if (status == nullptr) return err;
    const int rows = args.rows, width = args.width, vocab = args.vocab;
    const int bf16 = args.elem == ELEM_BF16;
    const BackwardSpace s = backward_space(args.ws, rows, width, vocab);
    const long long ld = up(width, 8), piece = piece_of(rows, vocab), acc_ld = up(width, 4);
    const int splits = splits_of(rows, width, vocab);
    place_rows_kernel<<<1, 1024, 0, stream>>>(args.target, args.lse, args.dloss, args.ignore, rows,
                                              vocab, !bf16, s.state, s.place, s.row_of, s.ptarget,
                                              s.plse2, s.pdloss, status);
    pack_rows_kernel<<<grid_for(rows * ld / 8), 256, 0, stream>>>(
        static_cast<const unsigned short *>(args.x), s.x, rows, width, static_cast<int>(ld),
        s.row_of, s.state);
    const unsigned short *w = static_cast<const unsigned short *>(args.weight);
    if (odd_rows(width)) {
        pack_rows_kernel<<<grid_for(vocab * ld / 8), 256, 0, stream>>>(
            w, s.w, vocab, width, static_cast<int>(ld), nullptr, nullptr);
        w = s.w;
    }
    CE_TRY(cudaGetLastError());
    CUtensorMap x_k, x_mn, grad_k, grad_mn;
    CE_TRY(make_map(&x_k, bf16, s.x, rows, width, ld, BM));
    CE_TRY(make_map(&x_mn, bf16, s.x, rows, width, ld, BK));
    CE_TRY(make_map(&grad_k, bf16, s.grad, up(rows, BM), piece, piece, BM));
    CE_TRY(make_map(&grad_mn, bf16, s.grad, up(rows, BM), piece, piece, BK));
    for (long long n0 = 0; n0 < vocab; n0 += piece) {
        const int n = static_cast<int>(vocab - n0 < piece ? vocab - n0 : piece);
        CUtensorMap w_k, w_mn;
        CE_TRY(make_map(&w_k, bf16, w + n0 * ld, n, width, ld, BN));
        CE_TRY(make_map(&w_mn, bf16, w + n0 * ld, n, width, ld, BK));
        GemmArgs g = {};
        g.state = s.state;
        g.bf16 = bf16;
        g.status = status;
        g.m = rows;
        g.n = n;
        g.k = width;
        g.ptarget = s.ptarget;
        g.plse2 = s.plse2;
        g.pdloss = s.pdloss;
        g.grad = s.grad;
        g.ld = piece;
        g.n0 = static_cast<int>(n0);
        CE_TRY((launch_gemm<false, false, EPI_GRAD>(x_k, w_k, g, stream)));
        if (args.dweight != nullptr) {
            g.m = n;
            g.n = width;
            g.k = rows;
            g.out = static_cast<unsigned short *>(args.dweight) + n0 * width;
            g.ld = width;
            CE_TRY((launch_gemm<true, true, EPI_DWEIGHT>(grad_mn, x_mn, g, stream)));
        }
        if (args.dx != nullptr) {
            g.m = rows;
            g.n = width;
            g.k = n;
            g.out = s.acc;
            g.ld = acc_ld;
            g.accumulate = n0 > 0;
            g.splits = splits;
            g.slice = up(rows, BM) * acc_ld;
            CE_TRY((launch_gemm<false, true, EPI_DX>(grad_k, w_mn, g, stream)));
        }
    }
    if (args.dx != nullptr) {
        finish_dx_kernel<<<grid_for(static_cast<long long>(rows) * width), 256, 0, stream>>>(
            s.acc, splits, up(rows, BM) * acc_ld, static_cast<int>(acc_ld), s.place, s.state, bf16,
            static_cast<unsigned short *>(args.dx), rows, width);
        CE_TRY(cudaGetLastError());
    }
    return cudaSuccess;
}

}  // namespace tile
