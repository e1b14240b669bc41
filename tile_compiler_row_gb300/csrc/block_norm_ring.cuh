// Block norm, backward: the kernel for rows of up to 8 CTAs' shared memory
// (block_norm_bwd.cu has the formulas and the fallback for wider rows).
//
// A program (one CTA, or a cluster of C that split the columns) walks over a
// contiguous range of rows.  Thread 0 copies the rows of the four inputs
// into a ring of shared-memory slots, one row a slot, with the bulk copy
// engine; every thread reads a row twice, once for its sums and once for its
// outputs, and its warp hands the slot back.  What a thread keeps in
// registers is only the parameters and the column sums of its 8 or 16
// columns, so the bytes in flight do not depend on registers.  (A warp of
// its own for the copies would leave 512 threads 96 registers instead of
// 128.)
//
// V = 1 (odd widths, pointers off 16 bytes): a slot holds the 16-byte blocks
// that cover the row, and a thread reads single elements at the row's
// offset in it.  The blocks that reach outside the matrix, at its first and
// last elements, are not copied; threads put their elements into the slot.
//
// A cluster adds its CTAs' sums by writing each CTA's six partial sums into
// every CTA (st.async on an mbarrier): no cluster-wide barrier in the loop.
//
// Waits are bounded: one that runs out sets the device status word and an
// abort flag, after which no thread of the CTA waits and nothing is copied;
// the outputs are then invalid, and the call ends.
#pragma once

#include "block_norm.cuh"
#include "tcgen05.cuh"

namespace tile {

enum { BLOCK_WAIT_TIMEOUT = 2u };

// Column sums of a program in the workspace [unit][slot][width].
enum { SLOT_PRE = 0, SLOT_POST = 1, SLOT_FIRST = 2, SLOT_LAST = 3, SLOTS = 4 };

constexpr int kRingMost = 8;   // slots

struct RingPlan {
    int workers;    // W: threads of a CTA
    int cluster;    // C
    int slots;
    int pitch;      // bytes of a slot's part for one input
    int smem;
};

// Six sums over the warp, by halving the set of values as the distance
// doubles: values 0..7 (two unused), so lane l ends with value l >> 2 & 7
// summed over the lanes that agree with it in l & 3, and two steps more
// join those.
__device__ __forceinline__ float warp_sum6(const float (&s)[6], int lane) {
    float a[4], b[2], c;
    const bool h16 = lane & 16, h8 = lane & 8, h4 = lane & 4;
    const float t[8] = {s[0], s[1], s[2], s[3], s[4], s[5], 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        a[i] = (h16 ? t[4 + i] : t[i]) + __shfl_xor_sync(0xffffffffu, h16 ? t[i] : t[4 + i], 16);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        b[i] = (h8 ? a[2 + i] : a[i]) + __shfl_xor_sync(0xffffffffu, h8 ? a[i] : a[2 + i], 8);
    c = (h4 ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, h4 ? b[0] : b[1], 4);
    c += __shfl_xor_sync(0xffffffffu, c, 2);
    c += __shfl_xor_sync(0xffffffffu, c, 1);
    return c;   // of value lane >> 2
}

__device__ __forceinline__ uint4 shared_raw(uint32_t at, uint4) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ unsigned int shared_raw(uint32_t at, unsigned int) {
    unsigned int v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ unsigned short shared_raw(uint32_t at, unsigned short) {
    unsigned short v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
    return v;
}

template <class T, int V, int E, bool CL>
__global__ void __launch_bounds__(512)
    block_norm_ring_kernel(const BlockArgs a, const RingPlan plan) {
    using A = Access<T, V>;
    constexpr int K = E / V;
    constexpr int G = V == 1 ? 2 : V, GK = G / V;   // columns handled together, in GK groups
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ __align__(16) float warp_part[2][6][16];
    __shared__ __align__(16) float cta_part[2][8][8];
    __shared__ __align__(8) uint64_t full[kRingMost], empty[kRingMost], peer[2];
    __shared__ int abort_flag;
    const int W = plan.workers, warps = W >> 5, slots = plan.slots;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = CL ? plan.cluster : 1;
    const int rank = CL ? static_cast<int>(cluster_rank()) : 0;
    volatile int *aborted = &abort_flag;

    // unused warps' partial sums stay 0
    for (int i = tid; i < 2 * 6 * 16; i += blockDim.x) (&warp_part[0][0][0])[i] = 0.0f;
    for (int i = tid; i < 2 * 8 * 8; i += blockDim.x) (&cta_part[0][0][0])[i] = 0.0f;
    if (tid == 0) {
        abort_flag = 0;
        for (int s = 0; s < slots; ++s) {
            bar_init(smem_u32(&full[s]), 1);
            bar_init(smem_u32(&empty[s]), warps);
        }
        bar_init(smem_u32(&peer[0]), 1);
        bar_init(smem_u32(&peer[1]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if constexpr (CL) cluster_barrier();

    const long long units = gridDim.x / C, unit = blockIdx.x / C;
    const long long begin = a.rows * unit / units, end = a.rows * (unit + 1) / units;
    const int col0 = rank * W * E;                           // this CTA's columns
    const int cols = a.width - col0 < W * E ? a.width - col0 : W * E;
    const bool has_x = a.post || a.gate != nullptr, has_dh = a.dhidden != nullptr;
    const void *const base[4] = {a.x, a.hidden, a.dhidden, a.dout};
    const bool use[4] = {has_x, a.pre != 0, has_dh, a.pre != 0};
    // bytes [from, to) of input t's part of a row, and the whole 16-byte
    // blocks inside the matrix that hold them
    struct Part {
        uintptr_t from, to, copy_from, copy_to;
    };
    auto part_of = [&](int t, long long row) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(base[t]);
        const uintptr_t hi = lo + static_cast<uintptr_t>(a.rows) * a.width * sizeof(T);
        Part p;
        p.from = lo + (static_cast<uintptr_t>(row) * a.width + col0) * sizeof(T);
        p.to = p.from + cols * sizeof(T);
        p.copy_from = p.from & ~static_cast<uintptr_t>(15);
        if (p.copy_from < lo) p.copy_from += 16;
        p.copy_to = (p.to + 15) & ~static_cast<uintptr_t>(15);
        if (p.copy_to > hi) p.copy_to -= 16;
        if (p.copy_to < p.copy_from) p.copy_to = p.copy_from;
        return p;
    };
    const uint32_t ring0 = smem_u32(ring);
    // thread 0: the copies of a row into its slot, each block at its offset
    // from the row's first block
    auto copy_row = [&](long long row, int s) {
        unsigned int bytes = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (use[t]) {
                const Part p = part_of(t, row);
                bytes += static_cast<unsigned int>(p.copy_to - p.copy_from);
            }
        bar_expect_tx(smem_u32(&full[s]), bytes);
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (use[t]) {
                const Part p = part_of(t, row);
                const unsigned int n = static_cast<unsigned int>(p.copy_to - p.copy_from);
                if (n > 0)
                    asm volatile(
                        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
                        "[%1], %2, [%3];" ::"r"(
                            ring0 + (s * 4 + t) * plan.pitch +
                            static_cast<uint32_t>(p.copy_from - (p.from & ~static_cast<uintptr_t>(15)))),
                        "l"(p.copy_from), "r"(n), "r"(smem_u32(&full[s]))
                        : "memory");
            }
    };
    long long issued = 0;   // thread 0: rows copied
    if (tid == 0)
        for (; issued < slots && begin + issued < end; ++issued)
            copy_row(begin + issued, static_cast<int>(issued));

    T *din = static_cast<T *>(a.din), *dres = static_cast<T *>(a.dresidual);
    const float inv_n = 1.0f / static_cast<float>(a.width);
    auto column = [&](int k) { return col0 + (k * W + tid) * V; };   // first of vector k
    float g2[E], w[E], sum_pre[E], sum_gate[E];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float p[V];
        if (column(k) < a.width) load_params<V>(a.gamma_pre, column(k), p);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            g2[k * V + j] = column(k) < a.width ? p[j] : 0.0f;
            w[k * V + j] = sum_pre[k * V + j] = sum_gate[k * V + j] = 0.0f;
        }
    }
    float *part = a.ws + unit * SLOTS * a.width;
    const long long first_gate = begin / a.per_gate;
    long long gate_row = first_gate - 1, gate_end = begin;
    for (long long row = begin; row < end; ++row) {
        const long long i_row = row - begin;
        const int s = static_cast<int>(i_row % slots);
        if (row == gate_end) {
            gate_row = row / a.per_gate;
            gate_end = (gate_row + 1) * a.per_gate;
            const float *gate = a.gate != nullptr ? a.gate + gate_row * a.width : nullptr;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (column(k) < a.width) {
                    float p[V], q[V];
                    load_params<V>(a.gamma_post, column(k), p);
                    load_params<V>(gate, column(k), q);
#pragma unroll
                    for (int j = 0; j < V; ++j) w[k * V + j] = p[j] * q[j];
                }
        }
        // the slot that the row before freed takes the next row
        if (tid == 0 && i_row > 0 && begin + issued < end) {
            const int f = static_cast<int>((i_row - 1) % slots);
            if (bar_wait(smem_u32(&empty[f]), static_cast<unsigned int>((i_row - 1) / slots) & 1u,
                         aborted, a.status, BLOCK_WAIT_TIMEOUT)) {
                copy_row(begin + issued, f);
                ++issued;
            }
        }
        __syncwarp();
        // where this thread's elements lie in the slot, for each input
        uint32_t at[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            at[t] = ring0 + (s * 4 + t) * plan.pitch + tid * V * static_cast<int>(sizeof(T));
            if (V == 1)
                at[t] += (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(base[t])) +
                          (static_cast<uint32_t>(row) * static_cast<uint32_t>(a.width) + col0) *
                              static_cast<uint32_t>(sizeof(T))) & 15u;
        }
        // columns of groups k .. k + GK - 1 of input t, 0 where it has none
        auto fetch = [&](int t, int k, float (&v)[G]) {
#pragma unroll
            for (int u = 0; u < GK; ++u) {
                typename A::Raw r{};
                if (use[t] && (V > 1 || column(k + u) < a.width))
                    r = shared_raw(at[t] + (k + u) * W * V * static_cast<int>(sizeof(T)),
                                   typename A::Raw{});
                float q[V];
                A::widen(r, q);
#pragma unroll
                for (int j = 0; j < V; ++j) v[u * V + j] = q[j];
            }
        };
        bar_wait(smem_u32(&full[s]), static_cast<unsigned int>(i_row / slots) & 1u, aborted,
                 a.status, BLOCK_WAIT_TIMEOUT);
        constexpr int kMost = 16 / sizeof(T);   // elements of a block
        if (V == 1 && (row * a.width < kMost || (a.rows - 1 - row) * a.width < kMost)) {
            // elements outside the copied blocks: at most 15 bytes at each end
            for (int i = tid; i < 4 * 2 * kMost; i += W) {
                const int t = i / (2 * kMost), e = i % kMost;
                if (!use[t]) continue;
                const Part p = part_of(t, row);
                const bool tail = (i / kMost) & 1;
                const uintptr_t from = tail ? (p.copy_to > p.from ? p.copy_to : p.from) : p.from;
                const uintptr_t to = tail ? p.to : (p.copy_from < p.to ? p.copy_from : p.to);
                const uintptr_t g = from + e * sizeof(T);
                if (g < to) {
                    const uint32_t d = ring0 + (s * 4 + t) * plan.pitch +
                                       static_cast<uint32_t>(g - (p.from & ~static_cast<uintptr_t>(15)));
                    if constexpr (sizeof(T) == 4)
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(d),
                                     "r"(*reinterpret_cast<const unsigned int *>(g)) : "memory");
                    else
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"(d),
                                     "h"(*reinterpret_cast<const unsigned short *>(g)) : "memory");
                }
            }
            // before a later copy into the slot, and for the threads that read
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            if (warps > 1)
                asm volatile("bar.sync 1, %0;" ::"r"(W) : "memory");
            else
                __syncwarp();
        }
        F2 acc[6] = {};   // h^2, gy h, b^2, w b dh, w b gy, w b h
#pragma unroll
        for (int k = 0; k < K; k += GK) {
            if (column(k) >= a.width) continue;
            float b[G], h[G], dh[G], dy[G];
            fetch(0, k, b);
            fetch(1, k, h);
            fetch(2, k, dh);
            fetch(3, k, dy);
#pragma unroll
            for (int i = 0; i < G / 2; ++i) {
                const int c = k * V / 2 + i;
                const F2 gy = mul2(pair(dy, i), pair(g2, c)), wb = mul2(pair(b, i), pair(w, c));
                acc[0] = fma2(pair(h, i), pair(h, i), acc[0]);
                acc[1] = fma2(gy, pair(h, i), acc[1]);
                acc[2] = fma2(pair(b, i), pair(b, i), acc[2]);
                acc[3] = fma2(wb, pair(dh, i), acc[3]);
                acc[4] = fma2(wb, gy, acc[4]);
                acc[5] = fma2(wb, pair(h, i), acc[5]);
            }
        }
        float sum[6];
#pragma unroll
        for (int i = 0; i < 6; ++i) sum[i] = acc[i].x + acc[i].y;
        const int turn = static_cast<int>(i_row & 1);
        const float mine = warp_sum6(sum, lane);
        if ((lane & 3) == 0 && lane < 24) warp_part[turn][lane >> 2][warp] = mine;
        if (warps > 1)
            asm volatile("bar.sync 1, %0;" ::"r"(W) : "memory");
        else
            __syncwarp();
        // the warps' partials: lane l adds four of value l >> 2, two steps
        // join the sixteen, and each value is read from one of its lanes
        const int value = (lane >> 2) < 6 ? lane >> 2 : 0;
        const float4 q = *reinterpret_cast<const float4 *>(&warp_part[turn][value][4 * (lane & 3)]);
        float joined = (q.x + q.y) + (q.z + q.w);
        joined += __shfl_xor_sync(0xffffffffu, joined, 1);
        joined += __shfl_xor_sync(0xffffffffu, joined, 2);
#pragma unroll
        for (int i = 0; i < 6; ++i) sum[i] = __shfl_sync(0xffffffffu, joined, 4 * i);
        if constexpr (CL) {
            // every CTA writes its six sums into every CTA's slot of its rank
            if (tid == 0) bar_expect_tx(smem_u32(&peer[turn]), 24u * C);
            if (tid < C) {
                const uint32_t to = smem_u32(&cta_part[turn][rank][0]), bar = smem_u32(&peer[turn]);
                uint32_t rto, rbar;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rto) : "r"(to), "r"(tid));
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                             : "=r"(rbar) : "r"(bar), "r"(tid));
#pragma unroll
                for (int i = 0; i < 6; ++i)
                    asm volatile(
                        "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, "
                        "[%2];" ::"r"(rto + 4 * i),
                        "r"(__float_as_uint(sum[i])), "r"(rbar)
                        : "memory");
            }
            bar_wait(smem_u32(&peer[turn]), static_cast<unsigned int>(i_row >> 1) & 1u, aborted,
                     a.status, BLOCK_WAIT_TIMEOUT);
            const volatile float *cp = &cta_part[turn][lane & 3][value];
            joined = cp[0] + cp[4 * 8];   // CTAs l & 3 and 4 more (0 where there are fewer)
            joined += __shfl_xor_sync(0xffffffffu, joined, 1);
            joined += __shfl_xor_sync(0xffffffffu, joined, 2);
#pragma unroll
            for (int i = 0; i < 6; ++i) sum[i] = __shfl_sync(0xffffffffu, joined, 4 * i);
        }
        // gh = dh + r2 gy - ch h,  db = r1 u - cb b
        const float r2 = a.pre ? inv_sqrt<T>(fmaf(sum[0], inv_n, a.eps)) : 0.0f;
        const float ch = r2 * r2 * r2 * (sum[1] * inv_n);
        const float r1 = a.post ? inv_sqrt<T>(fmaf(sum[2], inv_n, a.eps)) : 1.0f;
        const float ub = fmaf(r2, sum[4], sum[3]) - ch * sum[5];
        const float cb = a.post ? r1 * r1 * r1 * (ub * inv_n) : 0.0f;
        T *din_row = din + row * a.width + col0 + tid * V;
        T *dres_row = dres + row * a.width + col0 + tid * V;
#pragma unroll
        for (int k = 0; k < K; k += GK) {
            if (column(k) >= a.width) continue;
            float b[G], h[G], dh[G], dy[G], db[G], dr[G];
            fetch(0, k, b);
            fetch(1, k, h);
            fetch(2, k, dh);
            fetch(3, k, dy);
#pragma unroll
            for (int i = 0; i < G / 2; ++i) {
                const int c = k * V / 2 + i;
                const F2 gy = mul2(pair(dy, i), pair(g2, c));
                const F2 gh = fma2(pair(h, i), both(-ch), fma2(gy, both(r2), pair(dh, i)));
                put(sum_pre, c, fma2(mul2(pair(h, i), both(r2)), pair(dy, i), pair(sum_pre, c)));
                const F2 t = mul2(gh, both(r1));
                put(sum_gate, c, fma2(t, pair(b, i), pair(sum_gate, c)));
                put(dr, i, mul2(gh, both(a.scale)));
                put(db, i, fma2(t, pair(w, c), mul2(pair(b, i), both(-cb))));
            }
#pragma unroll
            for (int u = 0; u < GK; ++u)
                if (GK == 1 || column(k + u) < a.width) {
                    float o[V], q[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        o[j] = db[u * V + j];
                        q[j] = dr[u * V + j];
                    }
                    A::store(din_row + (k + u) * W * V, o);
                    A::store(dres_row + (k + u) * W * V, q);
                }
        }
        __syncwarp();
        if (lane == 0) bar_arrive(smem_u32(&empty[s]));
        // end of this gate row's part (without a gate: of the program)
        if (row + 1 == end || (a.gate != nullptr && row + 1 == gate_end)) {
            const bool first_part = gate_row == first_gate;
            const bool whole = gate_row * a.per_gate >= begin && (gate_end <= end || end == a.rows);
            const float *gate = a.gate != nullptr ? a.gate + gate_row * a.width : nullptr;
            float *seg = part + static_cast<long long>(first_part ? SLOT_FIRST : SLOT_LAST) * a.width;
            float *post = part + static_cast<long long>(SLOT_POST) * a.width;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (column(k) < a.width) {
                    float p[V], q[V];
                    load_params<V>(a.gamma_post, column(k), p);
                    load_params<V>(gate, column(k), q);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const int i = k * V + j, col = column(k) + j;
                        // read again only where a program holds several gate rows
                        if (a.dgamma_post != nullptr)
                            post[col] = fmaf(q[j], sum_gate[i], first_part ? 0.0f : post[col]);
                        if (a.dgate != nullptr) {
                            if (whole)
                                a.dgate[gate_row * a.width + col] = p[j] * sum_gate[i];
                            else
                                seg[col] = sum_gate[i];
                        }
                        sum_gate[i] = 0.0f;
                    }
                }
        }
    }
    if (a.dgamma_pre != nullptr)
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (column(k) < a.width)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    part[static_cast<long long>(SLOT_PRE) * a.width + column(k) + j] =
                        sum_pre[k * V + j];
    // an aborted CTA waits (bounded) for the copies it issued
    if (tid == 0 && *aborted)
        for (long long i = issued > slots ? issued - slots : 0; i < issued; ++i)
            for (unsigned int n = 0; n < kBarSpins; ++n)
                if (bar_test(smem_u32(&full[i % slots]), (i / slots) & 1)) break;
    __syncwarp();
    if constexpr (CL) cluster_barrier();   // no CTA leaves while a peer may write to it
}

}  // namespace tile
