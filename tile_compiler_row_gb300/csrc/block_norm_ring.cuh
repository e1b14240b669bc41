// Block norm, backward: the kernel for rows of up to 8 CTAs' shared memory
// (block_norm_bwd.cu has the formulas and the fallback for wider rows).
//
// A program (one CTA, or a cluster of C that split the columns) walks over
// rows.  Thread 0 copies the rows of the four inputs into a ring of
// shared-memory slots, one row a slot, with the bulk copy engine; every
// thread reads a row twice, once for its sums and once for its outputs.  The
// row before is out of its slot once every thread has reached a row's
// reduction, and thread 0 refills that slot then.  What a thread keeps in
// registers is only the parameters and the column sums of its 8 or 16
// columns, so the bytes in flight do not depend on registers.
//
// SHIFT (rows that are not whole vectors): rows start at one of 2, 4 or 8
// offsets into a 16-byte block, the same every so many rows.  A program takes
// rows of one such class, so each of its threads reads and writes the same
// aligned vectors of every row and owns the same columns; only the vectors
// at a row's two ends are masked.  The last block of the matrix, where it
// would reach past the end, is not copied; threads put its elements into
// the slot.
//
// Bound by memory from 4096 columns on (32768 x 4096 BF16 267 us, 6.0 TB/s),
// by the latency of a row's reduction below (8192 x 256 23 us), and with SHIFT
// by instruction issue (16384 x 4097 BF16 288 us: the masks and the stores by
// parts of the end vectors).
//
// A cluster adds its CTAs' sums by writing each CTA's six partial sums into
// every CTA (st.async on an mbarrier): no cluster-wide barrier in the loop.
//
// Waits are bounded: one that runs out sets the device status word and an
// abort flag, after which no thread of the CTA waits for a copy and nothing is
// copied; the sums are exchanged all the same, row by row.  The outputs are
// then invalid, and the call ends.
#pragma once

#include "block_norm.cuh"
#include "tcgen05.cuh"

namespace tile {

enum { BLOCK_WAIT_TIMEOUT = 2u };

// Column sums of a program in the workspace [unit][slot][width].
enum { SLOT_PRE = 0, SLOT_POST = 1, SLOT_FIRST = 2, SLOT_LAST = 3, SLOTS = 4 };

constexpr int kRingMost = 8;   // slots

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

__device__ __forceinline__ uint4 shared_vec(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

// WITHHELD (tests only): the first program's first row is not copied, and
// waits are short.
template <class T, int K, bool SHIFT, bool CL, int MAXT, int MINB, bool WITHHELD = false>
__global__ void __launch_bounds__(MAXT, MINB)
    block_norm_ring_kernel(const BlockArgs a, const RingPlan plan) {
    using X = Vec<T>;
    constexpr int N = X::N, P = X::P;   // elements, pairs of a vector
    constexpr unsigned int SPINS = WITHHELD ? kTestBarSpins : kBarSpins;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ __align__(16) float warp_part[2][6][16];
    __shared__ __align__(16) float cta_part[2][8][8];
    __shared__ __align__(8) uint64_t full[kRingMost], peer[2];
    __shared__ EdgeMasks masks;
    __shared__ int abort_flag;
    const int W = plan.workers, warps = W >> 5, slots = plan.slots;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = CL ? plan.cluster : 1;
    const int rank = CL ? static_cast<int>(cluster_rank()) : 0;
    volatile int *aborted = &abort_flag;
    const long long units = gridDim.x / C, unit = blockIdx.x / C;
    const RowWalk walk = row_walk(a.rows, a.per_gate, plan, unit, units);
    const int width = a.width;
    // elements of the rows' first block that lie before the row
    const int shift = SHIFT ? static_cast<int>((walk.first * width) & (N - 1)) : 0;

    // unused warps' and CTAs' partial sums stay 0
    for (int i = tid; i < 2 * 6 * 16; i += W) (&warp_part[0][0][0])[i] = 0.0f;
    for (int i = tid; i < 2 * 8 * 8; i += W) (&cta_part[0][0][0])[i] = 0.0f;
    if (tid == 0) {
        if (SHIFT) edge_masks<T>(masks, shift, width);
        abort_flag = 0;
        for (int s = 0; s < slots; ++s) bar_init(smem_u32(&full[s]), 1);
        bar_init(smem_u32(&peer[0]), 1);
        bar_init(smem_u32(&peer[1]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if constexpr (CL) cluster_barrier();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // this CTA's vectors of a row: [v0, v0 + nv) of those that hold it
    const int v0 = rank * W * K;
    const int vecs = (width + shift + N - 1) / N;
    const int nv = min(vecs - v0, W * K);
    const bool has_x = a.post || a.gate != nullptr, has_dh = a.dhidden != nullptr;
    const uint32_t ring0 = smem_u32(ring);
    // element of the matrix where this CTA's part of a row begins (its block)
    auto part_at = [&](long long row) { return row * width - shift + static_cast<long long>(v0) * N; };
    // thread 0: the copies of a row into its slot
    auto copy_row = [&](long long row, int s) {
        const long long at = part_at(row);
        int n = nv;
        if (SHIFT && at + static_cast<long long>(n) * N > a.rows * width) --n;
        const unsigned int bytes = n > 0 ? n * 16u : 0u;
        const uint32_t bar = smem_u32(&full[s]);
        bar_expect_tx(bar, bytes * ((has_x ? 1 : 0) + (has_dh ? 1 : 0) + (a.pre ? 2 : 0)));
        auto copy = [&](const void *from, int t) {
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, "
                "[%3];" ::"r"(ring0 + (s * 4 + t) * plan.pitch),
                "l"(static_cast<const T *>(from) + at), "r"(bytes), "r"(bar)
                : "memory");
        };
        if (bytes == 0) return;
        if (has_x) copy(a.x, 0);
        if (a.pre) copy(a.hidden, 1);
        if (has_dh) copy(a.dhidden, 2);
        if (a.pre) copy(a.dout, 3);
    };
    int issued = 0;   // thread 0: rows copied so far, at most `slots` ahead
    if (tid == 0)
        for (; issued < slots && issued < walk.count; ++issued)
            if (!WITHHELD || issued > 0 || blockIdx.x > 0) copy_row(walk.first + static_cast<long long>(issued) * walk.step, issued);

    auto first = [&](int k) { return (v0 + k * W + tid) * N - shift; };   // column of vector k
    auto mine = [&](int k) { return k * W + tid < nv; };
    auto params = [&](const float *p, int k, F2 (&v)[P]) {
        if constexpr (SHIFT) {
            params_at<N>(p, first(k), width, v);
        } else {
            float q[N];
            load_params<N>(p, first(k), q);
#pragma unroll
            for (int i = 0; i < P; ++i) v[i] = pack(q[2 * i], q[2 * i + 1]);
        }
    };
    F2 g2[K * P], w[K * P], sum_pre[K * P], sum_gate[K * P];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        F2 p[P] = {};
        if (mine(k)) params(a.gamma_pre, k, p);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            g2[k * P + i] = p[i];
            w[k * P + i] = sum_pre[k * P + i] = sum_gate[k * P + i] = 0;
        }
    }
    const float inv_n = 1.0f / static_cast<float>(width);
    float *part = a.ws + unit * SLOTS * width;
    const long long first_gate = walk.first / a.per_gate;
    long long gate_row = first_gate, gate_end = walk.first;
    int s = 0;                 // slot of the present row
    unsigned int phase = 0;    // and its barrier's phase
    for (int i_row = 0; i_row < walk.count; ++i_row) {
        const long long row = walk.first + static_cast<long long>(i_row) * walk.step;
        if (row >= gate_end) {
            gate_row = row / a.per_gate;
            gate_end = (gate_row + 1) * a.per_gate;
            const float *gate = a.gate != nullptr ? a.gate + gate_row * width : nullptr;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (mine(k)) {
                    F2 p[P], q[P];
                    params(a.gamma_post, k, p);
                    params(gate, k, q);
#pragma unroll
                    for (int i = 0; i < P; ++i) w[k * P + i] = mul2(p[i], q[i]);
                }
        }
        const uint32_t at = ring0 + s * 4 * plan.pitch + tid * 16;
        // this thread's vector k of input t, 0 where the input is not there
        auto fetch = [&](bool use, int t, int k, F2 (&v)[P]) {
            uint4 q = make_uint4(0, 0, 0, 0);
            if (use) {
                q = shared_vec(at + t * plan.pitch + k * W * 16);
                if (SHIFT) q = mask_vec(q, edge_of(v0 + k * W + tid, vecs), masks);
            }
            X::widen(q, v);
        };
        bar_wait<SPINS>(smem_u32(&full[s]), phase, aborted, a.status, BLOCK_WAIT_TIMEOUT);
        if (SHIFT && nv > 0 && part_at(row) + static_cast<long long>(nv) * N > a.rows * width) {
            // the block at the matrix's end: not copied
            if (tid < 4 * N) {
                const int t = tid / N, e = tid % N;
                const T *from = static_cast<const T *>(t == 0   ? a.x
                                                       : t == 1 ? a.hidden
                                                       : t == 2 ? a.dhidden
                                                                : a.dout);
                const long long g = part_at(row) + static_cast<long long>(nv - 1) * N + e;
                const bool use = t == 0 ? has_x : t == 2 ? has_dh : a.pre != 0;
                if (use && g < a.rows * width) {
                    const uint32_t d = ring0 + (s * 4 + t) * plan.pitch + (nv - 1) * 16 +
                                       e * static_cast<int>(sizeof(T));
                    if constexpr (sizeof(T) == 4)
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(d),
                                     "r"(*reinterpret_cast<const unsigned int *>(from + g)) : "memory");
                    else
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"(d),
                                     "h"(*reinterpret_cast<const unsigned short *>(from + g)) : "memory");
                }
            }
            // for the threads that read it, and before a later copy
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncthreads();
        }
        F2 acc[6] = {};   // h^2, gy h, b^2, w b dh, w b gy, w b h
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!mine(k)) continue;
            F2 b[P], h[P], dh[P], dy[P];
            fetch(has_x, 0, k, b);
            fetch(a.pre, 1, k, h);
            fetch(has_dh, 2, k, dh);
            fetch(a.pre, 3, k, dy);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const F2 gy = mul2(dy[i], g2[k * P + i]), wb = mul2(b[i], w[k * P + i]);
                acc[0] = fma2(h[i], h[i], acc[0]);
                acc[1] = fma2(gy, h[i], acc[1]);
                acc[2] = fma2(b[i], b[i], acc[2]);
                acc[3] = fma2(wb, dh[i], acc[3]);
                acc[4] = fma2(wb, gy, acc[4]);
                acc[5] = fma2(wb, h[i], acc[5]);
            }
        }
        float sum[6];
#pragma unroll
        for (int i = 0; i < 6; ++i) sum[i] = total(acc[i]);
        const int turn = i_row & 1;
        const float part_sum = warp_sum6(sum, lane);
        if ((lane & 3) == 0 && lane < 24) warp_part[turn][lane >> 2][warp] = part_sum;
        __syncthreads();
        // every thread is past the row before: its slot takes the next row
        if (tid == 0 && i_row > 0 && issued < walk.count && !*aborted) {
            copy_row(walk.first + static_cast<long long>(issued) * walk.step,
                     s == 0 ? slots - 1 : s - 1);
            ++issued;
        }
        __syncwarp();
        // the warps' partials: lane l adds four of value l >> 2, two steps
        // join the sixteen, and each value is read from one of its lanes
        const int value = (lane >> 2) < 6 ? lane >> 2 : 0;
        const float4 q4 = *reinterpret_cast<const float4 *>(&warp_part[turn][value][4 * (lane & 3)]);
        float joined = (q4.x + q4.y) + (q4.z + q4.w);
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
            __syncwarp();
            bar_wait_round<SPINS>(smem_u32(&peer[turn]), static_cast<unsigned int>(i_row >> 1) & 1u,
                                  aborted, a.status, BLOCK_WAIT_TIMEOUT);
            __syncwarp();
            const volatile float *cp = &cta_part[turn][lane & 3][value];
            joined = cp[0] + cp[4 * 8];   // CTAs l & 3 and 4 more (0 where there are fewer)
            joined += __shfl_xor_sync(0xffffffffu, joined, 1);
            joined += __shfl_xor_sync(0xffffffffu, joined, 2);
#pragma unroll
            for (int i = 0; i < 6; ++i) sum[i] = __shfl_sync(0xffffffffu, joined, 4 * i);
        }
        // gh = dh + r2 (gy - ch h),  db = r1 (u - cb b r1): no factor is a
        // power of r1 or r2 that rows far from 1 would take out of range
        const float r2 = a.pre ? inv_sqrt<T>(fmaf(sum[0], inv_n, a.eps)) : 0.0f;
        const float ch = r2 * (sum[1] * inv_n) * r2;
        const float r1 = a.post ? inv_sqrt<T>(fmaf(sum[2], inv_n, a.eps)) : 1.0f;
        const float ub = fmaf(r2, fmaf(-ch, sum[5], sum[4]), sum[3]);
        const float cb = a.post ? r1 * (ub * inv_n) : 0.0f;
        const F2 r1s = both(r1), r2s = both(r2), mch = both(-ch), mcb = both(-cb),
                 scale = both(a.scale);
        const long long o = part_at(row) + tid * N;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!mine(k)) continue;
            F2 b[P], h[P], dh[P], dy[P], db[P], dr[P];
            fetch(has_x, 0, k, b);
            fetch(a.pre, 1, k, h);
            fetch(has_dh, 2, k, dh);
            fetch(a.pre, 3, k, dy);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int c = k * P + i;
                const F2 gh = fma2(fma2(h[i], mch, mul2(dy[i], g2[c])), r2s, dh[i]);
                const F2 unit = mul2(b[i], r1s);
                sum_pre[c] = fma2(mul2(h[i], r2s), dy[i], sum_pre[c]);
                sum_gate[c] = fma2(gh, unit, sum_gate[c]);
                dr[i] = mul2(gh, scale);
                db[i] = mul2(fma2(unit, mcb, mul2(gh, w[c])), r1s);
            }
            T *din = static_cast<T *>(a.din) + o + k * W * N;
            T *dres = static_cast<T *>(a.dresidual) + o + k * W * N;
            if constexpr (SHIFT) {
                store_vec_at<T>(din, X::narrow(db), first(k), width);
                store_vec_at<T>(dres, X::narrow(dr), first(k), width);
            } else {
                __stcs(reinterpret_cast<uint4 *>(din), X::narrow(db));
                __stcs(reinterpret_cast<uint4 *>(dres), X::narrow(dr));
            }
        }
        if (++s == slots) {
            s = 0;
            phase ^= 1u;
        }
        // end of this gate row's part (without a gate: of the program)
        if (i_row + 1 < walk.count && (a.gate == nullptr || row + walk.step < gate_end)) continue;
        const bool first_part = gate_row == first_gate;
        const bool whole = plan.classes == 1 && gate_row * a.per_gate >= walk.first &&
                           (gate_end <= walk.first + walk.count || walk.first + walk.count == a.rows);
        const float *gate = a.gate != nullptr ? a.gate + gate_row * width : nullptr;
        float *seg = part + static_cast<long long>(first_part ? SLOT_FIRST : SLOT_LAST) * width;
        float *post = part + static_cast<long long>(SLOT_POST) * width;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!mine(k)) continue;
            F2 p[P], q[P];
            params(a.gamma_post, k, p);
            params(gate, k, q);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int col = first(k) + j;
                if (SHIFT && (col < 0 || col >= width)) continue;
                float sl, sh, pl, ph, ql, qh;
                unpack(sum_gate[k * P + j / 2], sl, sh);
                unpack(p[j / 2], pl, ph);
                unpack(q[j / 2], ql, qh);
                const float sg = j & 1 ? sh : sl, pp = j & 1 ? ph : pl, qq = j & 1 ? qh : ql;
                // read again only where a program holds several gate rows
                if (a.dgamma_post != nullptr)
                    post[col] = fmaf(qq, sg, first_part ? 0.0f : post[col]);
                if (a.dgate != nullptr) {
                    if (whole)
                        a.dgate[gate_row * width + col] = pp * sg;
                    else
                        seg[col] = sg;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < K * P; ++i) sum_gate[i] = 0;
    }
    // (a program without rows, of a short gate row: zeros)
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (!mine(k)) continue;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int col = first(k) + j;
            if (SHIFT && (col < 0 || col >= width)) continue;
            float lo, hi;
            unpack(sum_pre[k * P + j / 2], lo, hi);
            part[static_cast<long long>(SLOT_PRE) * width + col] = j & 1 ? hi : lo;
            if (SHIFT && walk.count == 0) {
                part[static_cast<long long>(SLOT_POST) * width + col] = 0.0f;
                part[static_cast<long long>(SLOT_FIRST) * width + col] = 0.0f;
            }
        }
    }
    // an aborted CTA waits (bounded) for the copies it issued
    if (tid == 0 && *aborted)
        for (int i = issued > slots ? issued - slots : 0; i < issued; ++i)
            for (unsigned int n = 0; n < SPINS; ++n)
                if (bar_test(smem_u32(&full[i % slots]), (i / slots) & 1)) break;
    __syncwarp();
    if constexpr (CL) cluster_barrier();   // no CTA leaves while a peer may write to it
}

}  // namespace tile
