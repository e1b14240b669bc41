// Block norm, backward.  With r1, r2 = 1 / sqrt(mean square + eps) of the
// block's output b and of h, w = gate * gamma_post and n the width:
//
//   gy = dy * gamma_pre
//   gh = dh + r2 gy - h r2^3 sum(gy h) / n            (the whole gradient of h)
//   dresidual = a gh,   dgamma_pre = sum_rows dy h r2
//   u  = w gh
//   db = r1 u - b r1^3 sum(u b) / n
//   S[gate row] = sum_rows gh b r1,   dgate = gamma_post S,
//   dgamma_post = sum over gate rows of gate S
//
// sum(u b) is linear in gh, so the six sums of h^2, gy h, b^2, w b dh,
// w b gy and w b h give every scalar of a row in one reduction round.
//
// Bound by DRAM: b, h, dh, dy are read once, db and dresidual written once.
// A program walks over many rows; parameters and the column sums of its
// columns stay in registers (FP32), and go to the workspace once at its end.
// Gate rows that lie within one program's range are written by it; the
// others, and the gamma sums, are joined in program order by a second
// kernel, so results do not depend on timing.
//
// block_norm_ring.cuh is the kernel for nearly every call;
// block_norm_backward_kernel here takes what that does not: the widest rows
// (above 65536 two-byte or 32768 FP32 columns, where a row of four inputs
// leaves a cluster of 8 CTAs no room for a second one), row matrices that
// are not all 16-byte aligned, and odd widths with more row classes in their
// gate rows than there may be programs (class_units).
// It loads each row into registers when its turn comes.
#include "block_norm_ring.cuh"
#include "device_status.h"

TILE_DEVICE_STATUS(block_norm_backward)

namespace tile {
namespace {

// Programs of a call: at most as many as may run at once, which the workspace
// has column sums for: registers hold no more than 16384 columns of programs on
// an SM, or 16 programs of narrow rows (40 MiB of column sums).
constexpr int kNarrow = 1024;   // columns
constexpr int kSms = 152;

// Row classes of gate rows that programs keep to (RowWalk): the limit for odd
// widths, whose programs may be more than run at once.
int class_units(int width) { return width <= kNarrow ? 16 * kSms : 1024; }

int most_units(int width) {
    const int resident = (kSms * 16384 + width - 1) / width;
    return resident < class_units(width) ? resident : class_units(width);
}

// As many programs as run at once (`slots`) where each has four rows and more;
// with fewer rows, four rows to a program, but a program for each SM; one row
// to a program where there are fewer rows than SMs.
long long units_of(const BlockArgs &a, long long slots) {
    const long long sms = sm_count_of_device();
    long long u = a.rows / 4 > slots ? slots : a.rows;
    if (a.rows / 4 <= slots && u > sms) u = a.rows / 4 > sms ? a.rows / 4 : sms;
    if (u > most_units(a.width)) u = most_units(a.width);
    return u < 1 ? 1 : u;
}

template <class T, int V, int K, bool CL>
__global__ void __launch_bounds__(512) block_norm_backward_kernel(const BlockArgs a, int cluster) {
    using A = Access<T, V>;
    constexpr int E = K * V;
    __shared__ ReduceMem<6> mem;
    const int W = blockDim.x;
    const int warps = W >> 5;
    const int rank = CL ? static_cast<int>(cluster_rank()) : 0;
    const long long units = gridDim.x / (CL ? cluster : 1);
    const long long unit = blockIdx.x / (CL ? cluster : 1);
    const long long begin = a.rows * unit / units, end = a.rows * (unit + 1) / units;
    const T *x = static_cast<const T *>(a.x), *hid = static_cast<const T *>(a.hidden);
    const T *dhid = static_cast<const T *>(a.dhidden), *dout = static_cast<const T *>(a.dout);
    T *din = static_cast<T *>(a.din), *dres = static_cast<T *>(a.dresidual);
    const float inv_n = 1.0f / static_cast<float>(a.width);
    const bool has_x = a.post || a.gate != nullptr, has_dh = dhid != nullptr;

    int col[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
        col[k] = ((k * (CL ? cluster : 1) + rank) * W + static_cast<int>(threadIdx.x)) * V;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    float g2[E], w[E], sum_pre[E], sum_post[E], sum_gate[E];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float p[V];
        if (col[k] < a.width) load_params<V>(a.gamma_pre, col[k], p);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = k * V + j;
            g2[i] = col[k] < a.width ? p[j] : 0.0f;
            w[i] = sum_pre[i] = sum_post[i] = sum_gate[i] = 0.0f;
        }
    }
    const long long first_gate = begin / a.per_gate;
    long long gate_row = first_gate - 1, gate_end = begin;
    int turn = 0;
    for (long long row = begin; row < end; ++row) {
        if (row == gate_end) {
            gate_row = row / a.per_gate;
            gate_end = (gate_row + 1) * a.per_gate;
            const float *gate = a.gate != nullptr ? a.gate + gate_row * a.width : nullptr;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (col[k] < a.width) {
                    float p[V], q[V];
                    load_params<V>(a.gamma_post, col[k], p);
                    load_params<V>(gate, col[k], q);
#pragma unroll
                    for (int j = 0; j < V; ++j) w[k * V + j] = p[j] * q[j];
                }
        }
        typename A::Raw xr[K], hr[K], dhr[K], dyr[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            xr[k] = hr[k] = dhr[k] = dyr[k] = typename A::Raw{};
            if (col[k] < a.width) {
                const long long at = row * a.width + col[k];
                if (has_x) xr[k] = A::load(x + at);
                if (a.pre) hr[k] = A::load(hid + at);
                if (has_dh) dhr[k] = A::load(dhid + at);
                if (a.pre) dyr[k] = A::load(dout + at);
            }
        }
        float s[6] = {};   // h^2, gy h, b^2, w b dh, w b gy, w b h
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float b[V], h[V], dh[V], dy[V];
            A::widen(xr[k], b);
            A::widen(hr[k], h);
            A::widen(dhr[k], dh);
            A::widen(dyr[k], dy);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float gy = dy[j] * g2[k * V + j], wb = w[k * V + j] * b[j];
                s[0] = fmaf(h[j], h[j], s[0]);
                s[1] = fmaf(gy, h[j], s[1]);
                s[2] = fmaf(b[j], b[j], s[2]);
                s[3] = fmaf(wb, dh[j], s[3]);
                s[4] = fmaf(wb, gy, s[4]);
                s[5] = fmaf(wb, h[j], s[5]);
            }
        }
        row_sum<6, CL>(s, mem, turn, warps, cluster);
        // gh = dh + r2 (gy - ch h), db = r1 (u - cb b r1), as in the ring kernel
        const float r2 = a.pre ? 1.0f / sqrtf(fmaf(s[0], inv_n, a.eps)) : 0.0f;
        const float ch = r2 * (s[1] * inv_n) * r2;
        const float r1 = a.post ? 1.0f / sqrtf(fmaf(s[2], inv_n, a.eps)) : 1.0f;
        const float ub = fmaf(r2, fmaf(-ch, s[5], s[4]), s[3]);
        const float cb = a.post ? r1 * (ub * inv_n) : 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (col[k] >= a.width) continue;
            float b[V], h[V], dh[V], dy[V], db[V], dr[V];
            A::widen(xr[k], b);
            A::widen(hr[k], h);
            A::widen(dhr[k], dh);
            A::widen(dyr[k], dy);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int i = k * V + j;
                const float gh = fmaf(r2, fmaf(-ch, h[j], dy[j] * g2[i]), dh[j]);
                const float unit = b[j] * r1;
                sum_pre[i] = fmaf(dy[j], h[j] * r2, sum_pre[i]);
                sum_gate[i] = fmaf(gh, unit, sum_gate[i]);
                dr[j] = a.scale * gh;
                db[j] = r1 * fmaf(-cb, unit, w[i] * gh);
            }
            const long long at = row * a.width + col[k];
            A::store(din + at, db);
            A::store(dres + at, dr);
        }
        if (row + 1 == end || row + 1 == gate_end) {   // end of this gate row's part
            const long long gate_begin = gate_row * a.per_gate;
            const bool whole = gate_begin >= begin && (gate_end <= end || end == a.rows);
            const int slot = gate_row == first_gate ? SLOT_FIRST : SLOT_LAST;
            float *part = a.ws + (unit * SLOTS + slot) * a.width;
            const float *gate = a.gate != nullptr ? a.gate + gate_row * a.width : nullptr;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (col[k] < a.width) {
                    float p[V], q[V];
                    load_params<V>(a.gamma_post, col[k], p);
                    load_params<V>(gate, col[k], q);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const int i = k * V + j;
                        sum_post[i] = fmaf(q[j], sum_gate[i], sum_post[i]);
                        if (a.dgate != nullptr) {
                            if (whole)
                                a.dgate[gate_row * a.width + col[k] + j] = p[j] * sum_gate[i];
                            else
                                part[col[k] + j] = sum_gate[i];
                        }
                        sum_gate[i] = 0.0f;
                    }
                }
        }
    }
    float *pre = a.ws + (unit * SLOTS + SLOT_PRE) * a.width;
    float *post = a.ws + (unit * SLOTS + SLOT_POST) * a.width;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (col[k] < a.width)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (a.dgamma_pre != nullptr) pre[col[k] + j] = sum_pre[k * V + j];
                if (a.dgamma_post != nullptr) post[col[k] + j] = sum_post[k * V + j];
            }
    if constexpr (CL) cluster_barrier();   // peers may still read this CTA's sums
}

// Joins the programs' column sums, in program order: blockIdx.y 0 and 1 the
// gamma gradients, the others the gate rows that more than one program
// holds.  A CTA sums COLS columns over RUNS contiguous runs of programs,
// joined in order, with a thread for V columns of a run: four where the width
// allows (4096 x 8192 FP32, sums not in cache: 8.5 us, 15 with a thread a
// column).  Rows of up to kNarrow columns have few columns and many programs:
// 8 columns and 128 runs to a CTA.  per_gate_units:
// programs of a gate row where programs keep to one, else 0 (contiguous
// ranges of rows).
template <int V>
struct Columns {
    float v[V];
};
template <int V>
__device__ __forceinline__ Columns<V> load_columns(const float *p) {
    Columns<V> r;
    if constexpr (V == 4) {
        const float4 q = *reinterpret_cast<const float4 *>(p);
        r = {{q.x, q.y, q.z, q.w}};
    } else {
        r.v[0] = *p;
    }
    return r;
}

template <int V, int COLS, int RUNS>
__global__ void __launch_bounds__(COLS / V *RUNS)
    block_norm_join_kernel(const BlockArgs a, long long units, long long gates,
                           int per_gate_units) {
    constexpr int LANES = COLS / V;
    __shared__ Columns<V> run_sum[RUNS][LANES];
    const int c = threadIdx.x % LANES, run = threadIdx.x / LANES;
    const int col = blockIdx.x * COLS + c * V;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the sums are written
    // sum of slot `slot0` of unit u0 and slot `slot` of the units after it
    auto join = [&](long long u0, long long u1, int slot0, int slot) {
        const long long n = u1 - u0 + 1;
        Columns<V> t = {};
        if (col < a.width) {
            const float *p = a.ws + (u0 * SLOTS + slot) * a.width + col;
            const long long step = static_cast<long long>(SLOTS) * a.width;
            int u = static_cast<int>(n * run / RUNS);
            const int to = static_cast<int>(n * (run + 1) / RUNS);
            if (u == 0 && to > 0) {
                t = load_columns<V>(p + static_cast<long long>(slot0 - slot) * a.width);
                u = 1;
            }
            for (; u < to; u += 8) {   // eight loads at once
                Columns<V> q[8] = {};
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (u + j < to) q[j] = load_columns<V>(p + (u + j) * step);
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) t.v[i] += q[j].v[i];
            }
        }
        run_sum[run][c] = t;
        __syncthreads();
        t = {};
        if (run == 0)
#pragma unroll
            for (int r = 0; r < RUNS; ++r)
#pragma unroll
                for (int i = 0; i < V; ++i) t.v[i] += run_sum[r][c].v[i];
        __syncthreads();
        return t;   // (run 0's)
    };
    if (blockIdx.y < 2) {
        float *to = blockIdx.y == 0 ? a.dgamma_pre : a.dgamma_post;
        const int slot = blockIdx.y == 0 ? SLOT_PRE : SLOT_POST;
        if (to == nullptr) return;
        const Columns<V> t = join(0, units - 1, slot, slot);
        if (run == 0 && col < a.width)
#pragma unroll
            for (int i = 0; i < V; ++i) to[col + i] = t.v[i];
        return;
    }
    for (long long g = blockIdx.y - 2; g < gates; g += gridDim.y - 2) {
        long long u0 = g * per_gate_units, u1 = u0 + per_gate_units - 1;
        int slot0 = SLOT_FIRST;
        if (per_gate_units == 0) {
            const long long end = (g + 1) * a.per_gate < a.rows ? (g + 1) * a.per_gate : a.rows;
            u0 = unit_of_row(g * a.per_gate, a.rows, units);
            u1 = unit_of_row(end - 1, a.rows, units);
            if (u0 == u1) continue;   // written by its program
            // the gate row is its first program's first, or its last, and
            // the first of every other program
            if (a.rows * u0 / units < g * a.per_gate) slot0 = SLOT_LAST;
        }
        const Columns<V> t = join(u0, u1, slot0, SLOT_FIRST);
        if (run == 0 && col < a.width)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float p = a.gamma_post != nullptr ? a.gamma_post[col + i] : 1.0f;
                a.dgate[g * a.width + col + i] = p * t.v[i];
            }
    }
}

// The ring kernel's layout of a row of `width` columns, or cluster 0 where
// it does not take the row.  A slot holds the four inputs' parts of a row:
// at most 64 KiB, so that three fit an SM.  Two vectors a thread: 16 columns
// of two-byte rows, 8 of FP32.
constexpr int kRingVecs = 2;

template <class T, bool SHIFT>
RingPlan ring_plan(int width) {
    constexpr int N = Vec<T>::N, K = kRingVecs;
    RingPlan p = {};
    // vectors that hold a row, wherever it starts
    const int vecs = (width + (SHIFT ? N - 1 : 0) + N - 1) / N;
    // (CTAs of 512 threads, one to an SM, before clusters: 8192 x 8192 BF16
    // took 177 us in clusters of two, two CTAs to an SM, and 149 us so; 4096 x
    // 16384 283 us in clusters of four and 183 us so)
    int c = 1;
    while (c <= 8 && (vecs + c - 1) / c > 512 * K) c *= 2;
    // But a single CTA of 288 or 320 threads leaves the registers for a second
    // one unused (13000 x 5120 BF16: 185 us, 174 us as a cluster of two of 160
    // threads, three to an SM), and four CTAs of one to an SM take longer than
    // eight smaller ones (2048 x 32768 BF16: 348 us and 291 us), except where
    // the masks of shifted rows come twice as often (2000 x 20001: 239 us and
    // 260 us).
    if (N == 8 && c == 1 && vecs > 256 * K && vecs <= 320 * K) c = 2;
    if (c == 4 && !SHIFT) c = 8;
    if (c > 8) return p;
    p.cluster = c;
    p.workers = ((vecs + c - 1) / c + 32 * K - 1) / (32 * K) * 32;
    p.pitch = (c == 1 ? vecs : p.workers * K) * 16;
    // as many CTAs to an SM as registers allow, the ring cut to fit
    int per_sm = 65536 / (p.workers * 128);
    if (N == 4 && (p.workers == 288 || p.workers == 320)) per_sm = 2;   // (up to 92 registers)
    per_sm = per_sm < 1 ? 1 : per_sm > 16 ? 16 : per_sm;
    p.slots = ((224 << 10) / per_sm - (3 << 10)) / (4 * p.pitch);
    p.slots = p.slots > kRingMost ? kRingMost : p.slots;
    p.smem = p.slots * 4 * p.pitch;
    p.classes = 1;
    while (SHIFT && static_cast<long long>(p.classes) * width % N != 0) p.classes *= 2;
    return p;
}

template <class Kernel, class Plan>
cudaError_t launch_programs(Kernel kernel, const BlockArgs &a, const Plan &plan, long long units,
                            int threads, int cluster, int smem, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(units * cluster));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    if (cluster > 1) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = cluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, kernel, a, plan);
}

// What the join needs to know of the programs.
struct Programs {
    long long units;
    int per_gate;   // programs of a gate row, 0: contiguous ranges of rows
};

template <class T, bool SHIFT, bool CL, int MAXT, int MINB, bool WITHHELD = false>
cudaError_t launch_ring(const BlockArgs &a, RingPlan p, cudaStream_t stream, Programs *out) {
    static OccupancyCache cache;
    const auto kernel = block_norm_ring_kernel<T, kRingVecs, SHIFT, CL, MAXT, MINB, WITHHELD>;
    int per_sm = 0;
    const cudaError_t err = occupancy(kernel, cache, p.workers, p.smem, &per_sm);
    if (err != cudaSuccess) return err;
    const long long room = static_cast<long long>(sm_count_of_device()) * per_sm / p.cluster;
    if (p.classes == 1) {
        *out = {units_of(a, room), 0};
    } else {
        const long long gates = (a.rows + a.per_gate - 1) / a.per_gate;
        long long parts = units_of(a, room) / (gates * p.classes);
        p.parts = parts < 1 ? 1 : static_cast<int>(parts);
        *out = {gates * p.classes * p.parts, p.classes * p.parts};
    }
    return launch_programs(kernel, a, p, out->units, p.workers, p.cluster, p.smem, stream);
}

template <class T, bool SHIFT>
cudaError_t launch_ring_typed(const BlockArgs &a, const RingPlan &p, cudaStream_t stream,
                              Programs *out) {
    const bool one = p.cluster == 1;
    if (a.withheld) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value && !SHIFT)
            if (p.workers <= 256)
                return one ? launch_ring<T, false, false, 256, 2, true>(a, p, stream, out)
                           : launch_ring<T, false, true, 256, 2, true>(a, p, stream, out);
        return cudaErrorNotSupported;
    }
    if (p.workers <= 256)
        return one ? launch_ring<T, SHIFT, false, 256, 2>(a, p, stream, out)
                   : launch_ring<T, SHIFT, true, 256, 2>(a, p, stream, out);
    // FP32 rows keep half as many columns in a thread's registers (2-byte ones
    // spilled here: 13000 x 5120 BF16 238 us)
    if constexpr (sizeof(T) == 4)
        if (p.workers <= 320)
            return one ? launch_ring<T, SHIFT, false, 320, 2>(a, p, stream, out)
                       : launch_ring<T, SHIFT, true, 320, 2>(a, p, stream, out);
    return one ? launch_ring<T, SHIFT, false, 512, 1>(a, p, stream, out)
               : launch_ring<T, SHIFT, true, 512, 1>(a, p, stream, out);
}

template <class T, int V, int E, bool CL>
cudaError_t launch_registers(const BlockArgs &a, cudaStream_t stream, Programs *out) {
    const int cluster = CL ? 8 : 1;
    const int threads = (a.width + cluster * E * 32 - 1) / (cluster * E * 32) * 32;
    static OccupancyCache cache;
    int per_sm = 0;
    const cudaError_t err =
        occupancy(block_norm_backward_kernel<T, V, E / V, CL>, cache, threads, 0, &per_sm);
    if (err != cudaSuccess) return err;
    const long long room = static_cast<long long>(sm_count_of_device()) * per_sm / cluster;
    *out = {units_of(a, room), 0};
    return launch_programs(block_norm_backward_kernel<T, V, E / V, CL>, a, cluster, out->units,
                           threads, cluster, 0, stream);
}

template <class T>
cudaError_t launch_typed(const BlockArgs &a, BlockAccess access, cudaStream_t stream,
                         Programs *out) {
    constexpr int N = Vec<T>::N;
    if (a.withheld && access != ACCESS_VECTORS) return cudaErrorNotSupported;
    if (access == ACCESS_VECTORS) {
        const RingPlan p = ring_plan<T, false>(a.width);
        if (a.withheld && p.cluster == 0) return cudaErrorNotSupported;
        if (p.cluster > 0) return launch_ring_typed<T, false>(a, p, stream, out);
        return launch_registers<T, N, 32, true>(a, stream, out);
    }
    if (access == ACCESS_SHIFTED) {
        const RingPlan p = ring_plan<T, true>(a.width);
        const long long gates = (a.rows + a.per_gate - 1) / a.per_gate;
        if (p.cluster > 0 && (p.classes == 1 || gates * p.classes <= class_units(a.width)))
            return launch_ring_typed<T, true>(a, p, stream, out);
    }
    if (a.width <= 512 * 16) return launch_registers<T, 1, 16, false>(a, stream, out);
    return launch_registers<T, 1, 32, true>(a, stream, out);
}

// Launched while the programs run (it waits for their end itself).
template <int V, int COLS, int RUNS>
cudaError_t launch_join(const BlockArgs &a, const Programs &programs, long long gates,
                        cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.width + COLS - 1) / COLS,
                       2 + static_cast<unsigned>(gates < 1024 ? gates : 1024));
    cfg.blockDim = dim3(COLS / V * RUNS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, block_norm_join_kernel<V, COLS, RUNS>, a, programs.units, gates,
                              programs.per_gate);
}

}  // namespace

size_t block_norm_backward_workspace(long long rows, int width, long long gates) {
    long long units = rows < most_units(width) ? rows : most_units(width);
    if (width % 8 != 0) {   // up to 8 row classes (of 2-byte elements) in each gate row
        const long long classes = 8 * gates < class_units(width) ? 8 * gates : class_units(width);
        if (classes > units) units = classes;
    }
    return static_cast<size_t>(units) * SLOTS * static_cast<size_t>(width) * sizeof(float);
}

cudaError_t launch_block_norm_backward(int elem, BlockAccess access, const BlockArgs &args,
                                       cudaStream_t stream) {
    BlockArgs a = args;
    cudaError_t err = cudaSuccess;
    a.status = status_address(&err);
    if (a.status == nullptr) return err;
    Programs programs = {};
    switch (elem) {
        case ELEM_F32: err = launch_typed<float>(a, access, stream, &programs); break;
        case ELEM_BF16: err = launch_typed<__nv_bfloat16>(a, access, stream, &programs); break;
        case ELEM_F16: err = launch_typed<__half>(a, access, stream, &programs); break;
        default: return cudaErrorInvalidValue;
    }
    if (err != cudaSuccess) return err;
    const long long gates = a.dgate != nullptr ? (a.rows + a.per_gate - 1) / a.per_gate : 0;
    if (a.dgamma_pre == nullptr && a.dgamma_post == nullptr && gates == 0) return cudaSuccess;
    const bool fours = a.width % 4 == 0;   // (the workspace is on 16 bytes)
    if (a.width <= kNarrow)
        return fours ? launch_join<4, 8, 128>(a, programs, gates, stream)
                     : launch_join<1, 8, 128>(a, programs, gates, stream);
    return fours ? launch_join<4, 32, 32>(a, programs, gates, stream)
                 : launch_join<1, 32, 32>(a, programs, gates, stream);
}

}  // namespace tile
