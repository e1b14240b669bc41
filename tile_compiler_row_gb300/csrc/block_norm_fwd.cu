// Block norm, forward: h = a r + gate * post(b), y = pre(h), both norms
// RMSNorms (v / sqrt(mean v^2 + eps) * gamma), each optional.
//
// Bound by DRAM: x and the residual are read once, h and y written once.
// One program a row, and enough of them on an SM that one row's reductions
// run under the others' loads; 32 two-byte or 16 FP32 columns a thread, as
// the two reductions cost each thread some 150 instructions whatever it
// holds.  gate, gamma_post and gamma_pre (12 bytes per element, against 8 of
// two-byte rows) come from L1, which the programs of an SM share.  The mean
// square of h is taken from the FP32 h that this row's threads hold, not
// from a combination of sums over x and r, which cancels where the block
// undoes the residual; y is computed from that h and rounded once.
#include "block_norm.cuh"
#include "device_status.h"

namespace tile {
namespace {

// A row is `workers` threads of each of `cluster` CTAs: whole warps, or a
// power of two of neighbours of a warp, which then holds several rows.
template <class T, int V, int K, bool CL, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB)
    block_norm_kernel(const BlockArgs a, int workers, int cluster) {
    using A = Access<T, V>;
    constexpr int G = V == 1 ? 2 : V, GK = G / V;   // columns handled together, in GK groups
    constexpr int E = K * V;
    static_assert(K % GK == 0, "whole pairs");
    __shared__ ReduceMem<1> mem;
    const int W = workers, warps = (W + 31) / 32, lanes = W < 32 ? W : 32;
    const int programs = CL ? 1 : blockDim.x / W;
    const int rank = CL ? static_cast<int>(cluster_rank()) : 0;
    const int worker = CL ? threadIdx.x : threadIdx.x % W;
    const long long row0 = CL ? blockIdx.x / cluster
                              : static_cast<long long>(blockIdx.x) * programs + threadIdx.x / W;
    // threads behind the last row do it once more, without stores
    const bool live = row0 < a.rows;
    const long long row = live ? row0 : a.rows - 1;
    const float inv_n = 1.0f / static_cast<float>(a.width);
    const int step = (CL ? cluster : 1) * W * V, first = (rank * W + worker) * V;
    const T *x = static_cast<const T *>(a.x) + row * a.width + first;
    const T *res = static_cast<const T *>(a.residual) + row * a.width + first;
    T *hid = static_cast<T *>(a.hidden_out) + row * a.width + first;
    T *out = static_cast<T *>(a.out) + row * a.width + first;
    const float *gate = a.gate != nullptr ? a.gate + row / a.per_gate * a.width : nullptr;

    typename A::Raw xr[K], rr[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        xr[k] = rr[k] = typename A::Raw{};
        if (first + k * step < a.width) {
            xr[k] = A::load(x + k * step);
            rr[k] = A::load(res + k * step);
        }
    }
    F2 v[E / 2], sq = 0;
#pragma unroll
    for (int k = 0; k < K; k += GK) {
        float p[G];
#pragma unroll
        for (int u = 0; u < GK; ++u) {
            float q[V];
            A::widen(xr[k + u], q);
#pragma unroll
            for (int j = 0; j < V; ++j) p[u * V + j] = q[j];
        }
#pragma unroll
        for (int i = 0; i < G / 2; ++i) v[k * V / 2 + i] = pack(p[2 * i], p[2 * i + 1]);
    }
    int turn = 0;
    float r1 = 1.0f;
    if (a.post) {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) sq = fma2(v[i], v[i], sq);
        float s[1] = {total(sq)};
        row_sum<1, CL>(s, mem, turn, warps, cluster, lanes);
        r1 = inv_sqrt<T>(fmaf(s[0], inv_n, a.eps));
    }
    sq = 0;
    const F2 r1s = both(r1), scale = both(a.scale);
#pragma unroll
    for (int k = 0; k < K; k += GK) {
        float p[G], q[G], g[G];
#pragma unroll
        for (int u = 0; u < GK; ++u) {
            float pu[V], qu[V], gu[V];
            A::widen(rr[k + u], gu);
            const int col = first + (k + u) * step;
            const bool in = col < a.width;
            load_params<V>(in ? a.gamma_post : nullptr, col, pu);
            load_params<V>(in ? gate : nullptr, col, qu);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                p[u * V + j] = pu[j];
                q[u * V + j] = qu[j];
                g[u * V + j] = gu[j];
            }
        }
#pragma unroll
        for (int i = 0; i < G / 2; ++i) {
            F2 &at = v[k * V / 2 + i];
            const F2 w = mul2(pack(p[2 * i], p[2 * i + 1]), pack(q[2 * i], q[2 * i + 1]));
            at = fma2(w, mul2(at, r1s), mul2(pack(g[2 * i], g[2 * i + 1]), scale));
            sq = fma2(at, at, sq);
            unpack(at, g[2 * i], g[2 * i + 1]);
        }
#pragma unroll
        for (int u = 0; u < GK; ++u)
            if (live && first + (k + u) * step < a.width) {
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = g[u * V + j];
                A::store(hid + (k + u) * step, o);
            }
    }
    if (a.pre) {
        float s[1] = {total(sq)};
        row_sum<1, CL>(s, mem, turn, warps, cluster, lanes);
        const F2 r2 = both(inv_sqrt<T>(fmaf(s[0], inv_n, a.eps)));
#pragma unroll
        for (int k = 0; k < K; k += GK) {
            float p[G];
#pragma unroll
            for (int u = 0; u < GK; ++u) {
                float q[V];
                const int col = first + (k + u) * step;
                load_params<V>(col < a.width ? a.gamma_pre : nullptr, col, q);
#pragma unroll
                for (int j = 0; j < V; ++j) p[u * V + j] = q[j];
            }
#pragma unroll
            for (int i = 0; i < G / 2; ++i)
                unpack(mul2(mul2(v[k * V / 2 + i], r2), pack(p[2 * i], p[2 * i + 1])), p[2 * i],
                       p[2 * i + 1]);
#pragma unroll
            for (int u = 0; u < GK; ++u)
                if (live && first + (k + u) * step < a.width) {
                    float o[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) o[j] = p[u * V + j];
                    A::store(out + (k + u) * step, o);
                }
        }
    }
    if constexpr (CL) cluster_barrier();   // peers may still read this CTA's sums
}

// Two-byte rows that are not whole vectors: a program takes rows that start at the
// same offset into a 16-byte block (every second, fourth or eighth), so each
// thread reads and writes the same aligned vectors of them and owns the same
// columns, whose parameters it keeps in registers (from L1 they would be
// single-element loads); the vectors at a row's ends are masked.  The next
// row is loaded before the present one is worked on.  Single-element
// accesses (the kernel above with V = 1) ran 16384 x 4097 BF16 in 291 us.
template <class T, int K, bool CL, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB)
    block_norm_shift_kernel(const BlockArgs a, const RingPlan plan) {
    using X = Vec<T>;
    constexpr int N = X::N, P = X::P;
    __shared__ ReduceMem<1> mem;
    const int W = plan.workers, warps = (W + 31) / 32, lanes = W < 32 ? W : 32;
    const int C = CL ? plan.cluster : 1, programs = CL ? 1 : blockDim.x / W;
    const int rank = CL ? static_cast<int>(cluster_rank()) : 0;
    const int width = a.width, tid = CL ? threadIdx.x : threadIdx.x % W;
    const RowWalk walk = row_walk(a.rows, a.rows, plan,
                                  CL ? blockIdx.x / C
                                     : static_cast<long long>(blockIdx.x) * programs + threadIdx.x / W,
                                  gridDim.x / C * static_cast<long long>(programs));
    // programs of one warp go round together, those without a row left idly
    long long rounds = walk.count;
    if (lanes < 32)
        for (int d = 16; d > 0; d >>= 1) {
            const long long o = __shfl_xor_sync(0xffffffffu, rounds, d);
            rounds = o > rounds ? o : rounds;
        }
    const int shift = static_cast<int>((walk.first * width) & (N - 1));
    // masks of this program's rows (programs of at most 32 threads share a CTA
    // of 256, so up to 256 of them)
    __shared__ EdgeMasks all_masks[CL ? 1 : 256];
    EdgeMasks &masks = all_masks[CL ? 0 : threadIdx.x / W];
    if (tid == 0) edge_masks<T>(masks, shift, width);
    __syncthreads();
    const int vecs = (width + shift + N - 1) / N;
    auto vec = [&](int k) { return rank * W * K + k * W + tid; };
    auto first = [&](int k) { return vec(k) * N - shift; };   // column of vector k
    const float inv_n = 1.0f / static_cast<float>(width);
    const long long size = a.rows * width;
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    auto load = [&](const T *p, long long row, int k) {
        const long long at = row * width + first(k);
        if (at + N <= size) return __ldcs(reinterpret_cast<const uint4 *>(p + at));
        unsigned int w[4] = {};   // the matrix ends in this block
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (at + j < size) {
                if constexpr (sizeof(T) == 4)
                    w[j] = reinterpret_cast<const unsigned int *>(p + at)[j];
                else
                    w[j / 2] |= static_cast<unsigned int>(
                                    reinterpret_cast<const unsigned short *>(p + at)[j])
                                << (16 * (j & 1));
            }
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    uint4 xr[K], rr[K];
    auto fetch = [&](long long row) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (vec(k) < vecs) {
                xr[k] = load(x, row, k);
                rr[k] = load(res, row, k);
            }
    };
    if (walk.count > 0) fetch(walk.first);
    F2 w[K * P], g2[K * P];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        F2 p[P];
        params_at<N>(a.gamma_pre, first(k), width, p);
#pragma unroll
        for (int i = 0; i < P; ++i) g2[k * P + i] = p[i];
    }
    long long gate_end = walk.first;
    int turn = 0;
    const F2 scale = both(a.scale);
    for (long long i_row = 0; i_row < rounds; ++i_row) {
        const long long row = walk.first + i_row * walk.step;
        const bool live = i_row < walk.count;
        if (live && row >= gate_end) {
            const long long gate_row = row / a.per_gate;
            gate_end = (gate_row + 1) * a.per_gate;
            const float *gate = a.gate != nullptr ? a.gate + gate_row * width : nullptr;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                F2 p[P], q[P];
                params_at<N>(a.gamma_post, first(k), width, p);
                params_at<N>(gate, first(k), width, q);
#pragma unroll
                for (int i = 0; i < P; ++i) w[k * P + i] = mul2(p[i], q[i]);
            }
        }
        F2 v[K * P], r[K * P], sq = 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            uint4 p = make_uint4(0, 0, 0, 0), q = p;
            if (live && vec(k) < vecs) {
                p = mask_vec(xr[k], edge_of(vec(k), vecs), masks);
                q = mask_vec(rr[k], edge_of(vec(k), vecs), masks);
            }
            F2 t[P], u[P];
            X::widen(p, t);
            X::widen(q, u);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                v[k * P + i] = t[i];
                r[k * P + i] = mul2(u[i], scale);
            }
        }
        if (i_row + 1 < walk.count) fetch(row + walk.step);
        float r1 = 1.0f;
        if (a.post) {
#pragma unroll
            for (int i = 0; i < K * P; ++i) sq = fma2(v[i], v[i], sq);
            float s[1] = {total(sq)};
            row_sum<1, CL>(s, mem, turn, warps, C, lanes);
            r1 = inv_sqrt<T>(fmaf(s[0], inv_n, a.eps));
        }
        const F2 r1s = both(r1);
        sq = 0;
#pragma unroll
        for (int i = 0; i < K * P; ++i) {
            v[i] = fma2(w[i], mul2(v[i], r1s), r[i]);
            sq = fma2(v[i], v[i], sq);
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (live && vec(k) < vecs) {
                F2 t[P];
#pragma unroll
                for (int i = 0; i < P; ++i) t[i] = v[k * P + i];
                store_vec_at<T>(static_cast<T *>(a.hidden_out) + row * width + first(k),
                                X::narrow(t), first(k), width);
            }
        if (a.pre) {
            float s[1] = {total(sq)};
            row_sum<1, CL>(s, mem, turn, warps, C, lanes);
            const F2 r2 = both(inv_sqrt<T>(fmaf(s[0], inv_n, a.eps)));
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (live && vec(k) < vecs) {
                    F2 t[P];
#pragma unroll
                    for (int i = 0; i < P; ++i)
                        t[i] = mul2(mul2(v[k * P + i], r2), g2[k * P + i]);
                    store_vec_at<T>(static_cast<T *>(a.out) + row * width + first(k), X::narrow(t),
                                    first(k), width);
                }
        }
    }
    if constexpr (CL) cluster_barrier();   // peers may still read this CTA's sums
}

// Launch of `grid` CTAs of `threads`, in clusters.
template <class Kernel, class... Args>
cudaError_t launch_grid(Kernel kernel, long long grid, int threads, int cluster,
                        cudaStream_t stream, Args... args) {
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    if (cluster > 1) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = cluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Threads of a row that is `groups` groups of columns, each thread taking at
// most `each`: a power of two up to a warp, then whole warps.
int threads_of(int groups, int each) {
    const int n = (groups + each - 1) / each;
    int w = 1;
    while (w < n && w < 32) w *= 2;
    return n <= 32 ? w : (n + 31) / 32 * 32;
}
// Threads of a CTA of programs of w threads: programs of at most a warp share
// one.
int cta_threads(int w) { return w <= 32 ? 256 : w; }

template <class T, bool CL, int MAXT, int MINB>
cudaError_t launch_shift(const BlockArgs &a, RingPlan p, cudaStream_t stream) {
    constexpr int N = Vec<T>::N, K = 2;
    const auto kernel = block_norm_shift_kernel<T, K, CL, MAXT, MINB>;
    const int threads = CL ? p.workers : cta_threads(p.workers);
    static OccupancyCache cache;
    int occ = 0;
    const cudaError_t err = occupancy(kernel, cache, threads, 0, &occ);
    if (err != cudaSuccess) return err;
    p.classes = 1;
    while (static_cast<long long>(p.classes) * a.width % N != 0) p.classes *= 2;
    const int programs = threads / p.workers;   // of a CTA
    const long long room =
        static_cast<long long>(sm_count_of_device()) * occ / p.cluster * programs;
    // parts of a class: as many as there is room for, but not more than rows
    long long parts = room / p.classes;
    const long long most = (a.rows + p.classes - 1) / p.classes;
    parts = parts > most ? most : parts < 1 ? 1 : parts;
    while (parts * p.classes % programs != 0) ++parts;   // whole CTAs
    p.parts = static_cast<int>(parts);
    return launch_grid(kernel, parts * p.classes / programs * p.cluster, threads, p.cluster, stream,
                       a, p);
}

template <class T, int V, int E, bool CL, int MAXT, int MINB>
cudaError_t launch_kernel(const BlockArgs &a, int cluster, cudaStream_t stream) {
    const int groups = (a.width + V - 1) / V;
    const int w = CL ? (groups + cluster * (E / V) * 32 - 1) / (cluster * (E / V) * 32) * 32
                     : threads_of(groups, E / V);
    const int threads = CL ? w : cta_threads(w), programs = threads / w;
    return launch_grid(block_norm_kernel<T, V, E / V, CL, MAXT, MINB>,
                       (a.rows + programs - 1) / programs * cluster, threads, cluster, stream, a, w,
                       cluster);
}

// 32 two-byte or 16 FP32 columns a thread, up to 512 threads a row, then a
// cluster of up to 8 CTAs, then 32 columns of either.  Two-byte rows of whole
// vectors take CTAs that leave room for three on an SM where there are 128 to
// 256 threads (80 registers, nothing spilled: 8192 x 8192 BF16 92 us, 105 us
// with two) and in clusters of them (2048 x 32768 153 us, 194 us with CTAs of
// 512 threads), but one CTA of 512 where that is full (4096 x 16384 138 us,
// 144 us as a cluster of two).
template <class T, int V>
cudaError_t launch_rows(const BlockArgs &a, cudaStream_t stream) {
    constexpr int E = V == 8 ? 32 : 16;
    constexpr int MINB = V == 8 ? 1 : 2;   // 64 registers for 16 columns
    // 96 for 32 up to 128 threads and where three CTAs do not fit (with 128
    // registers 16384 x 4096 BF16 took 107 us instead of 88)
    if constexpr (V == 8) {
        if (a.width > 128 * E && a.width <= 256 * E)
            return launch_kernel<T, V, E, false, 256, 3>(a, 1, stream);
        if (a.width <= 320 * E) return launch_kernel<T, V, E, false, 320, 2>(a, 1, stream);
        for (int c = 2; c <= 8; c *= 2)
            if (a.width <= 256 * E * c && (a.width <= 448 * E || a.width > 512 * E))
                return launch_kernel<T, V, E, true, 256, 3>(a, c, stream);
    }
    if (a.width <= 512 * E) return launch_kernel<T, V, E, false, 512, MINB>(a, 1, stream);
    for (int c = 2; c <= 8; c *= 2)
        if (a.width <= 512 * E * c) return launch_kernel<T, V, E, true, 512, MINB>(a, c, stream);
    return launch_kernel<T, V, 32, true, 512, 1>(a, 8, stream);
}

template <class T>
cudaError_t launch_typed(const BlockArgs &a, BlockAccess access, cudaStream_t stream) {
    constexpr int N = Vec<T>::N;
    if (access == ACCESS_VECTORS) return launch_rows<T, N>(a, stream);
    // (FP32 rows off the grid go by single elements: a warp's 128 bytes are
    // one line or two, as with vectors; 5000 x 1537 took 27 us, by shifted
    // vectors 41 us)
    if constexpr (N == 8) {
        const int vecs = (a.width + N - 1 + N - 1) / N;   // wherever a row starts
        if (access == ACCESS_SHIFTED && vecs <= 8 * 512 * 2) {
            RingPlan p = {};
            p.cluster = 1;
            p.workers = threads_of(vecs, 2);
            if (p.workers <= 256) return launch_shift<T, false, 256, 2>(a, p, stream);
            if (p.workers <= 320) return launch_shift<T, false, 320, 2>(a, p, stream);
            if (p.workers <= 512) return launch_shift<T, false, 512, 1>(a, p, stream);
            while (vecs > 2 * 512 * p.cluster) p.cluster *= 2;
            p.workers = ((vecs + p.cluster - 1) / p.cluster + 63) / 64 * 32;
            return launch_shift<T, true, 512, 1>(a, p, stream);
        }
    }
    return launch_rows<T, 1>(a, stream);
}

}  // namespace

cudaError_t launch_block_norm(int elem, BlockAccess access, const BlockArgs &a,
                              cudaStream_t stream) {
    switch (elem) {
        case ELEM_F32: return launch_typed<float>(a, access, stream);
        case ELEM_BF16: return launch_typed<__nv_bfloat16>(a, access, stream);
        case ELEM_F16: return launch_typed<__half>(a, access, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace tile
