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

TILE_DEVICE_STATUS(block_norm)

namespace tile {
namespace {

template <class T, int V, int K, bool CL>
__global__ void __launch_bounds__(512) block_norm_kernel(const BlockArgs a, int warps, int cluster) {
    using A = Access<T, V>;
    constexpr int G = V == 1 ? 2 : V, GK = G / V;   // columns handled together, in GK groups
    constexpr int E = K * V;
    static_assert(K % GK == 0, "whole pairs");
    __shared__ ReduceMem<1> mem;
    const int W = warps * 32;
    const int programs = CL ? 1 : blockDim.x / W;
    const int rank = CL ? static_cast<int>(cluster_rank()) : 0;
    const int worker = CL ? threadIdx.x : threadIdx.x % W;
    const long long row = CL ? blockIdx.x / cluster
                             : static_cast<long long>(blockIdx.x) * programs + threadIdx.x / W;
    if (row >= a.rows) return;   // whole warps: programs share a CTA only at one warp each
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
    float v[E];
    F2 sq = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float p[V];
        A::widen(xr[k], p);
#pragma unroll
        for (int j = 0; j < V; ++j) v[k * V + j] = p[j];
    }
    int turn = 0;
    float r1 = 1.0f;
    if (a.post) {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) sq = fma2(pair(v, i), pair(v, i), sq);
        float s[1] = {sq.x + sq.y};
        row_sum<1, CL>(s, mem, turn, warps, cluster);
        r1 = inv_sqrt<T>(fmaf(s[0], inv_n, a.eps));
    }
    sq = F2{0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < K; k += GK) {
        float p[G], q[G], g[G], h[G];
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
            const int at = k * V / 2 + i;
            const F2 n = mul2(pair(v, at), both(r1));
            const F2 t = fma2(mul2(pair(p, i), pair(q, i)), n, mul2(pair(g, i), both(a.scale)));
            sq = fma2(t, t, sq);
            put(v, at, t);
            put(h, i, t);
        }
#pragma unroll
        for (int u = 0; u < GK; ++u)
            if (first + (k + u) * step < a.width) {
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = h[u * V + j];
                A::store(hid + (k + u) * step, o);
            }
    }
    if (a.pre) {
        float s[1] = {sq.x + sq.y};
        row_sum<1, CL>(s, mem, turn, warps, cluster);
        const float r2 = inv_sqrt<T>(fmaf(s[0], inv_n, a.eps));
#pragma unroll
        for (int i = 0; i < E / 2; ++i) put(v, i, mul2(pair(v, i), both(r2)));
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int col = first + k * step;
            if (col >= a.width) continue;
            float p[V];
            load_params<V>(a.gamma_pre, col, p);
            if constexpr (V == 1) {
                p[0] *= v[k];
            } else {
#pragma unroll
                for (int i = 0; i < V / 2; ++i)
                    put(p, i, mul2(pair(v, k * V / 2 + i), pair(p, i)));
            }
            A::store(out + k * step, p);
        }
    }
    if constexpr (CL) cluster_barrier();   // peers may still read this CTA's sums
}

template <class T, int V, int E, bool CL>
cudaError_t launch_kernel(const BlockArgs &a, int cluster, cudaStream_t stream) {
    const int threads = (a.width + cluster * E * 32 - 1) / (cluster * E * 32) * 32;
    // rows of one warp share a CTA: 8 of them
    const int programs = threads == 32 && !CL ? 8 : 1;
    const long long grid = (a.rows + programs - 1) / programs * cluster;
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads * programs);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    if (CL) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = cluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, block_norm_kernel<T, V, E / V, CL>, a, threads / 32, cluster);
}

// One CTA a row up to 512 threads, then a cluster of up to 8, then (FP32 and
// single elements above 65536 columns) 32 columns a thread.
template <class T, int V>
cudaError_t launch_typed(const BlockArgs &a, cudaStream_t stream) {
    constexpr int E = V == 8 ? 32 : 16;
    if (a.width <= 512 * E) return launch_kernel<T, V, E, false>(a, 1, stream);
    for (int c = 2; c <= 8; c *= 2)
        if (a.width <= 512 * E * c) return launch_kernel<T, V, E, true>(a, c, stream);
    return launch_kernel<T, V, 32, true>(a, 8, stream);
}

}  // namespace

cudaError_t launch_block_norm(int elem, bool vec, const BlockArgs &args, cudaStream_t stream) {
    BlockArgs a = args;
    cudaError_t err = cudaSuccess;
    a.status = status_address(&err);
    if (a.status == nullptr) return err;
    switch (elem) {
        case ELEM_F32:
            return vec ? launch_typed<float, 4>(a, stream) : launch_typed<float, 1>(a, stream);
        case ELEM_BF16:
            return vec ? launch_typed<__nv_bfloat16, 8>(a, stream)
                       : launch_typed<__nv_bfloat16, 1>(a, stream);
        case ELEM_F16:
            return vec ? launch_typed<__half, 8>(a, stream) : launch_typed<__half, 1>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace tile
