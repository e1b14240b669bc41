// Block norm, forward: h = a r + gate * post(b), y = pre(h), both norms
// RMSNorms (v / sqrt(mean v^2 + eps) * gamma), each optional.
//
// Bound by DRAM: x and the residual are read once, h and y written once.  A
// program walks over a contiguous range of rows with gate * gamma_post and
// gamma_pre of its columns in registers (read for every row they would cost
// 12 bytes of L2 traffic per element against the 8 of two-byte rows), and
// loads the next row before it works on the present one.  The mean square of
// h is taken from the FP32 h that this row's threads hold, not from a
// combination of sums over x and r, which cancels where the block undoes the
// residual; y is computed from that h and rounded once.
#include "block_norm.cuh"
#include "device_status.h"

TILE_DEVICE_STATUS(block_norm)

namespace tile {
namespace {

template <class T, int V, int K, bool CL>
__global__ void __launch_bounds__(512) block_norm_kernel(const BlockArgs a, int cluster) {
    using A = Access<T, V>;
    constexpr int E = K * V;
    __shared__ ReduceMem<1> mem;
    const int W = blockDim.x;
    const int warps = W >> 5;
    const int rank = CL ? static_cast<int>(cluster_rank()) : 0;
    const long long units = gridDim.x / (CL ? cluster : 1);
    const long long unit = blockIdx.x / (CL ? cluster : 1);
    const long long begin = a.rows * unit / units, end = a.rows * (unit + 1) / units;
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    T *hid = static_cast<T *>(a.hidden_out), *out = static_cast<T *>(a.out);
    const float inv_n = 1.0f / static_cast<float>(a.width);

    int col[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
        col[k] = ((k * (CL ? cluster : 1) + rank) * W + static_cast<int>(threadIdx.x)) * V;

    typename A::Raw xr[K], rr[K];
    auto fetch = [&](long long row) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (col[k] < a.width) {
                xr[k] = A::load(x + row * a.width + col[k]);
                rr[k] = A::load(res + row * a.width + col[k]);
            }
    };
    if (begin < end) fetch(begin);

    float w[E], g2[E];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float p[V];
        if (col[k] < a.width) load_params<V>(a.gamma_pre, col[k], p);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            g2[k * V + j] = col[k] < a.width ? p[j] : 0.0f;
            w[k * V + j] = 0.0f;
        }
    }
    long long gate_end = begin;   // first row that needs the next gate row
    int turn = 0;
    for (long long row = begin; row < end; ++row) {
        if (row == gate_end) {
            const long long gate_row = row / a.per_gate;
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
        float v[E], r[E];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float p[V], q[V];
            if (col[k] < a.width) {
                A::widen(xr[k], p);
                A::widen(rr[k], q);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[k * V + j] = col[k] < a.width ? p[j] : 0.0f;
                r[k * V + j] = col[k] < a.width ? q[j] : 0.0f;
            }
        }
        if (row + 1 < end) fetch(row + 1);
        float r1 = 1.0f;
        if (a.post) {
            float s[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < E; ++i) s[0] = fmaf(v[i], v[i], s[0]);
            row_sum<1, CL>(s, mem, turn, warps, cluster);
            r1 = 1.0f / sqrtf(fmaf(s[0], inv_n, a.eps));
        }
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = fmaf(a.scale, r[i], w[i] * (v[i] * r1));
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (col[k] < a.width) {
                float p[V];
#pragma unroll
                for (int j = 0; j < V; ++j) p[j] = v[k * V + j];
                A::store(hid + row * a.width + col[k], p);
            }
        if (a.pre) {
            float s[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < E; ++i) s[0] = fmaf(v[i], v[i], s[0]);
            row_sum<1, CL>(s, mem, turn, warps, cluster);
            const float r2 = 1.0f / sqrtf(fmaf(s[0], inv_n, a.eps));
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (col[k] < a.width) {
                    float p[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) p[j] = (v[k * V + j] * r2) * g2[k * V + j];
                    A::store(out + row * a.width + col[k], p);
                }
        }
    }
    if constexpr (CL) cluster_barrier();   // peers may still read this CTA's sums
}

template <class T, int V, int K, bool CL>
cudaError_t launch_kernel(const BlockArgs &a, const BlockPlan &p, cudaStream_t stream) {
    static std::atomic<int> per_sm[kMaxDevices][17];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    int occ = per_sm[dev][p.threads / 32].load(std::memory_order_relaxed);
    if (occ == 0) {
        err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, block_norm_kernel<T, V, K, CL>,
                                                            p.threads, 0);
        if (err != cudaSuccess) return err;
        if (occ < 1) occ = 1;
        per_sm[dev][p.threads / 32].store(occ, std::memory_order_relaxed);
    }
    long long units = static_cast<long long>(sm_count_of_device()) * occ / p.cluster;
    if (units > a.rows) units = a.rows;
    if (units < 1) units = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(units * p.cluster));
    cfg.blockDim = dim3(p.threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    if (CL) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = p.cluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, block_norm_kernel<T, V, K, CL>, a, p.cluster);
}

template <class T, int V>
cudaError_t launch_typed(const BlockArgs &a, cudaStream_t stream) {
    const BlockPlan p = block_plan(a.width);
    if (p.elems == 8) return launch_kernel<T, V, 8 / V, false>(a, p, stream);
    if (p.elems == 32) return launch_kernel<T, V, 32 / V, true>(a, p, stream);
    return p.cluster > 1 ? launch_kernel<T, V, 16 / V, true>(a, p, stream)
                         : launch_kernel<T, V, 16 / V, false>(a, p, stream);
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
