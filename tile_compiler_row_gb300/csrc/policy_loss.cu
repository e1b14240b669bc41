// Clipped policy loss with a KL term, and its gradient.  For every token that
// counts, with x = old_nll - nll, r = exp(x) and q = nll - ref_nll,
//
//   l = -min(r A, clip(r, 1 - low, 1 + high) A) + beta (exp(q) - q - 1)
//   dl/dnll = (r A where it is the smaller one, else 0) + beta (exp(q) - 1)
//
// averaged over all tokens, or over sequences of means over their tokens.
//
// 24 bytes a token forward and 28 backward at most: bound by latency up to some
// 10^5 tokens, and by how many loads are on their way beyond.  A tile is 512 rows,
// two to a thread, all its loads issued before the sequences are looked for; the
// tiles' sums are joined by a second launch that comes up meanwhile, or, of up to
// 8 tiles, by the first CTA of their cluster.  (Device times in a graph: 1048576
// tokens, 512 sequences: 9.8 us forward, 7.4 backward, where the bytes are 4 us; 8191
// tokens: 5.1 and 3.1.  With expm1f alone for the KL term, tiles of 512, 1024 (four
// rows to a thread) and 256 rows: 9.4, 10.4 and 11.2; 7.3, 8.9 and 8.3; 4.8, 5.9 and
// 4.8; 3.0, 4.3 and 2.6.  A join of 1024 threads took 0.5 to 0.8 us more than one
// of 512.)
//
// One CTA joins: it looks at each sequence's offsets, and for means over sequences
// adds up each one's tiles.  That grows with the sequences: 16384 of 1048576 tokens
// take 19 us, and 58 for their means (512: 9.8 and 14.6).
//
// Whether a ratio is clipped is decided by x against the bounds' logarithms,
// as if x had not been rounded: r's own rounding would move tokens over the
// border, where the gradient jumps.  Sums are FP32 over a tile, in a fixed
// order, and compensated FP32 over tiles and sequences.
#include "device_status.h"
#include "policy_loss.h"

TILE_DEVICE_STATUS(policy_loss)

namespace tile {
namespace {

constexpr unsigned int kBadOffsets = 1;
constexpr int kThreads = 256, kRows = 2, kTile = kThreads * kRows, kWarps = kThreads / 32;
constexpr int kMostFused = 8;   // tiles that one cluster does, joined without another launch

// The last sequence in [low, high] that begins at or before row.
__device__ __forceinline__ int sequence_of(const long long *offsets, long long row, int low, int high) {
    while (low < high) {
        const int mid = low + (high - low + 1) / 2;
        if (__ldg(offsets + mid) <= row)
            low = mid;
        else
            high = mid - 1;
    }
    return low;
}
// The same by a whole warp, which looks at 32 places at a time.
__device__ __forceinline__ int sequence_of_warp(const long long *offsets, long long row, int low, int high) {
    const int lane = threadIdx.x & 31;
    while (low < high) {
        const int step = (high - low + 31) / 32, at = low + (lane + 1) * step;
        const bool before = at <= high && __ldg(offsets + at) <= row;
        const unsigned int mask = __ballot_sync(0xffffffffu, before);
        // places up to the first lane that is behind the row (offsets that fall: in range all the same)
        const int n = mask == 0xffffffffu ? 32 : __ffs(~mask) - 1;
        const int top = low + (n + 1) * step - 1;
        low += n * step;
        if (top < high) high = top;
    }
    return low;
}

// The tile's sequences; those of its rows lie in [low, high].
struct Span {
    int low, high;
    long long first, last;   // rows that belong to a sequence
};
// search: whether low and high are wanted (by all threads of the CTA; not
// yet visible to them).
__device__ __forceinline__ void find_span(const PolicyArgs &a, long long tile0, bool search, Span *span) {
    const long long tile1 = min(tile0 + kTile, static_cast<long long>(a.rows)) - 1;
    const int warp = threadIdx.x >> 5;
    if (a.offsets == nullptr) {
        if (threadIdx.x == 0) *span = Span{0, 0, 0, a.rows};
    } else if (warp < 2) {
        const long long edge = __ldg(a.offsets + (warp == 0 ? 0 : a.sequences));
        const int s = search ? sequence_of_warp(a.offsets, warp == 0 ? tile0 : tile1, 0, a.sequences - 1) : 0;
        if (threadIdx.x == 0) {
            span->low = s;
            span->first = edge;
        } else if (threadIdx.x == 32) {
            span->high = s;
            span->last = edge;
        }
    }
}

// Whether old - nll > bound (sign 1) or < bound (sign -1), unrounded.
__device__ __forceinline__ bool beyond(float old, float nll, float x, float bound, float rest, float sign) {
    if (x != bound) return sign * x > sign * bound;
    const float back = __fsub_rn(x, old);   // x + what its rounding cut off is old - nll
    const float cut = __fsub_rn(__fsub_rn(old, __fsub_rn(x, back)), __fadd_rn(nll, back));
    return sign * cut > sign * rest;
}

// A row's inputs.
struct Token {
    float nll, old, ref, adv;
    bool counts;
};

// Rows tile0 + thread + 256 u of the tile, with the loads on their way before
// the sequences are known.
__device__ __forceinline__ void load_tokens(const PolicyArgs &a, long long tile0, Token (&t)[kRows]) {
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const long long row = tile0 + threadIdx.x + u * kThreads;
        t[u] = Token{0.0f, 0.0f, 0.0f, 0.0f, false};
        if (row >= a.rows) continue;
        t[u].counts = a.target == nullptr || __ldcs(a.target + row) != a.ignore;
        t[u].nll = __ldcs(a.nll + row);
        t[u].old = __ldcs(a.old_nll + row);
        if (a.ref_nll != nullptr) t[u].ref = __ldcs(a.ref_nll + row);
        if (!a.sequence_advantage) t[u].adv = __ldcs(a.advantage + row);
    }
}
// Which of them count, and their sequences where those are wanted.
__device__ __forceinline__ void place_tokens(const PolicyArgs &a, long long tile0, const Span &span,
                                             Token (&t)[kRows], int (&of)[kRows], bool need_of) {
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const long long row = tile0 + threadIdx.x + u * kThreads;
        t[u].counts &= row >= span.first && row < span.last;
        of[u] = span.low;
        if (!t[u].counts || !(need_of || a.sequence_advantage)) continue;
        if (a.offsets != nullptr) of[u] = sequence_of(a.offsets, row, span.low, span.high);
        if (a.sequence_advantage) t[u].adv = __ldg(a.advantage + of[u]);
    }
}

__device__ __forceinline__ bool is_clipped(const PolicyArgs &a, const Token &t, float x) {
    return t.adv > 0.0f ? beyond(t.old, t.nll, x, a.high, a.high_rest, 1.0f)
                        : t.adv < 0.0f && beyond(t.old, t.nll, x, a.low, a.low_rest, -1.0f);
}

// e^q - q - 1.  Up to 1/2 as q^2 times a polynomial, (e^q - q - 1) / q^2 interpolated
// at Chebyshev's nodes (2^-25 of it; with the roundings 3.2 of 2^-24): the term is about
// q^2 / 2 there, and expm1f(q) - q would leave an ulp of q in it, as much as the
// term itself at |q| = 1e-7, where a policy is still at its reference.  (Both are
// computed.  In one run, 1048576 tokens: 9.6 us; with a branch between them 9.8,
// expm1f alone 9.4.)
__device__ __forceinline__ float kl_term(float q) {
    float p = 0.00019962186f;
    p = fmaf(p, q, 0.0013982197f);
    p = fmaf(p, q, 0.008333182f);
    p = fmaf(p, q, 0.041665791f);
    p = fmaf(p, q, 0.16666667f);
    p = fmaf(p, q, 0.5f);
    const float far = expm1f(q) - q;
    return fabsf(q) > 0.5f ? far : q * q * p;
}

// (surrogate, KL, clipped, 1) of a token; zeros for one that does not count.
__device__ __forceinline__ float4 parts_of(const PolicyArgs &a, const Token &t) {
    if (!t.counts) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float x = __fsub_rn(t.old, t.nll);
    const bool clipped = is_clipped(a, t, x);
    const float ratio = clipped ? (t.adv > 0.0f ? 1.0f + a.clip_high : 1.0f - a.clip_low) : expf(x);
    const float kl = a.ref_nll != nullptr ? kl_term(__fsub_rn(t.nll, t.ref)) : 0.0f;
    return make_float4(t.adv == 0.0f ? 0.0f : -ratio * t.adv, kl, clipped ? 1.0f : 0.0f, 1.0f);
}

__device__ __forceinline__ float4 add4(float4 p, float4 q) {
    return make_float4(p.x + q.x, p.y + q.y, p.z + q.z, p.w + q.w);
}
__device__ __forceinline__ float4 warp_sum(float4 v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, d);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, d);
        v.z += __shfl_xor_sync(0xffffffffu, v.z, d);
        v.w += __shfl_xor_sync(0xffffffffu, v.w, d);
    }
    return v;
}

struct TileMem {
    Span span;
    float4 part[kTile];
};

// Sums of a tile: slots[tile] of all its tokens or, by sequence, slots[tile +
// s] of those of sequence s (tile and s both grow along the rows: no other
// tile and sequence share that slot).
__device__ __forceinline__ void tile_sums(const PolicyArgs &a, int tile, float4 *slots, TileMem &mem) {
    const long long tile0 = static_cast<long long>(tile) * kTile;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Token t[kRows];
    int of[kRows];
    load_tokens(a, tile0, t);
    find_span(a, tile0, a.sequence_mean || a.sequence_advantage, &mem.span);
    __syncthreads();
    const Span span = mem.span;
    place_tokens(a, tile0, span, t, of, false);
    if (!a.sequence_mean) {
        float4 v = parts_of(a, t[0]);
#pragma unroll
        for (int u = 1; u < kRows; ++u) v = add4(v, parts_of(a, t[u]));
        v = warp_sum(v);
        if (lane == 0) mem.part[warp] = v;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kWarps; ++w) v = add4(v, mem.part[w]);
            slots[tile] = v;
        }
        return;
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) mem.part[threadIdx.x + u * kThreads] = parts_of(a, t[u]);
    __syncthreads();
    const int count = span.high - span.low + 1;
    // a warp for each sequence, or a thread where there are many
    const bool wide = count <= 8 * kWarps;
    for (int k = wide ? warp : threadIdx.x; k < count; k += wide ? kWarps : kThreads) {
        const int s = span.low + k;
        long long begin = 0, end = a.rows;
        if (a.offsets != nullptr) {
            begin = __ldg(a.offsets + s);
            end = __ldg(a.offsets + s + 1);
        }
        const long long most = kTile;   // (offsets that do not grow stay within the tile)
        const int from = static_cast<int>(max(min(begin - tile0, most), 0ll));
        const int to = static_cast<int>(max(min(end - tile0, most), 0ll));
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int i = from + (wide ? lane : 0); i < to; i += wide ? 32 : 1) v = add4(v, mem.part[i]);
        if (wide) v = warp_sum(v);
        if (!wide || lane == 0) slots[static_cast<long long>(tile) + s] = v;
    }
}

// An FP32 sum with what its roundings cut off (Knuth's two-sum): FP64 sums of
// the tiles by all threads took 40 us more of 1048576 tokens.
struct Sum {
    float s, cut;
    __device__ __forceinline__ void add(float x) {
        const float to = __fadd_rn(s, x), back = __fsub_rn(to, s);
        cut += __fadd_rn(__fsub_rn(s, __fsub_rn(to, back)), __fsub_rn(x, back));
        s = to;
    }
    __device__ __forceinline__ void add(Sum o) {
        add(o.s);
        cut += o.cut;
    }
    __device__ __forceinline__ float value() const { return isfinite(s) ? s + cut : s; }
};
struct Sums {
    Sum v[4];   // surrogate, KL, clipped, and tokens or sequences that count
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i].s = v[i].cut = 0.0f;
    }
    __device__ __forceinline__ void add(float4 p) {
        v[0].add(p.x);
        v[1].add(p.y);
        v[2].add(p.z);
        v[3].add(p.w);
    }
    // over the warp, for every lane
    __device__ __forceinline__ void warp() {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                Sum o;
                o.s = __shfl_xor_sync(0xffffffffu, v[i].s, d);
                o.cut = __shfl_xor_sync(0xffffffffu, v[i].cut, d);
                v[i].add(o);
            }
    }
};

// The slots' sums to stats and weights.
template <int THREADS>
__device__ __forceinline__ void join_sums(const PolicyArgs &a, const float4 *slots) {
    __shared__ Sums part[THREADS / 32];
    __shared__ float shared_share;
    const int tiles = (a.rows + kTile - 1) / kTile, tid = threadIdx.x, lane = tid & 31;
    Sums sum;
    sum.zero();
    bool bad = false;
    if (!a.sequence_mean)
        for (int t = tid; t < tiles; t += THREADS) sum.add(__ldcg(slots + t));
    for (int base = 0; base < a.sequences; base += THREADS) {
        const int s = base + tid;
        long long begin = 0, end = s < a.sequences ? a.rows : 0;
        if (a.offsets != nullptr && s < a.sequences) {
            begin = __ldg(a.offsets + s);
            end = __ldg(a.offsets + s + 1);
            if (begin < 0 || end < begin || end > a.rows) {
                bad = true;
                begin = end = 0;
            }
        }
        if (!a.sequence_mean) continue;
        Sums v;
        v.zero();
        const int first = static_cast<int>(begin / kTile);
        const int last = begin < end ? static_cast<int>((end - 1) / kTile) : first - 1;
        if (last - first < 32)
#pragma unroll 4
            for (int t = first; t <= last; ++t) v.add(__ldcg(slots + static_cast<long long>(t) + s));
        // long sequences: the warp together
        unsigned int left = __ballot_sync(0xffffffffu, last - first >= 32);
        while (left != 0) {
            const int from = __ffs(left) - 1;
            left &= left - 1;
            const int f = __shfl_sync(0xffffffffu, first, from), l = __shfl_sync(0xffffffffu, last, from);
            const int of = __shfl_sync(0xffffffffu, s, from);
            Sums w;
            w.zero();
            for (int t = f + lane; t <= l; t += 32) w.add(__ldcg(slots + static_cast<long long>(t) + of));
            w.warp();
            if (lane == from) v = w;
        }
        const float n = v.v[3].value();   // (a count below 2^30: to FP32's rounding)
        const bool counts = n > 0.0f;
        if (s < a.sequences) a.weights[s] = counts ? 1.0f / n : 0.0f;
        if (counts)
            sum.add(make_float4(v.v[0].value() / n, v.v[1].value() / n, v.v[2].value() / n, 1.0f));
    }
    bad = __syncthreads_or(bad);
    sum.warp();
    if (lane == 0) part[tid >> 5] = sum;
    __syncthreads();
    if (tid < 32) {
        sum.zero();
        if (tid < THREADS / 32) sum = part[tid];
        sum.warp();
        const float n = sum.v[3].value(), share = n > 0.0f ? 1.0f / n : 0.0f;
        if (tid == 0) {
            shared_share = share;
            const float nan = __int_as_float(0x7fffffff);
            if (bad) atomicOr(a.status, kBadOffsets);
            const float surrogate = bad ? nan : n > 0.0f ? sum.v[0].value() / n : 0.0f;
            const float kl = bad ? nan : n > 0.0f ? sum.v[1].value() / n : 0.0f;
            // (a term that is only looked at: e^q may be infinite, and 0 times it NaN)
            a.stats[0] = a.kl_coef != 0.0f ? fmaf(a.kl_coef, kl, surrogate) : surrogate;
            a.stats[1] = surrogate;
            a.stats[2] = kl;
            a.stats[3] = bad ? nan : n > 0.0f ? sum.v[2].value() / n : 0.0f;
        }
    }
    __syncthreads();
    const float share = shared_share;
    for (int s = tid; s < a.sequences; s += THREADS)   // (each thread its own ones)
        a.weights[s] = a.sequence_mean ? a.weights[s] * share : share;
}

__global__ void __launch_bounds__(kThreads) tiles_kernel(const PolicyArgs a) {
    __shared__ TileMem mem;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tile_sums(a, blockIdx.x, static_cast<float4 *>(a.ws), mem);
}

constexpr int kJoinThreads = 512;
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const PolicyArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the tiles' sums are written
    join_sums<kJoinThreads>(a, static_cast<const float4 *>(a.ws));
}

// A cluster of as many CTAs as there are tiles; the first one joins them.
__global__ void __launch_bounds__(kThreads) fused_kernel(const PolicyArgs a) {
    __shared__ TileMem mem;
    tile_sums(a, blockIdx.x, static_cast<float4 *>(a.ws), mem);
    __syncthreads();
    __threadfence();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (blockIdx.x == 0) join_sums<kThreads>(a, static_cast<const float4 *>(a.ws));
}

__global__ void __launch_bounds__(kThreads) backward_kernel(const PolicyArgs a) {
    __shared__ Span shared_span;
    const long long tile0 = static_cast<long long>(blockIdx.x) * kTile;
    const float up = a.dloss != nullptr ? __ldg(a.dloss) : 1.0f;
    Token t[kRows];
    int of[kRows];
    load_tokens(a, tile0, t);
    find_span(a, tile0, true, &shared_span);
    __syncthreads();
    const Span span = shared_span;
    place_tokens(a, tile0, span, t, of, true);
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const long long row = tile0 + threadIdx.x + u * kThreads;
        if (row >= a.rows) continue;
        float d = 0.0f;
        if (t[u].counts) {
            const float x = __fsub_rn(t[u].old, t[u].nll);
            if (t[u].adv != 0.0f && !is_clipped(a, t[u], x)) d = expf(x) * t[u].adv;
            if (a.ref_nll != nullptr) d = fmaf(a.kl_coef, expm1f(__fsub_rn(t[u].nll, t[u].ref)), d);
            d *= __ldg(a.weights + of[u]) * up;
        }
        __stcs(a.dnll + row, d);
    }
}

}  // namespace

size_t policy_loss_workspace(int rows, int sequences) {
    const size_t tiles = (static_cast<size_t>(rows) + kTile - 1) / kTile;
    return (tiles + static_cast<size_t>(sequences)) * sizeof(float4);
}

cudaError_t launch_policy_loss(PolicyArgs a, cudaStream_t stream) {
    cudaError_t err = cudaSuccess;
    a.status = status_address(&err);
    if (a.status == nullptr) return err;
    const int tiles = (a.rows + kTile - 1) / kTile;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(tiles);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    if (tiles <= kMostFused) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = tiles;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, fused_kernel, a);
    }
    err = cudaLaunchKernelEx(&cfg, tiles_kernel, a);
    if (err != cudaSuccess) return err;
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kJoinThreads);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel, a);
}

cudaError_t launch_policy_loss_backward(PolicyArgs a, cudaStream_t stream) {
    backward_kernel<<<(a.rows + kTile - 1) / kTile, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace tile
