// Embedding lookup, out[i] = scale weight[token[i]], and its gradient,
// dweight[v] (+)= scale (sum of dout[i] over the rows with token[i] = v).
//
// Both are bound by DRAM: the lookup reads each row of the weight that occurs
// and writes rows x width; the gradient reads rows x width and writes the
// whole weight's shape, or reads and writes the rows that occur where it adds.
//
// The gradient sums the rows of a token in the order of their positions, in
// FP32, so that results are bitwise reproducible.  Few rows: a CTA for each
// row looks for the row's token among all tokens, and the first row of a token
// sums them (one launch, no workspace).  More rows: positions are brought in
// the order of their tokens, up to 6144 by counting, more by a stable radix
// sort of up to 9 bits a pass; then the list is summed in runs of 8 to 64
// positions (more where the partial sums would pass 64 MiB), and a token that
// fills more than a run is joined from partial sums.  The rows of tokens that
// do not occur are zeroed by CTAs that the launches of this chain carry along.
//
// (One GB300, a copy moves 6.68 TB/s.  32768 x 4096 BF16 against 131072
// entries: lookup 59 us of the device's time, 0.93 of that rate; gradient 209
// us, 0.96, added to another 116, 0.60; in FP32 352, 1.03, and added 143, 0.69.
// 5000 x 1537 FP32 against 50001, a third of it ignored: 69 us, 0.71.  Rows off
// the 16-byte grid cost two loads a window and the shifts: 32768 x 4097 BF16 lookup
// 80 us, 0.69, gradient 254, 0.79, added 190, 0.37.)
#include "device_status.h"
#include "embedding.h"
#include "row_windows.cuh"

TILE_DEVICE_STATUS(embedding)

namespace tile {
namespace {

constexpr unsigned int kBadToken = 1;

// Token at i, or -1 where it has no row: ignored, or out of range (noted).
__device__ __forceinline__ int token_row(const EmbeddingArgs &a, long long t) {
    if (t == a.ignore) return -1;
    if (t >= 0 && t < a.vocab) return static_cast<int>(t);
    atomicOr(a.status, kBadToken);
    return -2;
}

template <class T>
__device__ __forceinline__ int windows_of(int width, bool vec) {
    constexpr int V = 16 / sizeof(T);
    return vec ? width / V : (width + V - 1) / V + 1;
}

// The next kernel of the chain may be set up; this one's inputs are written.  (What
// an earlier kernel of the chain wrote is not read through the read-only cache:
// this kernel may have begun before.)
__device__ __forceinline__ void let_next_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- lookup ---------------------------------------------------------------------

// `lanes` (a power of two) threads a row, up to 4 windows of it each at a time;
// of a row off the 16-byte grid, those that are whole, and the elements at its
// ends one by one.
template <class T, bool VEC>
__global__ void __launch_bounds__(256) lookup_kernel(const EmbeddingArgs a, int lanes) {
    constexpr int V = 16 / sizeof(T), U = 4;
    const int lane = threadIdx.x & (lanes - 1), per = 256 / lanes;
    const int row = blockIdx.x * per + threadIdx.x / lanes;
    if (row >= a.rows) return;
    const int token = token_row(a, __ldg(a.tokens + row));
    const T *src = static_cast<const T *>(a.weight) + static_cast<long long>(token < 0 ? 0 : token) * a.width;
    T *dst = static_cast<T *>(a.out) + static_cast<long long>(row) * a.width;
    auto scaled = [&](float v) {   // an ignored row is 0 whatever the scale, a bad one NaN
        return token >= 0 ? v * a.scale : token == -1 ? 0.0f : __int_as_float(0x7fffffff);
    };
    int head = 0;
    if constexpr (!VEC) {
        head = min((V - window_phase(dst)) % V, a.width);
        const int body = (a.width - head) / V * V;
        for (int e = lane; e < a.width - body; e += lanes) {
            const int at = e < head ? e : body + e;
            store_one(dst + at, scaled(token >= 0 ? static_cast<float>(src[at]) : 0.0f));
        }
    }
    const int windows = (a.width - head) / V;
    const Bounds bounds = bounds_of<T>(a.weight, a.vocab, a.width);
    for (int j = lane; j < windows; j += U * lanes) {
        RawWindow<VEC> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            raw[u] = fetch_window<T, VEC>(src, (j + u * lanes) * V + head, bounds,
                                          token >= 0 && j + u * lanes < windows);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j + u * lanes < windows) {
                const int at = (j + u * lanes) * V + head;
                float v[V];
                widen_vec<T>(token >= 0 ? join_window<T, VEC>(raw[u], src, at, a.width) : make_uint4(0, 0, 0, 0), v);
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = scaled(v[i]);
                store_window<T, V, true>(dst, at, a.width, v);
            }
    }
}

template <class T, bool VEC>
cudaError_t launch_lookup(const EmbeddingArgs &a, cudaStream_t stream) {
    const int windows = a.width / (16 / static_cast<int>(sizeof(T)));
    int lanes = 8;
    while (lanes < 256 && lanes * 4 < windows) lanes *= 2;
    // few rows: one window a thread
    const long long few = sm_count_of_device() * 512;
    while (lanes < 256 && lanes < windows && static_cast<long long>(a.rows) * lanes < few) lanes *= 2;
    const int per = 256 / lanes;
    lookup_kernel<T, VEC><<<(a.rows + per - 1) / per, 256, 0, stream>>>(a, lanes);
    return cudaGetLastError();
}

// ---- gradient: few rows ------------------------------------------------------------

// CTA (i, s): the rows of token[i], if i is the first of them; PER tokens of all
// rows in each thread's registers.  A token of many rows: each CTA has slice s
// of 32 windows, its warps parts of the rows.  One of a few: the CTAs of the
// first slices have a slice for each warp, and the others leave.
constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32, kMostFew = 2048;

template <class T, class D, bool VEC, int PER>
__global__ void __launch_bounds__(kFewThreads) few_rows_kernel(const EmbeddingArgs a) {
    constexpr int V = 16 / sizeof(T), U = 4;
    __shared__ unsigned short list[kFewThreads * PER];
    __shared__ int found[PER * kFewWarps];   // hits of each 32 tokens; then hits before them
    __shared__ int count;
    __shared__ float part[kFewWarps][32][V + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, i = blockIdx.x;
    const long long t = __ldg(a.tokens + i);
    unsigned int mask[PER];
    bool first = true;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int j = k * kFewThreads + tid;
        mask[k] = j < a.rows && __ldg(a.tokens + j) == t;
    }
    const int token = t == a.ignore || t < 0 || t >= a.vocab ? -1 : static_cast<int>(t);
    if (token < 0) {
        if (tid == 0 && blockIdx.y == 0) token_row(a, t);
        return;
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        first = first && !(mask[k] != 0 && k * kFewThreads + tid < i);
        mask[k] = __ballot_sync(0xffffffffu, mask[k] != 0);
        if (lane == 0) found[k * kFewWarps + warp] = __popc(mask[k]);
    }
    if (!__syncthreads_and(first)) return;
    int n = 0;
    if constexpr (PER == 1) {
        int before = 0;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            const int c = found[w];
            before += w < warp ? c : 0;
            n += c;
        }
        if (mask[0] >> lane & 1)
            list[before + __popc(mask[0] & ((1u << lane) - 1))] = static_cast<unsigned short>(tid);
    } else {
        if (warp == 0) {
            static_assert(PER * kFewWarps == 64, "two for each lane");
            const int one = found[2 * lane], two = found[2 * lane + 1];
            int sum = one + two;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += up;
            }
            found[2 * lane] = sum - one - two;
            found[2 * lane + 1] = sum - two;
            if (lane == 31) count = sum;
        }
        __syncthreads();
        n = count;
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (mask[k] >> lane & 1)
                list[found[k * kFewWarps + warp] + __popc(mask[k] & ((1u << lane) - 1))] =
                    static_cast<unsigned short>(k * kFewThreads + tid);
    }
    const bool split = n > kFewWarps / 2;
    const int slice = split ? blockIdx.y : blockIdx.y * kFewWarps + warp;
    D *dst = static_cast<D *>(a.dweight) + static_cast<long long>(token) * a.width;
    const int phase = VEC ? 0 : window_phase(dst);
    const int windows = windows_of<T>(a.width, VEC);
    if (!split && static_cast<int>(blockIdx.y) * kFewWarps * 32 >= windows) return;
    __syncthreads();
    const Bounds bounds = bounds_of<T>(a.dout, a.rows, a.width);
    const int from = split ? n * warp / kFewWarps : 0, to = split ? n * (warp + 1) / kFewWarps : n;
    const int at = (slice * 32 + lane) * V - phase;
    const bool in = slice * 32 + lane < windows;
    float sum[V] = {}, old[V] = {};
    if (a.add && in && (!split || warp == 0)) read_window<D, V, VEC>(dst, at, a.width, old);
    for (int k = from; k < to; k += U) {
        RawWindow<VEC> raw[U];
        const T *row[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            row[u] = static_cast<const T *>(a.dout) + static_cast<long long>(list[min(k + u, to - 1)]) * a.width;
            raw[u] = fetch_window<T, VEC>(row[u], at, bounds, in && k + u < to);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!in || k + u >= to) continue;
            float v[V];
            widen_vec<T>(join_window<T, VEC>(raw[u], row[u], at, a.width), v);
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] += v[e];
        }
    }
    if (split) {
#pragma unroll
        for (int e = 0; e < V; ++e) part[warp][lane][e] = sum[e];
        __syncthreads();
        if (warp != 0) return;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            sum[e] = 0.0f;
#pragma unroll
            for (int w = 0; w < kFewWarps; ++w) sum[e] += part[w][lane][e];
        }
    }
    if (!in) return;
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] = fmaf(sum[e], a.scale, old[e]);
    store_window<D, V, VEC>(dst, at, a.width, sum);
}

// Few rows: each CTA looks at all tokens, 1 to 2 ns a CTA, where ranking them,
// the sums and the join are a chain of launches.  The rule counts CTAs of 128 columns:
// FP32's, 16-bit types have half as many.  (Device times in a graph, all tokens
// different, new gradient of 4096 entries, few | ranked.  BF16: 256 x 4096 11.3 |
// 14.4 us, 512 x 1024 8.5 | 12.5, 1024 x 256 6.7 | 12.3, 1024 x 512 8.5 | 12.4, 1024 x
// 1024 12.9 | 13.6, 512 x 4096 23.7 | 14.8, 2048 x 256 9.5 | 12.4, of one token 29 |
// 27.  FP32: 256 x 4096 19.0 | 20.4, 512 x 1024 13.3 | 12.3, 1024 x 256 8.2 | 12.3,
// 1024 x 512 12.6 | 12.4, 2048 x 256 12.4 | 12.3.  Added to, in BF16 5.9 | 5.7, 6.2 |
// 6.2, 5.4 | 6.7, 6.7 | 7.0, 10.5 | 6.7, 18.0 | 6.7, 8.6 | 7.7; in FP32, where the
// rule keeps more than it should, 9.5 | 6.2, 9.8 | 5.9, 6.4 | 6.7, 10.3 | 6.7, 11.1 |
// 7.5.)
bool few_rows(int rows, int width) {
    const long long ctas = static_cast<long long>(rows) * (width / 128 + 1);
    return rows <= kFewThreads ? ctas <= 16384 : rows <= kMostFew && ctas <= 6000;
}

// ---- gradient: sorting positions by token --------------------------------------------

constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32, kMaxBits = 9;
constexpr int kMaxBins = 1 << kMaxBits;

struct Pair {
    unsigned int key, at;   // token (vocab: none) and position
};

struct SortPlan {
    int passes, bits, items, tiles;   // items a thread: 2, 4 or 16
};

SortPlan sort_plan(int rows, int vocab) {
    int all = 1;
    while ((1ll << all) <= vocab) ++all;   // keys 0 .. vocab
    SortPlan p;
    p.passes = (all + kMaxBits - 1) / kMaxBits;
    p.bits = (all + p.passes - 1) / p.passes;
    // Each tile adds up the counts of all tiles: short ones are done sooner while
    // they are few.  (The gradient of 64 BF16 columns, added, tokens by frequency, with
    // 2, 4 and 16 items: 32768 rows 34, 36 and 64 us, 65536 49, 54 and 73, 98304 66, 62
    // and 85, 140000 89, 80 and 100, 196608 112, 104 and 116, 262144 143, 140 and 139,
    // 393216 201, 193 and 186, 2^20 394, 249 and 211; with 1024 columns the orders
    // are the same.  The counts that all tiles read grow with the square of the
    // rows all the same: 2^24 rows take 3.6 ms, of which the bytes are 0.35.)
    p.items = rows <= 81920 ? 2 : rows <= 262144 ? 4 : 16;
    p.tiles = (rows + kSortThreads * p.items - 1) / (kSortThreads * p.items);
    return p;
}

__device__ __forceinline__ unsigned int key_at(const EmbeddingArgs &a, int i) {
    const int row = token_row(a, __ldg(a.tokens + i));
    return row < 0 ? static_cast<unsigned int>(a.vocab) : static_cast<unsigned int>(row);
}

// Counts of the first digit in each tile; the later passes' counts to zero;
// and, in `present`, a bit for each token that occurs (NULL: not wanted).
template <int ITEMS>
__global__ void __launch_bounds__(kSortThreads)
    digits_kernel(const EmbeddingArgs a, int *counts, unsigned int *present, int bits, int passes) {
    constexpr int U = ITEMS < 8 ? ITEMS : 8;
    __shared__ int bins[kMaxBins];
    let_next_start();
    const int n = 1 << bits, tiles = gridDim.x;
    for (int d = threadIdx.x; d < n; d += kSortThreads) bins[d] = 0;
    __syncthreads();
    const unsigned int none = a.vocab;
    for (int r = 0; r < ITEMS; r += U) {
        unsigned int key[U], word[U];
        const int begin = (blockIdx.x * ITEMS + r) * kSortThreads + threadIdx.x;
#pragma unroll
        for (int u = 0; u < U; ++u) key[u] = begin + u * kSortThreads < a.rows ? key_at(a, begin + u * kSortThreads) : ~0u;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (key[u] != ~0u) atomicAdd(&bins[key[u] & (n - 1)], 1);
            word[u] = present != nullptr && key[u] < none ? __ldcg(present + (key[u] >> 5)) : ~0u;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)   // a token that occurs often is mostly noted already
            if ((word[u] >> (key[u] & 31) & 1) == 0) atomicOr(present + (key[u] >> 5), 1u << (key[u] & 31));
    }
    __syncthreads();
    for (int d = threadIdx.x; d < n; d += kSortThreads) {
        const long long at = static_cast<long long>(blockIdx.x) * n + d;
        counts[at] = bins[d];
        for (int p = 1; p < passes; ++p) counts[at + static_cast<long long>(p) * tiles * n] = 0;
    }
}

// Zeros to the rows of dweight whose token does not occur: `each` rows from
// from + part * each on, below `to`, with `lanes` threads a row.  CTAs of the
// sort, the sums and the join have shares of them, so that DRAM is busy while
// those wait for loads.
struct Fill {
    const unsigned int *present;
    int from, to, each, lanes;
};
template <class D, bool VEC, int THREADS>
__device__ __forceinline__ void fill_rows(const EmbeddingArgs &a, const Fill &f, int part) {
    constexpr int N = 16 / sizeof(D);
    const int lane = threadIdx.x & (f.lanes - 1), per = THREADS / f.lanes;
    const int windows = windows_of<D>(a.width, VEC);
    const float zero[N] = {};
    const long long first = f.from + static_cast<long long>(part) * f.each;
    const long long end = min(first + f.each, static_cast<long long>(f.to));
    for (long long v = first + threadIdx.x / f.lanes; v < end; v += per) {
        if (f.present[v >> 5] >> (v & 31) & 1) continue;
        D *row = static_cast<D *>(a.dweight) + v * a.width;
        const int phase = VEC ? 0 : window_phase(row);
        for (int j = lane; j < windows; j += f.lanes)
            store_window<D, N, VEC>(row, j * N - phase, a.width, zero);
    }
}

// One stable pass: a pair goes behind those of smaller digits, and behind those
// of its digit in earlier tiles, warps and places.  Integer atomics count the
// next digit by the tile that a pair lands in; their order changes nothing.
template <class D, bool VEC, int ITEMS, bool FIRST>
__global__ void __launch_bounds__(kSortThreads)
    scatter_kernel(const EmbeddingArgs a, const Pair *in, Pair *out, const int *counts, int *next,
                   int bits, int shift, bool last, int tiles, const Fill fill) {
    let_next_start();
    wait_for_previous();
    if (static_cast<int>(blockIdx.x) >= tiles) {
        fill_rows<D, VEC, kSortThreads>(a, fill, blockIdx.x - tiles);
        return;
    }
    __shared__ int warp_bins[kSortWarps][kMaxBins];
    __shared__ int base[kMaxBins];
    __shared__ int sums[kSortWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = 1 << bits;
    const int begin = blockIdx.x * kSortThreads * ITEMS + warp * 32 * ITEMS;
    Pair pair[ITEMS];   // on their way while the counts are added up
#pragma unroll
    for (int r = 0; r < ITEMS; ++r) {
        const int i = begin + r * 32 + lane;
        pair[r] = Pair{0, 0};
        if (i < a.rows) {
            if constexpr (FIRST)
                pair[r] = Pair{key_at(a, i), static_cast<unsigned int>(i)};
            else
                pair[r] = in[i];
        }
    }
    for (int d = tid; d < kSortWarps * kMaxBins; d += kSortThreads) (&warp_bins[0][0])[d] = 0;
    // digits 2 tid and 2 tid + 1: pairs before this tile, and in all
    int before[2] = {}, total[2] = {};
    const int d0 = 2 * tid;
    if (d0 < n) {
#pragma unroll 8
        for (int t = 0; t < tiles; ++t) {
            const int2 c = *reinterpret_cast<const int2 *>(counts + static_cast<long long>(t) * n + d0);
            if (t < static_cast<int>(blockIdx.x)) {
                before[0] += c.x;
                before[1] += c.y;
            }
            total[0] += c.x;
            total[1] += c.y;
        }
    }
    int scan = total[0] + total[1];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += up;
    }
    if (lane == 31) sums[warp] = scan;
    __syncthreads();
    for (int w = 0; w < warp; ++w) scan += sums[w];
    scan -= total[0] + total[1];
    if (d0 < n) {
        base[d0] = scan + before[0];
        base[d0 + 1] = scan + total[0] + before[1];
    }
    int rank[ITEMS];
#pragma unroll
    for (int r = 0; r < ITEMS; ++r) {
        const bool live = begin + r * 32 + lane < a.rows;
        const int digit = live ? static_cast<int>(pair[r].key >> shift) & (n - 1) : -1;
        const unsigned int peers = __match_any_sync(0xffffffffu, digit);
        rank[r] = __popc(peers & ((1u << lane) - 1));
        const int had = live ? warp_bins[warp][digit] : 0;
        __syncwarp();
        if (live && rank[r] == 0) warp_bins[warp][digit] = had + __popc(peers);
        rank[r] += had;
        __syncwarp();
    }
    __syncthreads();
    for (int d = tid; d < n; d += kSortThreads) {
        int at = base[d];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = warp_bins[w][d];
            warp_bins[w][d] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ITEMS; ++r)
        if (begin + r * 32 + lane < a.rows) {
            const int to = warp_bins[warp][static_cast<int>(pair[r].key >> shift) & (n - 1)] + rank[r];
            out[to] = pair[r];
            if (!last)
                atomicAdd(next + static_cast<long long>(to / (kSortThreads * ITEMS)) * n +
                              (static_cast<int>(pair[r].key >> (shift + bits)) & (n - 1)), 1);
        }
}

// Up to kMostRanked positions go to their places at once: that of i is the
// number of j with a smaller key, or the same key and j < i.  CTA b counts them
// for positions 32 b .. 32 b + 31 against all keys in its shared memory.  (With the
// sums of 1024 columns, ranked | sorted by the passes above: 1000 rows 6.8 | 14.4
// us, 2500 9.2 | 16.7, 4000 11.3 | 18.6, 6000 17 | 20, 8192 23 | 21.)
constexpr int kMostRanked = 6144, kRankThreads = 512, kRankPer = 2;
__global__ void __launch_bounds__(kRankThreads)
    rank_kernel(const EmbeddingArgs a, Pair *out, unsigned int *present) {
    constexpr int U = 8;
    __shared__ uint4 keys[kMostRanked / 4];
    unsigned int *key = reinterpret_cast<unsigned int *>(keys);
    let_next_start();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int vectors = (a.rows + 127) / 128 * 32;   // of four keys: the same number for each lane
    for (int begin = tid; begin < vectors * 4; begin += U * kRankThreads) {
        long long t[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            t[u] = begin + u * kRankThreads < a.rows ? __ldg(a.tokens + begin + u * kRankThreads) : a.ignore;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = begin + u * kRankThreads;
            if (j >= vectors * 4) continue;
            const bool valid = t[u] != a.ignore && t[u] >= 0 && t[u] < a.vocab;
            if (blockIdx.x == 0 && !valid && t[u] != a.ignore) token_row(a, t[u]);
            key[j] = j >= a.rows ? ~0u : valid ? static_cast<unsigned int>(t[u]) : static_cast<unsigned int>(a.vocab);
        }
    }
    __syncthreads();
    const int base = blockIdx.x * 32, first = base + warp * kRankPer;
    unsigned int own[kRankPer];
    int count[kRankPer];
#pragma unroll
    for (int q = 0; q < kRankPer; ++q) {
        own[q] = key[first + q];   // (behind the last row: not used)
        // of this CTA's 32 positions, those before it with the same key
        count[q] = lane < warp * kRankPer + q && key[base + lane] == own[q];
    }
#pragma unroll 4
    for (int v = lane; v < vectors; v += 32) {
        const uint4 k = keys[v];
        const unsigned int more = v < base / 4;   // before this CTA's positions equal keys count
#pragma unroll
        for (int q = 0; q < kRankPer; ++q) {
            const unsigned int bound = own[q] + more;
            count[q] += (k.x < bound) + (k.y < bound) + (k.z < bound) + (k.w < bound);
        }
    }
#pragma unroll
    for (int q = 0; q < kRankPer; ++q) {
        const int place = __reduce_add_sync(0xffffffffu, count[q]);
        if (lane != q || first + q >= a.rows) continue;
        out[place] = Pair{own[q], static_cast<unsigned int>(first + q)};
        if (present != nullptr && own[q] < static_cast<unsigned int>(a.vocab))
            atomicOr(present + (own[q] >> 5), 1u << (own[q] & 31));
    }
}

// ---- gradient: sums of the sorted list ------------------------------------------------

constexpr int kSumThreads = 128;
struct SumPlan {
    int run, runs;   // positions of a run, and how many there are
};
// Where a run ends decides the order of additions, so its length goes by 152 SMs, a
// whole GPU of this kind, on every device: the same bits there.
constexpr int kRunSms = 152;
// 64 positions a run; fewer, down to 8, where that leaves SMs without enough
// threads (32768 x 1536 BF16, added: 77 us, with 64 82); more where the partial sums
// would pass 64 MiB (131072 x 4096: 128 positions, 2^20 x 4096: 1024).
// (vector: elements of a window; the workspace has room for the runs of 8, the most.)
SumPlan sum_plan(int rows, int width, int vector) {
    const long long windows = width / vector + 1;
    auto bytes = [&](int run) { return (static_cast<long long>(rows) + run - 1) / run * 8 * (width + 16); };
    SumPlan p;
    p.run = 64;
    while (p.run > 8 && rows / p.run * windows < kRunSms * 1536) p.run /= 2;
    while (bytes(p.run) > (64ll << 20) && p.run < rows) p.run *= 2;
    p.runs = (rows + p.run - 1) / p.run;
    return p;
}

// A token belongs to the run that it begins in, which goes on up to as many
// rows behind its end to finish it.  Longer ones leave FP32 partial sums
// [runs][2][windows][V]: of a run's first token where it began in an earlier run,
// and of its last where it began here and goes on.
template <int V, class F>
__device__ __forceinline__ F *partial_at(F *partial, int run, int slot, int windows, int j) {
    return partial + ((static_cast<long long>(run) * 2 + slot) * windows + j) * V;
}
template <int V>
__device__ __forceinline__ void store_partial(float *p, const float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
        *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}

// What a window of dweight holds, as it lies there.
template <class D, int V>
struct OldWindow {
    static constexpr int N = 16 / sizeof(D), COUNT = V / N;
    uint4 raw[COUNT];
    __device__ __forceinline__ void load(const D *p) {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) raw[i] = *reinterpret_cast<const uint4 *>(p + i * N);
    }
    __device__ __forceinline__ void widen(float (&v)[V]) const {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            float p[N];
            widen_vec<D>(raw[i], p);
#pragma unroll
            for (int j = 0; j < N; ++j) v[i * N + j] = p[j];
        }
    }
};

// before: what the window holds, where it was loaded ahead.
template <class T, class D, bool VEC>
__device__ __forceinline__ void finish_row(const EmbeddingArgs &a, D *dst, int at, float (&sum)[16 / sizeof(T)],
                                           const OldWindow<D, 16 / sizeof(T)> *before = nullptr) {
    constexpr int V = 16 / sizeof(T);
    float old[V] = {};
    if (before != nullptr)
        before->widen(old);
    else if (a.add)
        read_window<D, V, VEC>(dst, at, a.width, old);
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] = fmaf(sum[e], a.scale, old[e]);
    store_window<D, V, VEC>(dst, at, a.width, sum);
}

// AHEAD: dweight is added to, and its rows are loaded with the first row of each
// token rather than at its last (32768 x 4096 BF16, added: 136 us).
template <class T, class D, bool VEC, bool AHEAD>
__global__ void __launch_bounds__(kSumThreads)
    sum_kernel(const EmbeddingArgs a, const Pair *pairs, float *partial, int run, int runs, int lanes,
               int slices, int ctas, const Fill fill) {
    constexpr int V = 16 / sizeof(T), U = !VEC ? 2 : AHEAD ? 4 : 8;
    let_next_start();
    wait_for_previous();
    // (fillers evenly between the CTAs that sum: 32768 x 4096 BF16 239 us, behind them 220)
    const int cta = blockIdx.x;
    if (cta >= ctas) {
        fill_rows<D, VEC, kSumThreads>(a, fill, cta - ctas);
        return;
    }
    const int lane = threadIdx.x & (lanes - 1);
    const int r = cta / slices * (kSumThreads / lanes) + threadIdx.x / lanes;
    const int windows = windows_of<T>(a.width, VEC);
    const int j = cta % slices * lanes + lane;
    if (r >= runs || j >= windows) return;
    const int begin = r * run, end = min(begin + run, a.rows);
    const unsigned int none = a.vocab, edge = ~0u;
    auto key_of = [&](long long k) { return k >= 0 && k < a.rows ? pairs[k].key : edge; };
    const unsigned int before = key_of(begin - run - 1ll), prior = key_of(begin - 1ll), front = key_of(begin),
                       tail = key_of(end - 1ll), after = key_of(end), far = key_of(static_cast<long long>(end) + run);
    if (front == none) return;
    // the first token goes on from an earlier run: that run's, if it began in the
    // one before this and ends here
    const bool left = prior == front, taken = left && (begin == run || before != front) && after != front;
    // the last one goes on, began here and ends in the next run: this run's
    const bool extend = tail != none && after == tail && !(tail == front && left) && far != tail;
    const int stop = extend ? min(end + run, a.rows) : end;
    auto pair_at = [&](int k) {   // no token where the row is not this run's
        Pair p = k < stop ? pairs[k] : Pair{none, 0};
        if (k >= end ? p.key != tail : taken && p.key == front) p.key = none;
        return p;
    };
    Pair next[U];   // the pairs of the rows after these
#pragma unroll
    for (int u = 0; u < U; ++u) next[u] = pair_at(begin + u);
    unsigned int cur = taken ? none : front;
    bool here = !left;
    const T *dout = static_cast<const T *>(a.dout);
    const Bounds bounds = bounds_of<T>(dout, a.rows, a.width);
    auto window_at = [&](unsigned int key) {   // (any place for no token)
        return VEC ? j * V : j * V - window_phase(static_cast<const D *>(a.dweight) + static_cast<long long>(key) * a.width);
    };
    // (a window that a row's end cuts is read element by element, at the token's last row)
    auto inside = [&](int to) { return VEC || (to >= 0 && to + V <= a.width); };
    D *dst = static_cast<D *>(a.dweight) + static_cast<long long>(cur) * a.width;
    int at = window_at(cur);
    float sum[V] = {};
    OldWindow<D, V> held;   // of the present token
    for (int k = begin; k < stop; k += U) {
        Pair p[U];
        RawWindow<VEC> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            p[u] = next[u];
            next[u] = pair_at(k + U + u);
        }
        if (k >= end && p[0].key == none) break;
#pragma unroll
        for (int u = 0; u < U; ++u)
            raw[u] = fetch_window<T, VEC>(dout + static_cast<long long>(p[u].at) * a.width, window_at(p[u].key),
                                          bounds, p[u].key != none);
        OldWindow<D, V> old[AHEAD ? U : 1];
        if constexpr (AHEAD) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int to = window_at(p[u].key);
                if (p[u].key != none && p[u].key != (u > 0 ? p[u - 1].key : k == begin ? none : cur) && inside(to))
                    old[u].load(static_cast<const D *>(a.dweight) + static_cast<long long>(p[u].key) * a.width + to);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (p[u].key == none) continue;
            if (p[u].key != cur) {   // the token's last row was the one before
                if (cur == none)
                    ;
                else if (here)
                    finish_row<T, D, VEC>(a, dst, at, sum, AHEAD && inside(at) ? &held : nullptr);
                else
                    store_partial<V>(partial_at<V>(partial, r, 0, windows, j), sum);
                cur = p[u].key;
                here = true;
                dst = static_cast<D *>(a.dweight) + static_cast<long long>(cur) * a.width;
                at = window_at(cur);
#pragma unroll
                for (int e = 0; e < V; ++e) sum[e] = 0.0f;
                if constexpr (AHEAD) held = old[u];
            }
            if constexpr (AHEAD)
                if (u == 0 && k == begin) held = old[0];
            float v[V];
            widen_vec<T>(join_window<T, VEC>(raw[u], dout + static_cast<long long>(p[u].at) * a.width, at, a.width), v);
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] += v[e];
        }
    }
    if (cur == none) return;
    if (here && (extend || after != cur))
        finish_row<T, D, VEC>(a, dst, at, sum, AHEAD && inside(at) ? &held : nullptr);
    else
        store_partial<V>(partial_at<V>(partial, r, here ? 1 : 0, windows, j), sum);
}

// The tokens that begin in a run and go on behind the next one: their partial
// sums, in kJoinParts contiguous parts that are then added up (one part: a token
// of a twelfth of 32768 rows took 20 us).  A CTA for each 32 runs and slice.
constexpr int kJoinParts = 4, kJoinRuns = 32;
template <class T, class D, bool VEC>
__global__ void __launch_bounds__(kSumThreads * kJoinParts)
    join_kernel(const EmbeddingArgs a, const Pair *pairs, const float *partial, int run, int runs, int slices,
                int ctas, const Fill fill) {
    constexpr int V = 16 / sizeof(T);
    wait_for_previous();
    if (static_cast<int>(blockIdx.x) >= ctas) {
        fill_rows<D, VEC, kSumThreads * kJoinParts>(a, fill, blockIdx.x - ctas);
        return;
    }
    __shared__ float4 parts[kJoinParts - 1][V / 4][kSumThreads];
    __shared__ unsigned int live_runs;
    const int part = threadIdx.x / kSumThreads, thread = threadIdx.x % kSumThreads;
    const int first_run = static_cast<int>(blockIdx.x) / slices * kJoinRuns;
    const int windows = windows_of<T>(a.width, VEC);
    const int j = static_cast<int>(blockIdx.x) % slices * kSumThreads + thread;
    const unsigned int none = a.vocab;
    if (threadIdx.x < 32) {
        const long long begin = (static_cast<long long>(first_run) + threadIdx.x) * run, end = begin + run;
        bool live = false;
        if (end + run < a.rows) {
            const unsigned int tail = pairs[end - 1].key, after = pairs[end].key;
            const unsigned int far = pairs[end + run].key, front = pairs[begin].key;
            const unsigned int prior = begin > 0 ? pairs[begin - 1].key : ~0u;
            live = tail != none && after == tail && far == tail && !(tail == front && prior == front);
        }
        const unsigned int mask = __ballot_sync(0xffffffffu, live);
        if (threadIdx.x == 0) live_runs = mask;
    }
    __syncthreads();
    for (unsigned int left = live_runs; left != 0; left &= left - 1) {
        const int r = first_run + __ffs(left) - 1;
        const unsigned int cur = pairs[(r + 1) * run - 1].key;
        // the run that the token ends in
        auto goes_past = [&](int q) {   // whether it fills run q to the end
            return q < runs && pairs[min((q + 1) * run, a.rows) - 1].key == cur;
        };
        int low = r + 2, step = 1;      // runs before `low` do not end it
        while (goes_past(low + step - 1)) {
            low += step;
            step *= 2;
        }
        int high = min(low + step - 1, runs - 1);   // ... and one up to `high` does
        while (low < high) {
            const int mid = low + (high - low) / 2;
            if (goes_past(mid))
                low = mid + 1;
            else
                high = mid;
        }
        // (a token that ends with its run is not in the next one, and has no piece there)
        const bool there = low < runs && pairs[low * run].key == cur;
        const int pieces = low - r - (there ? 0 : 1);   // besides the one that begins here
        const int from = r + 1 + static_cast<int>(static_cast<long long>(pieces) * part / kJoinParts);
        const int to = r + 1 + static_cast<int>(static_cast<long long>(pieces) * (part + 1) / kJoinParts);
        float sum[V] = {};
        if (j < windows) {
            if (part == 0) {
                const float *own = partial_at<V>(partial, r, 1, windows, j);
#pragma unroll
                for (int e = 0; e < V; ++e) sum[e] = own[e];
            }
#pragma unroll 4
            for (int q = from; q < to; ++q) {
                const float *p = partial_at<V>(partial, q, 0, windows, j);
#pragma unroll
                for (int e = 0; e < V; e += 4) {
                    const float4 t = *reinterpret_cast<const float4 *>(p + e);
                    sum[e] += t.x;
                    sum[e + 1] += t.y;
                    sum[e + 2] += t.z;
                    sum[e + 3] += t.w;
                }
            }
        }
        if (part > 0)
#pragma unroll
            for (int e = 0; e < V; e += 4)
                parts[part - 1][e / 4][thread] = make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
        __syncthreads();
        if (part == 0 && j < windows) {
#pragma unroll
            for (int q = 0; q < kJoinParts - 1; ++q)
#pragma unroll
                for (int e = 0; e < V; e += 4) {
                    const float4 t = parts[q][e / 4][thread];
                    sum[e] += t.x;
                    sum[e + 1] += t.y;
                    sum[e + 2] += t.z;
                    sum[e + 3] += t.w;
                }
            D *dst = static_cast<D *>(a.dweight) + static_cast<long long>(cur) * a.width;
            finish_row<T, D, VEC>(a, dst, j * V - (VEC ? 0 : window_phase(dst)), sum);
        }
        __syncthreads();
    }
}

// ---- gradient: launches -----------------------------------------------------------------

// Workspace: two lists of pairs, the digit counts, the partial sums.
struct Layout {
    size_t list, counts, present, partial, bytes;
};
Layout layout(int rows, int width, int vocab) {
    const SortPlan s = sort_plan(rows, vocab);
    const SumPlan m = sum_plan(rows, width, 8);
    auto round = [](size_t n) { return (n + 255) / 256 * 256; };
    Layout l;
    l.list = round(static_cast<size_t>(rows) * sizeof(Pair));
    l.counts = 2 * l.list;
    l.present = l.counts + round(static_cast<size_t>(s.passes) * s.tiles * (1u << s.bits) * sizeof(int));
    l.partial = l.present + round((static_cast<size_t>(vocab) + 31) / 32 * sizeof(int));
    // the most windows are those of an FP32 row of any alignment
    l.bytes = l.partial + round(static_cast<size_t>(m.runs) * 2 * (static_cast<size_t>(width) + 16) * sizeof(float));
    return l;
}

// A kernel of the chain, set up while the one before it runs.
template <class... P, class... A>
cudaError_t launch_next(void (*kernel)(P...), unsigned int grid, int threads, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

template <class D, bool VEC, int ITEMS>
cudaError_t launch_pass(const EmbeddingArgs &a, const SortPlan &s, int pass, const Pair *in, Pair *out,
                        int *counts, const Fill &fill, int fillers, cudaStream_t stream) {
    const size_t table = static_cast<size_t>(s.tiles) << s.bits;
    int *c = counts + pass * table;
    const auto kernel = pass == 0 ? scatter_kernel<D, VEC, ITEMS, true> : scatter_kernel<D, VEC, ITEMS, false>;
    return launch_next(kernel, s.tiles + fillers, kSortThreads, stream, a, in, out, c, c + table, s.bits,
                       pass * s.bits, pass == s.passes - 1, s.tiles, fill);
}

template <class T, class D, bool VEC>
cudaError_t launch_gradient(const EmbeddingArgs &a, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T), N = 16 / sizeof(D);
    const int windows = VEC ? a.width / V : (a.width + V - 1) / V + 1;
    if (few_rows(a.rows, a.width)) {
        if (!a.add) {
            const cudaError_t err = cudaMemsetAsync(
                a.dweight, 0, static_cast<size_t>(a.vocab) * a.width * sizeof(D), stream);
            if (err != cudaSuccess) return err;
        }
        const dim3 grid(a.rows, (windows + 31) / 32);
        if (a.rows <= kFewThreads)
            few_rows_kernel<T, D, VEC, 1><<<grid, kFewThreads, 0, stream>>>(a);
        else
            few_rows_kernel<T, D, VEC, 8><<<grid, kFewThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    const SortPlan s = sort_plan(a.rows, a.vocab);
    const SumPlan m = sum_plan(a.rows, a.width, V);
    const Layout l = layout(a.rows, a.width, a.vocab);
    char *ws = static_cast<char *>(a.ws);
    Pair *list[2] = {reinterpret_cast<Pair *>(ws), reinterpret_cast<Pair *>(ws + l.list)};
    int *counts = reinterpret_cast<int *>(ws + l.counts);
    unsigned int *present = a.add ? nullptr : reinterpret_cast<unsigned int *>(ws + l.present);
    float *partial = reinterpret_cast<float *>(ws + l.partial);
    cudaError_t err = cudaSuccess;
    if (present != nullptr) {
        err = cudaMemsetAsync(present, 0, (static_cast<size_t>(a.vocab) + 31) / 32 * sizeof(int), stream);
        if (err != cudaSuccess) return err;
    }
    const int passes = a.rows <= kMostRanked ? 0 : s.passes;
    if (passes == 0)
        rank_kernel<<<(a.rows + 31) / 32, kRankThreads, 0, stream>>>(a, list[0], present);
    else if (s.items == 2)
        digits_kernel<2><<<s.tiles, kSortThreads, 0, stream>>>(a, counts, present, s.bits, s.passes);
    else if (s.items == 4)
        digits_kernel<4><<<s.tiles, kSortThreads, 0, stream>>>(a, counts, present, s.bits, s.passes);
    else
        digits_kernel<16><<<s.tiles, kSortThreads, 0, stream>>>(a, counts, present, s.bits, s.passes);
    err = cudaGetLastError();
    // Fillers: CTAs of about 32 KB each, in the order of the rows (few CTAs that
    // went through all rows filled 1 GiB at 6.5 TB/s, these at 7.5).  A pass of
    // the sort and the join get what DRAM takes while they run, some 5 us, the
    // sums the rest.
    Fill fill = {present, 0, 0, 1, 8};
    const long long row_bytes = static_cast<long long>(a.width) * sizeof(D);
    const int fill_windows = VEC ? a.width / N : (a.width + N - 1) / N + 1;
    while (fill.lanes < kSumThreads && fill.lanes < fill_windows) fill.lanes *= 2;
    fill.each = 32768 / (fill_windows * 16) + kSumThreads * kJoinParts / fill.lanes;
    const long long rows = present != nullptr ? a.vocab : 0;
    long long share = (64ll << 20) / row_bytes + 1;
    if (share > rows / (passes + 2)) share = rows / (passes + 2);
    auto fillers = [&](long long to) {   // of the rows up to `to`
        fill.from = fill.to;
        fill.to = static_cast<int>(to);
        return (fill.to - fill.from + fill.each - 1) / fill.each;
    };
    for (int p = 0; p < passes && err == cudaSuccess; ++p) {
        const int n = fillers(share * (p + 1));
        const auto pass = s.items == 2 ? launch_pass<D, VEC, 2> : s.items == 4 ? launch_pass<D, VEC, 4> : launch_pass<D, VEC, 16>;
        err = pass(a, s, p, list[(p + 1) & 1], list[p & 1], counts, fill, n, stream);
    }
    if (err != cudaSuccess) return err;
    const Pair *sorted = list[passes == 0 ? 0 : (passes - 1) & 1];
    int lanes = 8;
    while (lanes < kSumThreads && lanes < windows) lanes *= 2;
    const int per = kSumThreads / lanes, slices = (windows + lanes - 1) / lanes;
    const int ctas = (m.runs + per - 1) / per * slices;
    const bool join = m.runs > 2;
    int n = fillers(join ? rows - share : rows);
    const auto sums = a.add ? sum_kernel<T, D, VEC, true> : sum_kernel<T, D, VEC, false>;
    err = launch_next(sums, ctas + n, kSumThreads, stream, a, sorted, partial, m.run, m.runs,
                      lanes, slices, ctas, fill);
    if (err != cudaSuccess || !join) return err;
    n = fillers(rows);
    const int join_slices = (windows + kSumThreads - 1) / kSumThreads;
    const int join_ctas = (m.runs + kJoinRuns - 1) / kJoinRuns * join_slices;
    return launch_next(join_kernel<T, D, VEC>, join_ctas + n, kSumThreads * kJoinParts, stream, a, sorted,
                       static_cast<const float *>(partial), m.run, m.runs, join_slices, join_ctas, fill);
}

template <class T, class D>
cudaError_t launch_gradient(bool vectors, const EmbeddingArgs &a, cudaStream_t stream) {
    return vectors ? launch_gradient<T, D, true>(a, stream) : launch_gradient<T, D, false>(a, stream);
}

}  // namespace

cudaError_t launch_embedding(int elem, bool vectors, EmbeddingArgs a, cudaStream_t stream) {
    cudaError_t err = cudaSuccess;
    a.status = status_address(&err);
    if (a.status == nullptr) return err;
    switch (elem) {
        case ELEM_F32:
            return vectors ? launch_lookup<float, true>(a, stream) : launch_lookup<float, false>(a, stream);
        case ELEM_BF16:
            return vectors ? launch_lookup<__nv_bfloat16, true>(a, stream)
                           : launch_lookup<__nv_bfloat16, false>(a, stream);
        default:
            return vectors ? launch_lookup<__half, true>(a, stream) : launch_lookup<__half, false>(a, stream);
    }
}

size_t embedding_backward_workspace(int rows, int width, int vocab) {
    return few_rows(rows, width) ? 0 : layout(rows, width, vocab).bytes;
}

cudaError_t launch_embedding_backward(int elem, int into, bool vectors, EmbeddingArgs a,
                                      cudaStream_t stream) {
    cudaError_t err = cudaSuccess;
    a.status = status_address(&err);
    if (a.status == nullptr) return err;
    switch (elem) {
        case ELEM_F32: return launch_gradient<float, float>(vectors, a, stream);
        case ELEM_BF16:
            return into == ELEM_F32 ? launch_gradient<__nv_bfloat16, float>(vectors, a, stream)
                                    : launch_gradient<__nv_bfloat16, __nv_bfloat16>(vectors, a, stream);
        default:
            return into == ELEM_F32 ? launch_gradient<__half, float>(vectors, a, stream)
                                    : launch_gradient<__half, __half>(vectors, a, stream);
    }
}

}  // namespace tile
