// Softmax cross entropy of a linear head, without keeping the logits.
//
//   l = x W^T,  lse = log sum_v exp(l_v),  loss = lse - l_target
//   g = (exp(l - lse) - onehot(target)) dloss,  dx = g W,  dW = g^T x
//
// Every product is a matrix product on the fifth-generation tensor cores
// with FP32 accumulators in tensor memory (gemm_kernel); what becomes of a
// 256 x 256 tile of it is the epilogue:
//
//   forward    a tile of l, without the targets' entries, is reduced to each
//              row's maximum and sum of exponentials, two numbers per tile
//              and row; a second kernel joins them with the target's logit, a
//              dot product of its own in FP32 FMAs:
//              loss = log(1 + sum_{v != target} exp(l_v - l_target)).
//              So a token that the head is sure of has a loss that keeps its
//              digits, and never one below 0, though a logit of the tensor
//              cores is off by more than it (logit_scale).
//   backward   in pieces of the vocabulary: l is computed again, turned into
//              g and kept in 16 bits for this piece only; then dW of the
//              piece's rows is g^T x, and g W is added to an FP32 dx.  At the
//              target g is expm1(l - lse) of an FP32 dot product again.
//
// Backward first packs the rows whose target counts (and whose dloss is not
// 0) to the front of a copy of x, so rows that are ignored cost nothing and
// a NaN in one of them reaches no gradient.  Forward does so where the
// product is long enough to pay for it.
#include "linear_ce.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "device_status.h"
#include "tcgen05.cuh"

TILE_DEVICE_STATUS(linear_ce)

namespace tile {
namespace {

enum { CE_WAIT_TIMEOUT = 2u, CE_BAD_TARGET = 8u };

constexpr int BM = 256, BN = 256, BK = 64;               // a CTA pair's tile
constexpr int CM = BM / 2;                               // a CTA's rows of it
constexpr int MOST_STAGES = 12;
constexpr int PIPE_BYTES = 192 << 10;                    // stages of A and B tiles
constexpr int EPI_WARPS = 8;                             // two for each 32 rows of a CTA's tile
constexpr int STORE_BYTES = EPI_WARPS * 4096;            // 32 rows x 128 bytes for each
constexpr int GEMM_SMEM = PIPE_BYTES + STORE_BYTES + 1024;   // + slack to align to 1024
constexpr int GEMM_THREADS = 32 * (EPI_WARPS + 2);       // and TMA, MMA
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

enum { EPI_NONE, EPI_LSE, EPI_GRAD, EPI_DWEIGHT, EPI_DX };

// What a call learns on the device before its products.
struct CeState {
    int valid;        // packed rows
    float unscale;    // what the scaled gradients are multiplied by at the end
};

// One product of a launch.
struct Job {
    int m, n, k;                // extents (rows of A, rows of B, reduction)
    int bn;                     // columns of a tile (256, or less to even out the CTAs)
    int a_rows;                 // rows of A that a CTA loads (fewer than 128 in a short call)
    int splits;                 // parts of k, each with its own slice of out (EPI_DX)
    int band;                   // tile rows that are gone down before the next column
    void *out;                  // EPI_DWEIGHT, EPI_DX
    long long ld;               // its elements per row
    int store;                  // EPI_DWEIGHT: through shared memory and map_out
};

struct GemmArgs {
    Job job[2];
    const CeState *state;       // limits the packed rows (m of GRAD and DX, k of DWEIGHT), or NULL
    float2 *partial;            // EPI_LSE: [m][2 n tiles], each half of a tile's columns
    const long long *target;    // EPI_LSE: the rows' targets where they are not packed
    // packed rows' target and, for EPI_GRAD, lse log2(e), p - 1 at the target
    // and scaled dloss
    const int *ptarget;
    const float *plse2, *pmiss, *pdloss;
    int n0;                     // first vocabulary entry of the piece
    int accumulate;             // EPI_DX: add to what is there
    long long slice;            // elements of a slice
    unsigned int *status;
};

struct GemmMaps {
    CUtensorMap a[2], b[2], out;
};

__device__ __forceinline__ unsigned int cluster_ctarank() {
    unsigned int r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// A logit is added up on the tensor cores in parts of PART_BLOCKS k blocks
// (4096 columns), joined in FP32 registers: what a sum loses grows with its
// steps, and ends there.  More and shorter parts lose less, but each stops the
// tensor cores for some 500 cycles (parts of 1024 columns: 4096 x 4096 x 131072
// BF16 4 % slower, 64 x 8192 x 65536 10 %, 7 % with 2048, 2 % with 4096).
constexpr int PART_BLOCKS = 64;

// log2(e), by which logits of the tensor cores are multiplied, with some of
// what they lost put back.  The tensor cores cut off as they add: each 16
// products added lose, of the sum so far, next to nothing where everything
// fits its 24 bits (few or small products), 2^-25 to 2^-24 in random rows
// (so 2^-26 to 2^-25 of a sum that grows evenly), and 2^-24 (BF16) to 2^-23
// (FP16) of it where all products have one sign, whose low bits are lost too.
// Put back is 2^-26 a step, the least that random rows lose: 4096 columns lost
// 3.9e-6 of a logit there and 256 2^-26 = 3.8e-6 are put back (the lse of 256
// rows over 32768 entries was 8.8e-6 too small, every row alike).  Sums that
// lose nothing come out that much too large.
__device__ __forceinline__ float logit_scale(int k_blocks) {
    return kLog2e * (1.0f + static_cast<float>(min(k_blocks, PART_BLOCKS) * (BK / 16)) * 0x1p-26f);
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// How an epilogue's product lies in memory: K-major operands are [m or n][k],
// MN-major ones [k][m or n].
__device__ __forceinline__ constexpr bool a_mn(int epi) { return epi == EPI_DWEIGHT; }
__device__ __forceinline__ constexpr bool b_mn(int epi) { return epi == EPI_DWEIGHT || epi == EPI_DX; }

// Tile t of a product: down the rows of a band of `band` tiles first, then
// along the columns, then the next band.  The band's A tiles stay in L2 while
// B streams by: 4096 rows of 4096 columns for the logits; for dx, whose
// operands are both long, about as many rows as columns at work at a time;
// for dW, whose A is the piece of g, as many tiles as keep about one round of
// pairs in a band, so that g is read from DRAM once.
struct Tile {
    int m, n, split;
};

// A divisor of tile numbers (below 2^30) with its reciprocal, for quotients in
// a dozen instructions: every role works out the place of every tile.
struct Divisor {
    int d;
    float inv;
};
__device__ __forceinline__ Divisor divisor(int d) {
    return Divisor{d, 1.0f / static_cast<float>(d)};
}
__device__ __forceinline__ int divide(int a, Divisor v, int &rest) {
    // the first estimate is off by up to a / d 2^-22 (256 at most), the
    // second by one
    int q = static_cast<int>(static_cast<float>(a) * v.inv);
    rest = a - q * v.d;
    const int more = static_cast<int>(floorf(static_cast<float>(rest) * v.inv));
    q += more;
    rest -= more * v.d;
    if (rest < 0) {
        rest += v.d;
        --q;
    } else if (rest >= v.d) {
        rest -= v.d;
        ++q;
    }
    return q;
}

// The tile grid of a job: `plane` tiles a split, in bands of `band` rows.
struct Raster {
    int band, bands;
    Divisor plane, band_tiles, high, last;   // tiles of a band; its rows, and the last band's
};
__device__ __forceinline__ Raster raster(int m_tiles, int n_tiles, int band) {
    Raster r;
    r.band = band;
    r.bands = (m_tiles + band - 1) / band;
    r.plane = divisor(max(1, m_tiles * n_tiles));
    r.band_tiles = divisor(max(1, band * n_tiles));
    r.high = divisor(band);
    r.last = divisor(max(1, m_tiles - (r.bands - 1) * band));
    return r;
}
__device__ __forceinline__ Tile tile_of(int t, const Raster &r) {
    Tile w;
    int rest;
    w.split = divide(t, r.plane, t);
    const int b = divide(t, r.band_tiles, rest);
    w.n = divide(rest, b == r.bands - 1 ? r.last : r.high, w.m);
    w.m += b * r.band;
    return w;
}

struct Extents {
    int m, n, k, m_tiles, n_tiles, k_blocks, splits, tiles;
};
template <int EPI>
__device__ __forceinline__ Extents extents(const Job &j, const CeState *state) {
    Extents e;
    e.m = j.m;
    e.n = j.n;
    e.k = j.k;
    if (state != nullptr) {
        // (a product that is not wanted has no rows)
        if (EPI == EPI_LSE || EPI == EPI_GRAD || EPI == EPI_DX) e.m = min(j.m, state->valid);
        if (EPI == EPI_DWEIGHT) e.k = state->valid;
    }
    e.m_tiles = (e.m + BM - 1) / BM;
    e.n_tiles = (e.n + j.bn - 1) / j.bn;
    e.k_blocks = (e.k + BK - 1) / BK;
    e.splits = EPI == EPI_DX ? j.splits : 1;
    e.tiles = EPI == EPI_NONE ? 0 : e.m_tiles * e.n_tiles * e.splits;
    return e;
}

// 32 rows x 64 columns (thread = row, `value` of column j) as 16-bit rows in
// memory, through this warp's part of shared memory and a tensor-map store
// (128-byte swizzled; whole lines whatever the row stride, and clipped at the
// matrix's edges).
template <bool BF16, class F>
__device__ __forceinline__ void store_64(const CUtensorMap *map, uint32_t buf, int lane, int row,
                                         int col, F value) {
    float v[64];
#pragma unroll
    for (int j = 0; j < 64; ++j) v[j] = value(j);
    if (lane == 0) store_wait_read<0>();   // the buffer's last store has read it
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 64; j += 8)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                         buf + lane * 128 + 16 * ((j / 8) ^ (lane & 7))),
                     "r"(pack2<BF16>(v[j], v[j + 1])), "r"(pack2<BF16>(v[j + 2], v[j + 3])),
                     "r"(pack2<BF16>(v[j + 4], v[j + 5])), "r"(pack2<BF16>(v[j + 6], v[j + 7]))
                     : "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
        tma_store(map, col, row, buf);
        store_commit();
    }
}
// A tile of FP32 accumulators so, 64 columns at a time; `value` maps column
// c + j's accumulator.
template <bool BF16, class F>
__device__ __forceinline__ void store_tile16(const CUtensorMap *map, uint32_t tmem, uint32_t buf,
                                             int lane, int row0, int col0, int from, int end,
                                             F value) {
    for (int c = from; c < end; c += 64) {
        float v[64];
        tmem_load64(tmem + c, v);
        store_64<BF16>(map, buf, lane, row0, col0 + c, [&](int j) { return value(v[j], c + j); });
    }
}

// The same for rows off the 16-byte grid, which tensor-map stores do not
// take: 32 rows x 64 columns through shared memory, then row by row, a warp
// writing one row's 64 elements as 4-byte words (and single elements at its
// ends where the row starts on an odd element).
template <bool BF16, class F>
__device__ __forceinline__ void store_rows16(unsigned short *out, long long ld, uint32_t tmem,
                                             uint32_t buf, int lane, int row0, int rows, int col0,
                                             int from, int end, F value) {
    for (int c = from; c < end; c += 64) {
        float v[64];
        tmem_load64(tmem + c, v);   // (its barrier: the rows before are out of the buffer)
#pragma unroll
        for (int j = 0; j < 64; j += 2)
            // word w of row r lies at word w ^ r of the row's 32
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(buf + lane * 128 + 4 * ((j / 2) ^ lane)),
                         "r"(pack2<BF16>(value(v[j]), value(v[j + 1])))
                         : "memory");
        __syncwarp();
        // without branches, so that the rows' shared-memory reads and shuffles
        // run side by side (row after row, 18 x 3356 x 68330 took 539 us)
        const int n = min(64, end - c), count = min(32, rows - row0);
        unsigned short *to = out + static_cast<long long>(row0) * ld + col0 + c;
#pragma unroll 8
        for (int r = 0; r < 32; ++r) {
            unsigned int w;
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(buf + r * 128 + 4 * (lane ^ r)));
            const unsigned int next = __shfl_down_sync(0xffffffffu, w, 1);
            unsigned short *at = to + r * ld;
            // on an odd element the words are elements 2 l + 1, 2 l + 2
            const int odd = (reinterpret_cast<uintptr_t>(at) >> 1) & 1;
            const int e = 2 * lane + odd;
            const unsigned int word = odd ? __funnelshift_r(w, next, 16) : w;
            if (r < count && e + 1 < n) *reinterpret_cast<unsigned int *>(at + e) = word;
            // the elements that no word holds: the first, and the last
            if (r < count && odd && lane == 0) at[0] = static_cast<unsigned short>(w);
            if (r < count && e + 1 == n) at[e] = static_cast<unsigned short>(word);
        }
    }
}

// C[m][n] = sum_k A[m][k] B[n][k] for one or two jobs, tile by tile on a
// persistent grid of CTA pairs: in each CTA a TMA warp fills a ring of A and
// B tiles in shared memory, one thread of the pair issues the MMAs into one of
// two accumulators in tensor memory (256 columns each), and eight warps turn
// the other into the epilogue's output.  A pair reads 32 KiB per CTA and 64
// columns of K from L2, where a CTA with a tile of its own reads 48, which bound
// the gradients' products with single CTAs (56 % of the tensor cores' time in
// use; with pairs L2 moves 17 TB/s there).  At 4096 tokens x 4096 columns
// x 32768 entries in BF16 the tensor cores work 95 % of the time for the
// logits (0.52 ms), 91 % for g (0.55 ms) and 88 % for dx and dW (1.15 ms): the
// clock under the power limit is what bounds long calls.  A few rows against a
// large weight are bound by reading it (5 x 2048 x 32768: 29 us, 20 at the
// rate of a copy); their backward reads it twice.
//
// With two jobs the tiles of the first come first; they are long (their
// reduction is the piece of the vocabulary) and few, 256 of them over 76
// pairs leave a sixth of the pairs' time.  So pairs that get one less of
// them start on the second job's short tiles while the others do their last
// long one, and all go on in turn from there (tile_at).
//
// PARTS: sums of more than PART_BLOCKS k blocks, one accumulator a part.
// WITHHELD (tests only): the first pair's first copies are not made, and waits
// are short.
template <int EPI0, int EPI1, bool BF16, bool PARTS, bool WITHHELD>
__device__ __forceinline__ void gemm(const GemmMaps &maps, const GemmArgs &g) {
    constexpr unsigned int SPINS = WITHHELD ? kTestBarSpins : kBarSpins;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * MOST_STAGES + 4];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (MOST_STAGES + s); };
    auto acc_full = [&](int s) { return bar0 + 8u * (2 * MOST_STAGES + s); };
    auto acc_empty = [&](int s) { return bar0 + 8u * (2 * MOST_STAGES + 2 + s); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    volatile int *aborted = &abort_flag;
    // a stage holds the larger job's tiles; A's part may be short (its last
    // rows are then what follows, and only rows that are not there read it)
    const int a_bytes = max(g.job[0].a_rows, EPI1 ? g.job[1].a_rows : 0) * BK * 2;
    const int stage_bytes = a_bytes + max(g.job[0].bn, EPI1 ? g.job[1].bn : 0) / 2 * BK * 2;
    const int stages = min(MOST_STAGES, PIPE_BYTES / stage_bytes);

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < stages; ++s) {
            bar_init(full(s), 1);      // rank 0's: its own arrival, both CTAs' bytes
            bar_init(empty(s), 1);     // the MMAs' commit
        }
        for (int s = 0; s < 2; ++s) {
            bar_init(acc_full(s), 1);
            bar_init(acc_empty(s), 2 * EPI_WARPS);   // rank 0's: both CTAs' epilogue warps
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&maps.a[0]);
        prefetch_map(&maps.b[0]);
    }
    if (warp == EPI_WARPS + 1) tmem_alloc(smem_u32(&tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *const_cast<volatile uint32_t *>(&tmem_slot);
    dependency_wait();
    dependency_launch();

    const Extents e0 = extents<EPI0>(g.job[0], g.state);
    const Extents e1 = extents<EPI1>(g.job[EPI1 ? 1 : 0], g.state);
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    // The i-th tile of this pair, or -1.  The first job's tiles go round the
    // pairs; its last round serves `last` of them, and the others do `ahead`
    // tiles of the second job in that time.
    const int rounds = e0.tiles / pairs, last = e0.tiles % pairs;
    // (a short tile of few k blocks takes as long as its output's way to
    // memory, about that of 6: 128 KiB of a pair's share of 6.8 TB/s)
    const int cost = max(e1.k_blocks, 6);
    const int ahead = EPI1 && last > 0 ? (e0.k_blocks / e0.splits + cost / 2) / cost : 0;
    auto tile_at = [&](int i) {
        if (i < rounds || (i == rounds && pair < last)) return i * pairs + pair;
        if (!EPI1) return -1;
        int j = i - rounds;   // tiles of the second job before this one, counted
        long long t;          // as if the pairs with a last long tile did `ahead` short ones
        if (pair < last) j += ahead - 1;
        if (j < ahead)
            t = static_cast<long long>(j) * (pairs - last) + pair - last;
        else
            t = static_cast<long long>(ahead) * (pairs - last) +
                static_cast<long long>(j - ahead) * pairs +
                (pair < last ? pair + pairs - last : pair - last);
        return t < e1.tiles ? static_cast<int>(e0.tiles + t) : -1;
    };
    const Raster r0 = raster(e0.m_tiles, e0.n_tiles, g.job[0].band);
    const Raster r1 = raster(e1.m_tiles, e1.n_tiles, g.job[EPI1 ? 1 : 0].band);
    // f(job, tile, first and last k block) for tile t, the job's number as a
    // constant: what f reads of the launch's arguments is then at fixed places
    // (looked up by a variable, and with the scale read again for every tile,
    // the epilogue of a short tile took 4850 cycles, 2200 of them for that)
    auto on_tile = [&](int t, auto f) {
        if constexpr (EPI1 != EPI_NONE)
            if (t >= e0.tiles) {
                f(std::integral_constant<int, 1>{}, tile_of(t - e0.tiles, r1), 0, e1.k_blocks);
                return;
            }
        const Tile w = tile_of(t, r0);
        int kb0 = 0, kb1 = e0.k_blocks;
        if (EPI0 == EPI_DX) {
            kb0 = static_cast<int>(static_cast<long long>(e0.k_blocks) * w.split / e0.splits);
            kb1 = static_cast<int>(static_cast<long long>(e0.k_blocks) * (w.split + 1) / e0.splits);
        }
        f(std::integral_constant<int, 0>{}, w, kb0, kb1);
    };

    if (warp == EPI_WARPS && lane == 0) {   // TMA producer
        int stage = 0;
        unsigned int phase = 0;
        long long issued = 0;
        bool ok = true;
        int t;
        for (int i = 0; ok && (t = tile_at(i)) >= 0; ++i) {
            on_tile(t, [&](auto j, Tile w, int kb0, int kb1) {
                constexpr int J = decltype(j)::value, EPI = J ? EPI1 : EPI0;
                const Job &job = g.job[J];
                const int half = job.bn / 2;
                const int m0 = w.m * BM + rank * CM, n0 = w.n * job.bn + rank * half;
                const unsigned int bytes = (job.a_rows + half) * BK * 2;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!(ok = bar_wait<SPINS>(empty(stage), phase ^ 1u, aborted, g.status,
                                               CE_WAIT_TIMEOUT)))
                        break;
                    const uint32_t a = base + stage * stage_bytes, b = a + a_bytes;
                    const uint32_t bar = peer_addr(full(stage), 0);
                    if (!WITHHELD || issued > 0 || pair > 0) {
                        if (rank == 0) bar_expect_tx(full(stage), 2 * bytes);
                        if (a_mn(EPI)) {
                            tma_load(a, &maps.a[J], m0, kb * BK, bar);
                            tma_load(a + 8192, &maps.a[J], m0 + 64, kb * BK, bar);
                        } else {
                            tma_load(a, &maps.a[J], kb * BK, m0, bar);
                        }
                        if (b_mn(EPI)) {   // (256 columns to a tile)
                            tma_load(b, &maps.b[J], n0, kb * BK, bar);
                            tma_load(b + 8192, &maps.b[J], n0 + 64, kb * BK, bar);
                        } else {
                            tma_load(b, &maps.b[J], kb * BK, n0, bar);
                        }
                    }
                    ++issued;
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            });
        }
        // An aborted pair waits (bounded) for the copies it issued: none may
        // land in shared memory that it no longer owns.
        if (*aborted && rank == 0)
            for (long long i = issued > stages ? issued - stages : 0; i < issued; ++i)
                for (unsigned int n = 0; n < SPINS; ++n)
                    if (bar_test(full(static_cast<int>(i % stages)), (i / stages) & 1)) break;
    } else if (warp == EPI_WARPS + 1 && lane == 0 && rank == 0) {   // MMA issuer
        int stage = 0, acc = 0;
        unsigned int phase = 0, acc_phase = 0;
        bool ok = true;
        int t;
        for (int i = 0; ok && (t = tile_at(i)) >= 0; ++i) {
            on_tile(t, [&](auto j, Tile, int kb0, int kb1) {
                constexpr int J = decltype(j)::value, EPI = J ? EPI1 : EPI0;
                const uint32_t idesc = mma_idesc(BF16, a_mn(EPI), b_mn(EPI), BM, g.job[J].bn);
                int kb = kb0;
                do {   // the whole sum, or a part of it
                    if (!(ok = bar_wait<SPINS>(acc_empty(acc), acc_phase ^ 1u, aborted, g.status,
                                               CE_WAIT_TIMEOUT)))
                        return;
                    tc_fence_after();
                    const uint32_t d = tmem + acc * BN;
                    const int end = PARTS ? min(kb1, kb + PART_BLOCKS) : kb1;
                    bool first = true;
                    for (; kb < end; ++kb) {
                        if (!(ok = bar_wait<SPINS>(full(stage), phase, aborted, g.status,
                                                   CE_WAIT_TIMEOUT)))
                            break;
                        tc_fence_after();
                        const uint32_t a = base + stage * stage_bytes, b = a + a_bytes;
                        const uint64_t da = smem_desc(a, a_mn(EPI) ? 8192 : 16, 1024);
                        const uint64_t db = smem_desc(b, b_mn(EPI) ? 8192 : 16, 1024);
#pragma unroll
                        for (int k = 0; k < BK / 16; ++k) {
                            // 16 elements along K: 32 bytes of a K-major row, or
                            // 16 rows of 128 bytes
                            tc_mma(d, da + k * (a_mn(EPI) ? 2048 >> 4 : 32 >> 4),
                                   db + k * (b_mn(EPI) ? 2048 >> 4 : 32 >> 4), idesc, !first);
                            first = false;
                        }
                        tc_commit(empty(stage));
                        if (++stage == stages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    tc_commit(acc_full(acc));
                    acc ^= 1;
                    if (acc == 0) acc_phase ^= 1u;
                } while (PARTS && ok && kb < kb1);
            });
        }
        if (*aborted) {   // wait (bounded) until no MMA touches the pair's memory
            tc_commit(acc_full(acc));
            for (unsigned int n = 0; n < SPINS; ++n)
                if (bar_test(acc_full(acc), acc_phase)) break;
        }
    } else if (warp < EPI_WARPS) {
        // epilogue: thread = row of the tile; warps w and w + 4 share 32 rows
        // (a warp reads the quarter of tensor memory's lanes of its number
        // modulo 4) and take half of the columns each
        int acc = 0;
        unsigned int acc_phase = 0;
        const uint32_t buf = base + PIPE_BYTES + warp * 4096;
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t drained0 = peer_addr(acc_empty(0), 0), drained1 = peer_addr(acc_empty(1), 0);
        const float unscale = EPI1 == EPI_DWEIGHT ? g.state->unscale : 1.0f;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        // whether the accumulator that is due has come
        auto ready = [&] {
            const bool in =
                __all_sync(0xffffffffu, bar_wait<SPINS>(acc_full(acc), acc_phase, aborted, g.status,
                                                        CE_WAIT_TIMEOUT));
            if (in) tc_fence_after();
            return in;
        };
        auto drained = [&] {   // this warp has read it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive_peer(acc ? drained1 : drained0);
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        };
        int t;
        for (int i = 0; (t = tile_at(i)) >= 0; ++i) {
            bool ok = true;
            on_tile(t, [&](auto j, Tile w, int kb0, int kb1) {
                constexpr int J = decltype(j)::value, EPI = J ? EPI1 : EPI0;
                const Job &job = g.job[J];
                const Extents &e = J ? e1 : e0;
                const int row0 = w.m * BM + rank * CM + quarter * 32, row = row0 + lane;
                const int col0 = w.n * job.bn;
                int skip = -1;   // the tile's column that this row leaves out
                if (EPI == EPI_LSE && row < e.m) {
                    const long long t = g.ptarget != nullptr ? g.ptarget[row] : g.target[row];
                    if (t >= col0 && t < e.n) skip = static_cast<int>(t) - col0;
                }
                // this warp's columns of the tile: [from, to), and those that exist
                const int from = half * (job.bn / 2), to = from + job.bn / 2;
                const int end = min(to, e.n - col0);
                float sum[PARTS ? BN / 2 : 1];   // this row's logits, part after part
                if constexpr (PARTS) {
#pragma unroll
                    for (int j = 0; j < BN / 2; ++j) sum[j] = 0.0f;
                    for (int kb = kb0;; kb += PART_BLOCKS) {
                        if (!(ok = ready())) return;
                        const uint32_t d = tmem + acc * BN + lanes + from;
                        if (row0 < e.m)
#pragma unroll
                            for (int j = 0; j < BN / 2; j += 16)
                                if (from + j < end) tmem_add16(d + j, sum + j);
                        if (kb + PART_BLOCKS >= kb1) break;
                        drained();
                    }
                } else {
                    if (!(ok = ready())) return;
                }
                const uint32_t d = tmem + acc * BN + lanes;
                const bool none = kb0 == kb1;   // no product was made: zero
                // rows of this warp that are looked at: those that are there, and
                // for g those up to the next 64, which dW's reduction reads
                if (row0 >= (EPI == EPI_GRAD ? (e.m + BK - 1) / BK * BK : e.m)) return;
                if constexpr (EPI == EPI_LSE) {
                    // the maximum and the sum over exponents of 2
                    const float scale = logit_scale(e.k_blocks);
                    float m = -INFINITY, s = 0.0f;
                    auto chunk = [&](int c, float (&v)[32]) {
                        const int limit = end - c;
                        if (limit < 32)
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (j >= limit) v[j] = -INFINITY;
                        const int hit = skip - c;
                        if (__any_sync(0xffffffffu, hit >= 0 && hit < 32))
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (j == hit) v[j] = -INFINITY;
                        float top = v[0];
#pragma unroll
                        for (int j = 1; j < 32; ++j) top = fmaxf(top, v[j]);
                        top = fmaxf(m, top * scale);
                        const float ref = top == -INFINITY ? 0.0f : top;
                        s *= ex2(m - ref);
                        float part[4] = {};
#pragma unroll
                        for (int j = 0; j < 32; ++j) part[j & 3] += ex2(fmaf(v[j], scale, -ref));
                        s += (part[0] + part[1]) + (part[2] + part[3]);
                        m = top;
                    };
                    if constexpr (PARTS) {
#pragma unroll
                        for (int j = 0; j < BN / 2; j += 32)
                            if (from + j < end) chunk(from + j, *reinterpret_cast<float (*)[32]>(sum + j));
                    } else {
                        for (int c = from; c < end; c += 32) {
                            float v[32];
                            tmem_load32(d + c, v);
                            chunk(c, v);
                        }
                    }
                    if (row < e.m)
                        g.partial[(static_cast<long long>(row) * e.n_tiles + w.n) * 2 + half] =
                            make_float2(m, s);
                } else if constexpr (EPI == EPI_GRAD) {
                    const bool in = row < e.m;
                    const int want = in ? g.ptarget[row] - g.n0 - col0 : -1;
                    const float lse2 = in ? g.plse2[row] : 0.0f, dl = in ? g.pdloss[row] : 0.0f;
                    const float miss = in ? g.pmiss[row] : 0.0f;
                    const float scale = logit_scale(e.k_blocks);
                    const int limit = in ? e.n - col0 : 0;
                    auto grad = [&](float v, int c) {
                        const float p = ex2(fmaf(v, scale, -lse2));
                        return c < limit ? (want == c ? miss : p) * dl : 0.0f;
                    };
                    if constexpr (PARTS) {
#pragma unroll
                        for (int h = 0; h < BN / 2; h += 64)
                            store_64<BF16>(&maps.out, buf, lane, row0, col0 + from + h, [&](int j) {
                                return grad(sum[h + j], from + h + j);
                            });
                    } else {
                        store_tile16<BF16>(&maps.out, d, buf, lane, row0, col0, from, to, grad);
                    }
                } else if constexpr (EPI == EPI_DWEIGHT) {
                    const float f = unscale;
                    if (job.store) {
                        store_tile16<BF16>(&maps.out, d, buf, lane, row0, col0, from, end,
                                           [&](float v, int) { return none ? 0.0f : v * f; });
                    } else {
                        store_rows16<BF16>(static_cast<unsigned short *>(job.out), job.ld, d, buf, lane,
                                           row0, e.m, col0, from, end,
                                           [&](float v) { return none ? 0.0f : v * f; });
                    }
                } else if constexpr (EPI == EPI_DX) {   // FP32, ld a multiple of 4: rows of whole vectors
                    float *out = static_cast<float *>(job.out) + w.split * g.slice +
                                 static_cast<long long>(row) * job.ld + col0;
                    for (int c = from; c < to && col0 + c < job.ld; c += 32) {
                        float v[32];
                        tmem_load32(d + c, v);
                        if (row < e.m)
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                if (col0 + c + j >= job.ld) break;
                                float4 q = none ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                                                : make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                                float4 *p = reinterpret_cast<float4 *>(out + c + j);
                                if (g.accumulate) {
                                    const float4 o = *p;
                                    q = make_float4(q.x + o.x, q.y + o.y, q.z + o.z, q.w + o.w);
                                }
                                *p = q;
                            }
                    }
                }
            });
            if (!ok) break;
            drained();
        }
        if (lane == 0) store_wait<0>();   // the stores are written before the CTA ends
    }
    // (after an abort: and the copies that the producer's wait does not count, of
    // a stage that only one CTA of the pair has issued: 0.1 ms, they take 1 us)
    if (*aborted)
        for (int i = 0; i < 100; ++i) __nanosleep(1000);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // neither CTA leaves while the other uses its memory
    tc_fence_after();
    if (warp == EPI_WARPS + 1) tmem_free(tmem, 512);
}

template <int EPI0, int EPI1, bool BF16>
__global__ void __launch_bounds__(GEMM_THREADS, 1)
    gemm_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmArgs g) {
    gemm<EPI0, EPI1, BF16, false, false>(maps, g);
}
__global__ void __launch_bounds__(GEMM_THREADS, 1)
    gemm_withheld_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmArgs g) {
    gemm<EPI_LSE, EPI_NONE, true, false, true>(maps, g);
}
// 16 registers fewer than 320 threads could have leave room for a CTA of the
// next kernel beside this one, whose dot products (join_lse_kernel) then run
// under these products (1024 x 16384 x 16384 BF16 345 us, 372 us without).
template <int EPI, bool BF16>
__global__ void __maxnreg__(152)
    gemm_parts_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmArgs g) {
    gemm<EPI, EPI_NONE, BF16, true, false>(maps, g);
}

// ---- a row's own logit -----------------------------------------------------------------

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

// ---- packing rows ----------------------------------------------------------------------

struct PackArgs {
    const unsigned short *x, *weight;
    const long long *target;
    const float *lse, *dloss;           // NULL in a forward call
    long long ignore;
    int rows, width, vocab, ld;
    int bf16;                           // FP16: gradients are scaled by 2^15
    int row_ctas;                       // CTAs that pack x; the others copy the weight (to pw)
    int cta_rows;                       // rows of a CTA that packs x
    unsigned short *px, *pw;
    CeState *state;
    int *place, *ptarget;
    float *plse2, *pmiss, *pdloss;
    unsigned int *status;
};

__device__ __forceinline__ bool counts(long long t, long long ignore, int vocab, float dl) {
    return t != ignore && t >= 0 && t < vocab && dl != 0.0f;
}

// `lanes` neighbours (8, 16 or 32) copy a row of `width` two-byte elements, from any 2-byte
// alignment, to a row of `ld` (a multiple of 8; 16-byte aligned), padded with
// zeros; `from` NULL: zeros.  Two aligned source blocks make one of the
// target's; the second is the next lane's first.
__device__ __forceinline__ void copy_row16(const unsigned short *from, unsigned short *to, int width,
                                           int ld, int lanes) {
    const int lane = threadIdx.x & (lanes - 1);
    // the next lane of this row, the first after the last
    const int beside = (threadIdx.x & 31 & ~(lanes - 1)) | ((lane + 1) & (lanes - 1));
    const int vecs = ld / 8;
    uint4 *out = reinterpret_cast<uint4 *>(to);
    if (from == nullptr) {
        for (int i = lane; i < vecs; i += lanes) out[i] = make_uint4(0, 0, 0, 0);
        return;
    }
    if (width % 8 == 0 && (reinterpret_cast<uintptr_t>(from) & 15) == 0) {
        const uint4 *in = reinterpret_cast<const uint4 *>(from);
#pragma unroll 4
        for (int i = lane; i < vecs; i += lanes)
            out[i] = i < width / 8 ? __ldg(in + i) : make_uint4(0, 0, 0, 0);
        return;
    }
    const uintptr_t begin = reinterpret_cast<uintptr_t>(from);
    const uintptr_t end = begin + static_cast<uintptr_t>(width) * 2;
    const int skew = static_cast<int>(begin & 15);
    const uintptr_t block0 = begin - skew;
    // a block with bytes outside the row is read by element
    auto block = [&](int b) {
        const uintptr_t at = block0 + static_cast<uintptr_t>(b) * 16;
        if (at >= begin && at + 16 <= end) return __ldg(reinterpret_cast<const uint4 *>(at));
        unsigned int w[4] = {};
        if (at < end)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uintptr_t p = at + 2 * j;
                if (p >= begin && p < end)
                    w[j / 2] |= static_cast<unsigned int>(
                                    *reinterpret_cast<const unsigned short *>(p)) << (16 * (j & 1));
            }
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    const int words = skew >> 2, bits = (skew & 3) * 8;
    for (int i0 = 0; i0 < vecs; i0 += 4 * lanes) {
        uint4 a[5];   // the loads of four rounds at once
#pragma unroll
        for (int u = 0; u < 4; ++u) a[u] = block(i0 + u * lanes + lane);
        // the block after these, for the last lane
        a[4] = block(i0 + 4 * lanes);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            // the next lane's block; for the last lane the first of the next round
            uint4 b;
            b.x = __shfl_sync(0xffffffffu, lane == 0 ? a[u + 1].x : a[u].x, beside);
            b.y = __shfl_sync(0xffffffffu, lane == 0 ? a[u + 1].y : a[u].y, beside);
            b.z = __shfl_sync(0xffffffffu, lane == 0 ? a[u + 1].z : a[u].z, beside);
            b.w = __shfl_sync(0xffffffffu, lane == 0 ? a[u + 1].w : a[u].w, beside);
            // bytes [skew, skew + 16) of a, b: words moved by `words`, in two steps
            unsigned int w[8] = {a[u].x, a[u].y, a[u].z, a[u].w, b.x, b.y, b.z, b.w};
            if (words & 1)
#pragma unroll
                for (int j = 0; j < 7; ++j) w[j] = w[j + 1];
            if (words & 2)
#pragma unroll
                for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
            const int i = i0 + u * lanes + lane;
            if (i < vecs)
                out[i] = make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
        }
    }
}

// The rows that count, packed to the front of px in their order (place[i] =
// position of row i or -1; target, lse and dloss by position), rows
// behind them zero; and the weight's rows copied to whole vectors.  A CTA
// packs a few rows and counts the rows before them for itself (the targets of a
// call are small and in L2), so there is no pass before it.
//
// dloss is held over its largest magnitude: the equal weights of a mean
// become 1, so that the 16-bit gradients round p - onehot and not its
// product with, say, 1 / 48, which is off by the same 2^-9 in every row's
// largest entry (dx of 48 rows was 2.6e-3 off in the 2-norm with dloss in
// it, 1.8e-3 without; the output's own rounding is 1.7e-3).  FP16 gradients
// are scaled by 2^15 too: |p - onehot| <= 1, so nothing overflows, and what
// underflows is below 2^-40 of the largest.
__global__ void __launch_bounds__(256) pack_rows_kernel(const PackArgs a) {
    __shared__ int warp_before[8], warp_total[8], row_at[32];
    __shared__ float warp_top[8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    dependency_launch();
    if (static_cast<int>(blockIdx.x) >= a.row_ctas) {
        const int ctas = gridDim.x - a.row_ctas, cta = blockIdx.x - a.row_ctas;
        // short rows two or four to a warp, so that its loads fill a round
        const int lanes = a.ld > 512 ? 32 : a.ld > 256 ? 16 : 8, each = 32 / lanes;
        for (long long r0 = (static_cast<long long>(cta) * 8 + warp) * each; r0 < a.vocab;
             r0 += ctas * 8ll * each) {
            // (behind the last row: that row once more)
            const long long r = min(static_cast<long long>(a.vocab) - 1, r0 + lane / lanes);
            copy_row16(a.weight + r * a.width, a.pw + r * a.ld, a.width, a.ld, lanes);
        }
        return;
    }
    const int r0 = blockIdx.x * a.cta_rows, r1 = min(a.rows, r0 + a.cta_rows);
    int before = 0, valid = 0;   // packed rows before this CTA's, and all of them
    float top = 0.0f;
#pragma unroll 4
    for (int i = tid; i < a.rows; i += 256) {
        const long long t = a.target[i];
        const float dl = a.dloss != nullptr ? a.dloss[i] : 1.0f;
        const bool in = counts(t, a.ignore, a.vocab, dl);
        valid += in;
        before += in && i < r0;
        if (in && isfinite(dl)) top = fmaxf(top, fabsf(dl));
    }
    for (int d = 16; d > 0; d >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, d);
        valid += __shfl_xor_sync(0xffffffffu, valid, d);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    }
    if (lane == 0) {
        warp_before[warp] = before;
        warp_total[warp] = valid;
        warp_top[warp] = top;
    }
    __syncthreads();
    before = valid = 0;
    top = 0.0f;
    for (int i = 0; i < 8; ++i) {
        before += warp_before[i];
        valid += warp_total[i];
        top = fmaxf(top, warp_top[i]);
    }
    // 32768 / top and top / 32768 are finite and not 0 for any normal top
    top = fminf(fmaxf(top, 1e-30f), 1e30f);
    const float full = a.bf16 ? 1.0f : 32768.0f;
    if (blockIdx.x == 0 && tid == 0) {
        a.state->valid = valid;
        a.state->unscale = top / full;
    }
    for (int c = r0; c < r1; c += 32) {   // up to 32 rows at a time, a lane of warp 0 each
        if (warp == 0) {
            const int i = c + lane;
            const bool mine = i < r1;
            const long long t = mine ? a.target[i] : a.ignore;
            const float dl = mine && a.dloss != nullptr ? a.dloss[i] : 1.0f;
            const bool in = mine && counts(t, a.ignore, a.vocab, dl);
            const unsigned int mask = __ballot_sync(0xffffffffu, in);
            const int at = before + __popc(mask & ((1u << lane) - 1u));
            before += __popc(mask);
            row_at[lane] = in ? at : -1;
            if (mine) {
                a.place[i] = in ? at : -1;
                if (t != a.ignore && (t < 0 || t >= a.vocab)) atomicOr(a.status, CE_BAD_TARGET);
            }
            if (in) a.ptarget[at] = static_cast<int>(t);
            if (in && a.dloss != nullptr) {
                a.plse2[at] = a.lse[i] * kLog2e;
                a.pdloss[at] = full * (dl / top);
            }
        }
        __syncthreads();
        for (int q = warp; q < 32; q += 8) {
            const int i = c + q, at = row_at[q];
            if (i >= r1) break;
            const unsigned short *x = a.x + static_cast<long long>(i) * a.width;
            if (at >= 0)
                copy_row16(x, a.px + static_cast<long long>(at) * a.ld, a.width, a.ld, 32);
            if (at >= 0 && a.dloss != nullptr) {
                const unsigned short *w = a.weight + a.target[i] * a.width;
                const float l = a.bf16 ? warp_dot<__nv_bfloat16>(x, w, a.width, lane)
                                       : warp_dot<__half>(x, w, a.width, lane);
                if (lane == 0) a.pmiss[at] = expm1f(l - a.lse[i]);
            }
            if (i >= valid)
                copy_row16(nullptr, a.px + static_cast<long long>(i) * a.ld, 0, a.ld, 32);
        }
        __syncthreads();
    }
}

// ---- forward: joining the tiles --------------------------------------------------

struct JoinArgs {
    const float2 *partial;              // exponents of 2
    const unsigned short *x, *weight;   // as they were multiplied
    long long x_ld, weight_ld;
    const long long *target;
    const int *place;   // where a row was packed, or NULL
    long long ignore;
    int rows, width, vocab, partials;
    float *loss, *lse;
    unsigned int *status;
};

// One warp a row: lanes over the half tiles, joined in a fixed tree.
template <class T>
__global__ void __launch_bounds__(128) join_lse_kernel(const JoinArgs a) {
    const int row = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (row >= a.rows) return;
    // The target's logit needs nothing of the product before, only what that
    // waited for before it let this kernel start.
    const long long t = a.target[row];
    const bool in = t >= 0 && t < a.vocab;
    const int at = a.place != nullptr ? a.place[row] : row;
    const float l = in && t != a.ignore ? warp_dot<T>(a.x + at * a.x_ld, a.weight + t * a.weight_ld,
                                                      a.width, lane)
                                        : NAN;
    dependency_wait();
    if (t == a.ignore) {
        if (lane == 0) a.loss[row] = a.lse[row] = 0.0f;
        return;
    }
    if (!in) {   // not among the rows that were multiplied, or of no use there
        if (lane == 0) {
            a.loss[row] = NAN;
            a.lse[row] = 0.0f;
            atomicOr(a.status, CE_BAD_TARGET);
        }
        return;
    }
    const float2 *p = a.partial + static_cast<long long>(at) * a.partials;
    float m = -INFINITY;
    for (int i = lane; i < a.partials; i += 32) m = fmaxf(m, p[i].x);
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float ref = m == -INFINITY ? 0.0f : m;
    float s = 0.0f;   // sum over the other entries of 2^(l_v log2(e) - ref)
    for (int i = lane; i < a.partials; i += 32) {
        const float2 q = p[i];
        s += q.y * exp2f(q.x - ref);
    }
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane != 0) return;
    // log(1 + sum exp(l_v - l)), from the larger of the two exponents; the
    // first where there is no other entry (or none above -infinity: s is 0)
    const float d = fmaf(l, kLog2e, -m);
    if (!(d < 0.0f)) {
        const float log_s = log1pf(s == 0.0f ? 0.0f : s * exp2f(-d));
        a.lse[row] = l + log_s;
        a.loss[row] = (l - l) + log_s;   // (NaN for an infinite logit)
    } else {
        const float log_s = log2f(s + exp2f(d));
        a.lse[row] = kLn2 * (ref + log_s);
        a.loss[row] = kLn2 * (log_s - d);
    }
}

// ---- backward: the end ----------------------------------------------------------------

// dx[i] = the sum of the slices' rows place[i], scaled back and rounded; 0
// for rows that do not count.  A CTA does 512 columns of a row, its slices'
// loads 16 at a time.
constexpr int FINISH_COLS = 512;

template <class T>
__global__ void __launch_bounds__(FINISH_COLS / 4)
    finish_dx_kernel(const float *acc, int splits, long long slice, int acc_ld, const int *place,
                     const CeState *state, T *dx, int width) {
    dependency_wait();
    const int chunks = (width + FINISH_COLS - 1) / FINISH_COLS;
    const long long r = blockIdx.x / chunks;
    const int c = static_cast<int>(blockIdx.x % chunks) * FINISH_COLS + threadIdx.x * 4;
    if (c >= width) return;
    const int p = place[r];
    const float f = state->unscale;
    float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (p >= 0) {
        const float *from = acc + static_cast<long long>(p) * acc_ld + c;
        for (int s = 0; s < splits; s += 16) {
            float4 q[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (s + i < splits) q[i] = __ldcs(reinterpret_cast<const float4 *>(from + (s + i) * slice));
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (s + i < splits)
                    t = make_float4(t.x + q[i].x, t.y + q[i].y, t.z + q[i].z, t.w + q[i].w);
        }
    }
    T *to = dx + r * width;
    constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
    const uint32_t lo = pack2<BF16>(t.x * f, t.y * f), hi = pack2<BF16>(t.z * f, t.w * f);
    if (width % 4 == 0 && (reinterpret_cast<uintptr_t>(dx) & 7) == 0) {
        *reinterpret_cast<uint2 *>(to + c) = make_uint2(lo, hi);
    } else {
        unsigned short *o = reinterpret_cast<unsigned short *>(to);
        o[c] = static_cast<unsigned short>(lo);
        if (c + 1 < width) o[c + 1] = static_cast<unsigned short>(lo >> 16);
        if (c + 2 < width) o[c + 2] = static_cast<unsigned short>(hi);
        if (c + 3 < width) o[c + 3] = static_cast<unsigned short>(hi >> 16);
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

// A launch that may start before the kernel before it has ended (that kernel
// lets it, and it waits itself).
template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), unsigned grid, unsigned cluster, unsigned block,
                             size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

long long job_tiles(const Job &j) { return up(j.m, BM) / BM * (up(j.n, j.bn) / j.bn) * j.splits; }

template <class Kernel>
cudaError_t launch_gemm_kernel(Kernel kernel, std::atomic<int> (&ready)[kMaxDevices],
                               const GemmMaps &maps, const GemmArgs &g, long long tiles,
                               cudaStream_t stream) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (ready[dev].load(std::memory_order_acquire) == 0) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, GEMM_SMEM);
        if (err != cudaSuccess) return err;
        ready[dev].store(1, std::memory_order_release);
    }
    if (tiles > 0x3fffffff) return cudaErrorInvalidValue;   // tile numbers are ints
    long long pairs = sm_count_of_device() / 2;
    if (pairs > tiles) pairs = tiles;
    if (pairs < 1) pairs = 1;
    return launch_dependent(kernel, static_cast<unsigned>(2 * pairs), 2, GEMM_THREADS, GEMM_SMEM,
                            stream, maps, g);
}
template <int EPI0, int EPI1, bool BF16>
cudaError_t launch_gemm_typed(const GemmMaps &maps, const GemmArgs &g, cudaStream_t stream) {
    static std::atomic<int> ready[2][kMaxDevices];
    const long long tiles = job_tiles(g.job[0]) + (EPI1 ? job_tiles(g.job[1]) : 0);
    if constexpr (EPI0 == EPI_LSE || EPI0 == EPI_GRAD)
        if (g.job[0].k > PART_BLOCKS * BK)
            return launch_gemm_kernel(gemm_parts_kernel<EPI0, BF16>, ready[1], maps, g, tiles,
                                      stream);
    return launch_gemm_kernel(gemm_kernel<EPI0, EPI1, BF16>, ready[0], maps, g, tiles, stream);
}
template <int EPI0, int EPI1>
cudaError_t launch_gemm(int bf16, const GemmMaps &maps, const GemmArgs &g, cudaStream_t stream) {
    return bf16 ? launch_gemm_typed<EPI0, EPI1, true>(maps, g, stream)
                : launch_gemm_typed<EPI0, EPI1, false>(maps, g, stream);
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

// Rows of an odd width are copied (TMA wants strides of 16 bytes), and copies
// have rows of whole 128-byte lines: with 16-byte strides every 128-byte row
// of a box lies in two lines, and the products of 1537 columns used the
// tensor cores 62 % of the time.
bool odd_rows(int width) { return width % 8 != 0; }
long long copied_ld(int width) { return up(width, 64); }

// Whether a forward call packs the rows that count: where x is copied
// anyway, and where the product takes some 300 us, against which finding and
// copying the rows (about 10 us) is little even if none is ignored.
bool forward_packs(int rows, int width, int vocab) {
    return odd_rows(width) ||
           (rows > BM && 2.0 * rows * width * static_cast<double>(vocab) > 5e11);
}

struct ForwardSpace {
    CeState *state;
    int *place, *ptarget;
    unsigned short *x, *w;
    float2 *partial;
    size_t bytes;
};

// Columns of a forward call's tiles: 256 or a little less, so that the last
// round of tiles leaves few SMs idle (32768 columns over 76 pairs: two rounds
// of 224 instead of two of 256).
int forward_columns(int rows, int vocab) {
    const long long m_tiles = up(rows, BM) / BM;
    int best = BN;
    long long least = 0;
    for (int bn = BN; bn >= 192; bn -= 32) {
        const long long tiles = m_tiles * (up(vocab, bn) / bn);
        // a tile costs its columns and about 4 more for its start
        const long long cost = (tiles + 75) / 76 * (bn + 4);
        if (bn == BN || cost < least) {
            least = cost;
            best = bn;
        }
    }
    return best;
}

ForwardSpace forward_space(void *ws, int rows, int width, int vocab) {
    Carver c{static_cast<unsigned char *>(ws), 0};
    ForwardSpace s = {};
    const long long ld = copied_ld(width);
    const int bn = forward_columns(rows, vocab);
    s.partial = c.take<float2>(rows * (up(vocab, bn) / bn) * 2);
    if (forward_packs(rows, width, vocab)) {
        s.state = c.take<CeState>(1);
        s.place = c.take<int>(rows);
        s.ptarget = c.take<int>(rows);
        s.x = c.take<unsigned short>(rows * ld);
        if (odd_rows(width)) s.w = c.take<unsigned short>(vocab * ld);
    }
    s.bytes = c.at;
    return s;
}

// A piece of the vocabulary: as many columns as keep its 16-bit gradients
// within 512 MiB, at least 4096 (each piece adds to the FP32 dx once more),
// and pieces of even size.
long long piece_of(int rows, int vocab) {
    long long n = (512ll << 20) / (2 * up(rows, BM)) / BN * BN;
    if (n < 4096) n = 4096;
    const long long pieces = (vocab + n - 1) / n;
    return up((vocab + pieces - 1) / pieces, BN);
}

// Parts of a dx product's reduction: where its tiles alone would leave SMs
// idle, the vocabulary is split, in parts of at least 512 columns.
int splits_of(int rows, int width, int vocab) {
    const long long tiles = up(rows, BM) / BM * (up(width, BN) / BN);
    long long s = 76 / tiles;
    const long long most = piece_of(rows, vocab) / 512;
    if (s > most) s = most;
    return s < 1 ? 1 : static_cast<int>(s);
}

struct BackwardSpace {
    CeState *state;
    int *place, *ptarget;
    float *plse2, *pmiss, *pdloss;
    int pieces;
    unsigned short *x, *w, *grad;
    float *acc;
    size_t bytes;
};

BackwardSpace backward_space(void *ws, int rows, int width, int vocab) {
    Carver c{static_cast<unsigned char *>(ws), 0};
    BackwardSpace s;
    const long long ld = copied_ld(width), piece = piece_of(rows, vocab);
    s.pieces = static_cast<int>((vocab + piece - 1) / piece);
    s.state = c.take<CeState>(1);
    s.place = c.take<int>(rows);
    s.ptarget = c.take<int>(rows);
    s.plse2 = c.take<float>(rows);
    s.pmiss = c.take<float>(rows);
    s.pdloss = c.take<float>(rows);
    s.x = c.take<unsigned short>(rows * ld);
    s.w = odd_rows(width) ? c.take<unsigned short>(vocab * ld) : nullptr;
    s.grad = c.take<unsigned short>(up(rows, BM) * piece);
    s.acc = c.take<float>(splits_of(rows, width, vocab) * up(rows, BM) * up(width, 4));
    s.bytes = c.at;
    return s;
}

// The pack kernel's CTAs for x, and with a weight to copy two waves more.
cudaError_t launch_pack(PackArgs p, cudaStream_t stream) {
    // 8 rows to a CTA, in long calls as many as leave 1024 CTAs, which all read
    // all targets
    p.cta_rows = p.rows <= 8192 ? 8 : static_cast<int>(up((p.rows + 1023) / 1024, 32));
    p.row_ctas = (p.rows + p.cta_rows - 1) / p.cta_rows;
    int weight_ctas = 0;
    if (p.pw != nullptr) {
        weight_ctas = sm_count_of_device() * 8;
        if (weight_ctas > (p.vocab + 7) / 8) weight_ctas = (p.vocab + 7) / 8;
    }
    pack_rows_kernel<<<p.row_ctas + weight_ctas, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

int rows_of_a(int rows) { return rows >= CM ? CM : static_cast<int>(up(rows, 8)); }

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
    long long x_ld = width, w_ld = width;
    const void *x = args.x, *w = args.weight;
    const bool packs = forward_packs(rows, width, vocab);
    if (packs) {
        PackArgs p = {};
        p.x = static_cast<const unsigned short *>(x);
        p.weight = static_cast<const unsigned short *>(w);
        p.target = args.target;
        p.ignore = args.ignore;
        p.rows = rows;
        p.width = width;
        p.vocab = vocab;
        x_ld = copied_ld(width);
        p.ld = static_cast<int>(x_ld);
        p.px = s.x;
        p.pw = s.w;
        p.state = s.state;
        p.place = s.place;
        p.ptarget = s.ptarget;
        p.status = status;
        CE_TRY(launch_pack(p, stream));
        x = s.x;
        if (odd_rows(width)) {
            w = s.w;
            w_ld = x_ld;
        }
    }
    const int bn = forward_columns(rows, vocab);
    GemmMaps maps = {};
    GemmArgs g = {};
    g.job[0] = {rows, vocab, width, bn, rows_of_a(rows), 1, 16, nullptr, 0, 0};
    g.state = packs ? s.state : nullptr;
    g.partial = s.partial;
    g.target = args.target;
    g.ptarget = packs ? s.ptarget : nullptr;
    g.status = status;
    CE_TRY(make_map(&maps.a[0], bf16, x, rows, width, x_ld, g.job[0].a_rows));
    CE_TRY(make_map(&maps.b[0], bf16, w, vocab, width, w_ld, bn / 2));
    if (args.withheld) {
        static std::atomic<int> ready[kMaxDevices];
        if (!bf16 || width > PART_BLOCKS * BK) return cudaErrorNotSupported;
        CE_TRY(launch_gemm_kernel(gemm_withheld_kernel, ready, maps, g, job_tiles(g.job[0]), stream));
    } else {
        CE_TRY((launch_gemm<EPI_LSE, EPI_NONE>(bf16, maps, g, stream)));
    }
    const JoinArgs j = {s.partial, static_cast<const unsigned short *>(x),
                        static_cast<const unsigned short *>(w), x_ld, w_ld, args.target,
                        packs ? s.place : nullptr, args.ignore, rows, width, vocab,
                        static_cast<int>(up(vocab, bn) / bn * 2), args.loss, args.lse, status};
    return launch_dependent(bf16 ? join_lse_kernel<__nv_bfloat16> : join_lse_kernel<__half>,
                            (rows + 3) / 4, 1, 128, 0, stream, j);
}

cudaError_t launch_linear_ce_backward(const LinearCeArgs &args, cudaStream_t stream) {
    cudaError_t err = cudaSuccess;
    unsigned int *status = status_address(&err);
    if (status == nullptr) return err;
    const int rows = args.rows, width = args.width, vocab = args.vocab;
    const int bf16 = args.elem == ELEM_BF16;
    const BackwardSpace s = backward_space(args.ws, rows, width, vocab);
    const long long ld = copied_ld(width), w_ld = odd_rows(width) ? ld : width;
    const long long piece = piece_of(rows, vocab), acc_ld = up(width, 4);
    const int splits = splits_of(rows, width, vocab), a_rows = rows_of_a(rows);
    const unsigned short *w = static_cast<const unsigned short *>(args.weight);
    PackArgs p = {};
    p.x = static_cast<const unsigned short *>(args.x);
    p.weight = w;
    p.target = args.target;
    p.lse = args.lse;
    p.dloss = args.dloss;
    p.ignore = args.ignore;
    p.rows = rows;
    p.width = width;
    p.vocab = vocab;
    p.ld = static_cast<int>(ld);
    p.bf16 = bf16;
    p.px = s.x;
    p.pw = s.w;
    p.state = s.state;
    p.place = s.place;
    p.ptarget = s.ptarget;
    p.plse2 = s.plse2;
    p.pmiss = s.pmiss;
    p.pdloss = s.pdloss;
    p.status = status;
    CE_TRY(launch_pack(p, stream));
    if (odd_rows(width)) w = s.w;
    // dweight through shared memory and tensor-map stores where its rows allow
    const bool store = width % 8 == 0 && reinterpret_cast<uintptr_t>(args.dweight) % 16 == 0;
    const int n_tiles = static_cast<int>(up(width, BN) / BN);
    const int band = n_tiles >= 19 ? 4 : n_tiles <= 4 ? 19 : 76 / n_tiles;
    GemmMaps grad = {}, both = {};
    CE_TRY(make_map(&grad.a[0], bf16, s.x, rows, width, ld, a_rows));
    CE_TRY(make_map(&grad.out, bf16, s.grad, up(rows, BM), piece, piece, 32));
    CE_TRY(make_map(&both.a[0], bf16, s.grad, up(rows, BM), piece, piece, a_rows));   // dx: g
    CE_TRY(make_map(&both.a[1], bf16, s.grad, up(rows, BM), piece, piece, BK));       // dW: g^T
    CE_TRY(make_map(&both.b[1], bf16, s.x, rows, width, ld, BK));                      // dW: x
    GemmArgs g = {};
    g.state = s.state;
    g.status = status;
    g.ptarget = s.ptarget;
    g.plse2 = s.plse2;
    g.pmiss = s.pmiss;
    g.pdloss = s.pdloss;
    g.slice = up(rows, BM) * acc_ld;
    for (int i = 0; i < s.pieces; ++i) {
        const long long n0 = i * piece;
        const int n = static_cast<int>(vocab - n0 < piece ? vocab - n0 : piece);
        CE_TRY(make_map(&grad.b[0], bf16, w + n0 * w_ld, n, width, w_ld, BN / 2));
        CE_TRY(make_map(&both.b[0], bf16, w + n0 * w_ld, n, width, w_ld, BK));             // dx: W
        g.n0 = static_cast<int>(n0);
        g.accumulate = i > 0;
        g.job[0] = {rows, n, width, BN, a_rows, 1, 16, nullptr, 0, 0};
        CE_TRY((launch_gemm<EPI_GRAD, EPI_NONE>(bf16, grad, g, stream)));
        g.job[0] = {args.dx != nullptr ? rows : 0, width, n, BN, a_rows, splits, 8, s.acc, acc_ld, 0};
        g.job[1] = {args.dweight != nullptr ? n : 0, width, rows, BN, CM, 1, band, nullptr, width,
                    store};
        if (args.dweight != nullptr) {
            unsigned short *to = static_cast<unsigned short *>(args.dweight) + n0 * width;
            g.job[1].out = to;
            if (store) CE_TRY(make_map(&both.out, bf16, to, n, width, width, 32));
        }
        CE_TRY((launch_gemm<EPI_DX, EPI_DWEIGHT>(bf16, both, g, stream)));
    }
    if (args.dx == nullptr) return cudaSuccess;
    const long long finish = rows * (up(width, FINISH_COLS) / FINISH_COLS);
    if (finish > 0x7fffffffll) return cudaErrorInvalidValue;
    const unsigned ctas = static_cast<unsigned>(finish);
    if (bf16)
        return launch_dependent(finish_dx_kernel<__nv_bfloat16>, ctas, 1, FINISH_COLS / 4, 0, stream,
                                static_cast<const float *>(s.acc), splits, g.slice,
                                static_cast<int>(acc_ld), static_cast<const int *>(s.place),
                                static_cast<const CeState *>(s.state),
                                static_cast<__nv_bfloat16 *>(args.dx), width);
    return launch_dependent(finish_dx_kernel<__half>, ctas, 1, FINISH_COLS / 4, 0, stream,
                            static_cast<const float *>(s.acc), splits, g.slice,
                            static_cast<int>(acc_ld), static_cast<const int *>(s.place),
                            static_cast<const CeState *>(s.state), static_cast<__half *>(args.dx),
                            width);
}

}  // namespace tile
