// Inline PTX of the fifth-generation tensor cores (tcgen05), the tensor-map
// copies (TMA) and mbarriers with bounded waits, for sm_103a.  MMAs, their
// tensor memory and their loads are those of a CTA pair (cta_group::2): a
// cluster of two CTAs works on one tile of 256 rows, each with half of A's
// rows and half of B's in its shared memory and half of the accumulators'
// rows in its tensor memory; the CTA of rank 0 issues.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace tile {

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---- mbarriers -----------------------------------------------------------------
__device__ __forceinline__ void bar_init(uint32_t bar, unsigned int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect_tx(uint32_t bar, unsigned int bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
// The address that shared memory at `addr` of this CTA has in CTA `rank` of
// the cluster.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Arrives on a barrier of any CTA of the cluster (a peer_addr).  What it tells
// of is this thread's reads of tensor memory (ordered by tc_fence_before), no
// memory that the other CTA reads: the release is the CTA's, as a release to
// the cluster waits for every store of the thread.
__device__ __forceinline__ void bar_arrive_peer(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_test(uint32_t bar, unsigned int parity) {
    unsigned int ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}

// Polls of a barrier before a wait gives up.  A poll suspends the thread for
// up to 4.0 us (measured), so a wait that runs out has lasted 2 s; a tile
// takes microseconds, or 0.1 s where a gradient sums over 20 million tokens.
constexpr unsigned int kBarSpins = 1u << 19;
constexpr unsigned int kTestBarSpins = 1u << 12;   // where a test withholds a copy: 16 ms

// Bounded wait for the phase `parity` of a barrier.  A wait that runs out
// sets `bit` in the device status word and the CTA's abort flag; every
// other wait of the CTA then gives up too, so no wait can hang the GPU.
template <unsigned int SPINS = kBarSpins>
__device__ __forceinline__ bool bar_wait(uint32_t bar, unsigned int parity, volatile int *abort_flag,
                                         unsigned int *status, unsigned int bit) {
    for (unsigned int i = 0; i < SPINS; ++i) {
        if (bar_test(bar, parity)) return true;
        if ((i & 63u) == 63u && *abort_flag) return false;
    }
    if (*abort_flag == 0) *abort_flag = 1;
    atomicOr(status, bit);
    return false;
}

// The same for what every CTA of a cluster sends in each round, whether its own
// waits gave up or not: it goes on where only a bar_wait has, since a CTA that
// left out a round would count a later round's bytes for it, and waits four
// times as long, as the others may have waited for something first.  One that
// runs out all the same is the CTA's last.
template <unsigned int SPINS = kBarSpins>
__device__ __forceinline__ void bar_wait_round(uint32_t bar, unsigned int parity,
                                               volatile int *abort_flag, unsigned int *status,
                                               unsigned int bit) {
    for (unsigned int i = 0; i < 4 * SPINS; ++i) {
        if (bar_test(bar, parity)) return;
        if ((i & 63u) == 63u && *abort_flag == 2) return;
    }
    *abort_flag = 2;
    atomicOr(status, bit);
}

// ---- TMA -------------------------------------------------------------------------
// A box at (x, y) into this CTA's shared memory, counted on `bar`, a
// peer_addr of either CTA of the pair.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y,
                                         uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// Shared memory to the box of `map` at (x, y); what lies outside the matrix
// is not written.  x and y lie inside it.
__device__ __forceinline__ void tma_store(const CUtensorMap *map, int x, int y, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     map),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void store_commit() {
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Until at most N of this thread's groups of stores still read shared memory.
template <int N>
__device__ __forceinline__ void store_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void store_wait() {
    asm volatile("cp.async.bulk.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---- tensor memory and MMA -----------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t slot, unsigned int columns) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, unsigned int columns) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns)
                 : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Arrives on the barrier at `bar` of both CTAs of the pair when every MMA
// issued so far by this thread is done.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"(static_cast<unsigned short>(3))
        : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(static_cast<unsigned int>(accumulate))
                 : "memory");
}
// 32 consecutive FP32 columns of this warp's 32 lanes (thread = lane), there
// after tmem_wait().
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32]) {
    __syncwarp();   // the load is a whole warp's; a branch before it may have split it
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
// Until this thread's loads are there.  The values pass through it, so that
// nothing that uses them is moved before it.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                   "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28])
                 :
                 : "memory");
    asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
    uint32_t r[32];
    tmem_load32(addr, r);
    tmem_wait(r);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// 16 columns, added to v.
__device__ __forceinline__ void tmem_add16(uint32_t addr, float *v) {
    uint32_t r[16];
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(r[i]);
}
// 64 columns, both loads at once.
__device__ __forceinline__ void tmem_load64(uint32_t addr, float (&v)[64]) {
    uint32_t a[32], b[32];
    tmem_load32(addr, a);
    tmem_load32(addr + 32, b);
    tmem_wait(a);
    tmem_wait(b);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        v[i] = __uint_as_float(a[i]);
        v[32 + i] = __uint_as_float(b[i]);
    }
}

// Shared-memory descriptor of a 128-byte-swizzled operand whose tiles start
// on 1024 bytes.  K-major (rows of 64 two-byte elements along K, 8-row
// groups 1024 bytes apart): lead unused, stride 1024.  MN-major (rows of 64
// elements along M or N, one row per k): lead = bytes from one 64-element
// column block to the next, stride 1024 from 8 k rows to the next 8.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
    return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) |
           (static_cast<uint64_t>(lead >> 4) << 16) | (static_cast<uint64_t>(stride >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// Instruction descriptor of kind::f16 with FP32 accumulation.
__device__ __forceinline__ uint32_t mma_idesc(bool bf16, bool a_mn, bool b_mn, int m, int n) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) |
           ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// ---- dependent launches ------------------------------------------------------------
// A kernel launched with programmatic stream serialisation may start before
// the one before it in the stream has ended, and waits here for its end
// (and its writes) before it touches memory.
__device__ __forceinline__ void dependency_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void dependency_launch() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace tile
