// Tensor-core building blocks of the experts' products: mbarriers with
// bounded waits, tiled TMA loads, TMEM allocation and loads, tcgen05.mma
// descriptors, and the schedule of tiles over ragged groups of rows.
#pragma once

#include <cuda.h>  // CUtensorMap and the encode call's types; the call itself is fetched at run time
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_internal.cuh"
#include "pdl.cuh"

namespace moe {

// ---- shared memory and mbarriers -------------------------------------------

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mb_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mb_init_fence() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void mb_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mb_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mb_try(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// The same where the other block of a pair may have arrived after writing what
// is read next: the wait acquires for the cluster, not for the block alone.
__device__ __forceinline__ bool mb_try_pair(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// A value that every lane of a converged warp holds: the compiler then knows
// that it is the same in all of them, keeps it in uniform registers and takes
// branches on it without considering divergence.
__device__ __forceinline__ int same(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// One lane of a converged warp, the same one every time.  The warps that issue
// loads and mma run their loops whole and enclose only the issue in this
// test: within `if (lane == 0)` around the loop, every operand that the
// instructions want in a uniform register was fetched the slow way (fp8
// product: 1100 cycles a block, 480 of them to issue four mma).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// Every wait is bounded: after `polls` polls (each may suspend briefly), or once
// another warp of the block has given up, it returns false and the block's
// word `gave_up` is set; each role then leaves its loop, copies in flight are
// waited for (again bounded), TMEM is freed and the kernel ends.  A failing poll is
// suspended for 3.9 us on GB300, which nothing promises: kPolls are 4 s, and
// 10 ms if polls took as little as 10 ns, where a stage takes well under 10 us; a
// wait that spans more adds kStepPolls (16 ms, or 40 us) for each stage.
constexpr long long kPolls = 1 << 20, kStepPolls = 1 << 12;

// The limit of a role's waits where they may span whole tiles, some of which
// have no stages but results to be written (zeros, 256 KB a pair: 3 us at the
// rate of HBM, a stage's allowance again).  Roles run ahead of
// one another through such tiles without waiting, so all that came before count
// for every later wait, of tiles with stages those since the last wait.
struct WaitLimit {
    long long stages = 0, empty_tiles = 0;
    __host__ __device__ void tile(int steps) {  // each tile, as the role comes to it
        if (steps > 0) stages += steps;
        else ++empty_tiles;
    }
    __host__ __device__ void waited() { stages = 0; }
    __host__ __device__ long long polls() const { return kPolls + (stages + empty_tiles) * kStepPolls; }
};
__device__ __forceinline__ bool mb_wait(uint32_t bar, uint32_t parity, volatile int *gave_up, long long polls = kPolls) {
    for (long long i = 0; i < polls; ++i) {
        if (mb_try(bar, parity)) return true;
        if ((i & 15) == 15 && *gave_up) return false;
    }
    *gave_up = 1;
    return false;
}
__device__ __forceinline__ bool mb_wait_warp(uint32_t bar, uint32_t parity, volatile int *gave_up,
                                             long long polls = kPolls) {
    if (__all_sync(0xffffffffu, mb_try(bar, parity))) return true;
    return __all_sync(0xffffffffu, mb_wait(bar, parity, gave_up, polls));
}
__device__ __forceinline__ bool mb_wait_warp_pair(uint32_t bar, uint32_t parity, volatile int *gave_up, long long polls) {
    const bool ok = mb_wait_warp(bar, parity, gave_up, polls);
    return ok && __all_sync(0xffffffffu, mb_try_pair(bar, parity));  // complete: acquires, does not wait
}
__device__ __forceinline__ void mb_drain(uint32_t bar, uint32_t parity) {  // bounded, result not needed
    for (long long i = 0; i < kPolls && !mb_try(bar, parity); ++i) {
    }
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t v) {  // the low half of v
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"((unsigned short)v) : "memory");
}
__device__ __forceinline__ void st_shared32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_shared128(uint32_t addr, const uint4 &v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint4 ld_shared128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
// Two f32 (bits) rounded to bf16, the first in the low half.
__device__ __forceinline__ uint32_t bf16x2(uint32_t first, uint32_t second) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(second)), "f"(__uint_as_float(first)));
    return r;
}

// silu(g) u; exp within 2 units in the last place, the fast division too.
// A divisor above 2^126 (g below -87.3; exp(-g) = infinity too) gives 0, and NaN for
// g = -infinity.
__device__ __forceinline__ float silu_mul(float g, float u) { return __fdividef(g, 1.f + expf(-g)) * u; }

// Position in a ring of kSlots slots: the slot and the parity of its use.
template <int kSlots>
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == kSlots) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// Waits (bounded, all slots together) for the last use of every slot of a
// ring: r is the producer's position after its last load.  Nothing may still be
// landing in shared memory, loads or arrivals at a barrier, when the block ends.
// On `full` barriers the last loads have landed, on `empty` ones mma has read
// them too.  A pair's loads are counted on the leader's `full` barriers alone,
// and after a wait that gave up the two producers may be at different places:
// each block knows about its own loads, and about the arrivals that the leader's
// commits send it, by its own `empty` barriers.
template <int kSlots>
__device__ __forceinline__ void drain_ring(uint32_t bars, Ring<kSlots> r, long long left = kPolls) {
    for (int i = 0; i < kSlots; ++i) {
        while (!mb_try(bars + 8 * r.slot, r.phase ^ 1u) && left > 0) --left;
        r.next();
    }
}

// This translation unit's error word (device symbols are per unit): set by a
// block whose wait gave up, read and cleared by take_tc_error.
static __device__ int g_tc_error = 0;
__device__ __forceinline__ void record_timeout() { atomicCAS(&g_tc_error, 0, MOE_ERR_TIMEOUT); }

// ---- tiled TMA loads ---------------------------------------------------------

__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            dst),
        "l"(m), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int c0, int c1,
                                            int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];" ::"r"(dst),
        "l"(m), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
// Rows of a row-major operand by boxes of 128, 64 and 32 rows of 128 bytes: a
// block's rows of a tile, at most 128, rounded up to 32, in as few loads as
// the number has binary digits.  (A load costs the TMA about as much as 40
// rows: 16384 tokens by K = 2048, F = 4096 took 274 us with boxes of 32 rows
// only, 212 with boxes of 64.)
struct RowMaps {
    CUtensorMap m[3];
    int first;  // the largest box that any tile of the batch can need; larger ones have no map
};
__device__ __forceinline__ void prefetch_maps(const RowMaps &maps) {
    for (int i = maps.first; i < 3; ++i) tma_prefetch_map(&maps.m[i]);
}
__host__ __device__ constexpr int rows_loaded(int n) { return (n + 31) & ~31; }
__device__ __forceinline__ void load_rows(uint32_t dst, const RowMaps &maps, uint32_t bar, int c0, int row, int n) {
    const int rows = rows_loaded(n);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int box = 128 >> i;
        if (rows & box) {
            tma_load_2d(dst, &maps.m[i], bar, c0, row);
            dst += box * 128;
            row += box;
        }
    }
}

// ---- TMEM and tcgen05.mma ----------------------------------------------------

__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t cols) {  // one whole warp
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {  // the allocating warp
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Arrives on `bar` once every mma this thread has issued so far is done.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}

// Loads of 32 lanes x 32 columns of 32 bits; a warp reaches the 32 lanes of its
// place in its group of four.
// The load alone: its registers may be read after tmem_wait32 on them.
__device__ __forceinline__ void tmem_load32_async(uint32_t addr, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait32(uint32_t *r) {  // waits for every load of the warp
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t *r) {  // complete on return
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}

// Most elements of a sum that bf16 results take in one accumulator.  The tensor
// core cuts off what it adds: a sum of n terms comes out small by about 1e-9 n of
// itself, 5e-9 n where all terms have one sign.  After these many that is 8e-5,
// a fiftieth of what the rounding to bf16 alone may be off by (2^-8).
constexpr int kWhole = 1 << 14;

// ---- pairs of blocks (clusters of two; cta_group::2) --------------------------
//
// One tcgen05.mma spans the two SMs of a cluster: each block holds half of A
// (its 128 rows of M) and half of B's columns, and gets its 128 rows of the
// result in its own TMEM.  Both halves' loads are counted on the leader's
// (rank 0's) barrier; the leader issues mma and its commits arrive on both
// blocks' barriers.

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {  // every thread of both blocks
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t at_leader(uint32_t addr) {  // the same place in rank 0's shared memory
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}
// Arrives at a barrier of the leader (bar from at_leader).  The released form
// orders the thread's writes before it, for which it waits until its global
// stores have reached L2: 2000 to 3400 cycles after a tile's results.  What
// frees an accumulator only orders TMEM loads, which are complete (wait::ld,
// then tc_fence_before): the relaxed form does.
__device__ __forceinline__ void mb_arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mb_arrive_remote_relaxed(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *m, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4}], [%2];" ::"r"(dst),
        "l"(m), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *m, uint32_t bar, int c0, int c1,
                                                 int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4, %5}], [%2];" ::"r"(dst),
        "l"(m), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ void tma_load_5d_pair(uint32_t dst, const CUtensorMap *m, uint32_t bar, int c0, int c1,
                                                 int c2, int c3, int c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4, %5, %6, %7}], [%2];" ::"r"(dst),
        "l"(m), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
}
__device__ __forceinline__ void load_rows_pair(uint32_t dst, const RowMaps &maps, uint32_t bar, int c0, int row, int n) {
    const int rows = rows_loaded(n);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int box = 128 >> i;
        if (rows & box) {
            tma_load_2d_pair(dst, &maps.m[i], bar, c0, row);
            dst += box * 128;
            row += box;
        }
    }
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t cols) {  // one warp of each block
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_commit_pair(uint32_t bar) {  // arrives in both blocks
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((unsigned short)3)
        : "memory");
}
__device__ __forceinline__ void mma_bf16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(desc), "r"((uint32_t)accumulate)
        : "memory");
}

// Shared-memory operand with 128-byte swizzle (the layout tiled TMA writes
// with CU_TENSOR_MAP_SWIZZLE_128B from 1024-byte aligned tiles): groups of
// eight 128-byte lines are `stride` bytes apart; for an operand whose
// reduction is not the contiguous dimension, blocks of 64 16-bit elements of
// the contiguous one are `lead` bytes apart.
__device__ __forceinline__ uint64_t smem_operand(uint32_t addr, uint32_t lead, uint32_t stride) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: f32 accumulation; formats 0 = f16 / e4m3, 1 = bf16;
// transposed operands are those whose reduction is not contiguous.
__host__ __device__ constexpr uint32_t mma_desc(int fmt, bool a_transposed, bool b_transposed, int M, int N) {
    return (1u << 4) | ((uint32_t)fmt << 7) | ((uint32_t)fmt << 10) | ((uint32_t)a_transposed << 15) |
           ((uint32_t)b_transposed << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(desc), "r"((uint32_t)accumulate)
        : "memory");
}

// ---- groups of rows -----------------------------------------------------------

// The experts' rows in the receive regions, one entry per expert, in shared
// memory: first row, number of rows (what fits the region), and the
// exclusive prefix sum of their tiles.
struct Groups {
    int *row;     // [E]
    int *count;   // [E]
    int *prefix;  // [E + 1], in the order in which the tiles are taken
    int *order;   // [E], the experts in that order
    int shift;    // log2 of the most rows (or columns) of a tile
    int sorted;   // `order` is not the experts' own
};
__host__ __device__ constexpr int groups_bytes(int E, bool ordered = false) {
    return (((ordered ? 4 : 3) * E + 1) * 4 + 127) / 128 * 128;
}

__device__ __forceinline__ int scan(int v, int lane) {  // sum over the lanes up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Fills the tables from expert_offsets; every thread of the block calls it.
// tiles(count, shift) is the number of tiles of a group when a tile takes at
// most 2^shift rows.  The shift is kMost, made less (down to kLeast) as long
// as all tiles then still run at once in the `units` of the grid: tiles that
// leave some idle are made shorter.  Where they take more than kRounds rounds
// (fewer gain less than the sorting takes), and kRanks > 1, the groups are
// taken in the order of rank(count), 0 to kRanks - 1 (for groups without
// rows), so that the tiles of a round are alike.  Groups stay inside the regions
// and within `most` rows whatever the offsets are; offsets that no batch of
// `pairs` rows has (they descend, or span more) stand for no rows at all: the
// number of tiles, checked by the host for `pairs` rows, could pass 32 bits.
constexpr int kRounds = 4;
template <int kMost, int kLeast, int kRanks, class Tiles, class Rank>
__device__ __forceinline__ Groups make_groups(int *mem, const int32_t *__restrict__ offsets, int E, int L, int64_t cap,
                                              int64_t most, int64_t pairs, int units, Tiles tiles, Rank rank) {
    constexpr bool kSort = kRanks > 1;
    __shared__ int s_shift, s_sorted;
    Groups g{mem, mem + E, mem + 2 * E, mem + 3 * E + 1, kMost, 0};
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        const int d = e / L;
        // four loads at once: one behind the others costs 0.3 us a call
        const int64_t first = __ldg(offsets), base = __ldg(offsets + d * L);
        int64_t lo = (int64_t)__ldg(offsets + e) - base, hi = (int64_t)__ldg(offsets + e + 1) - base;
        const bool descends = (hi < lo) | (base + hi - first > pairs);
        lo = lo < 0 ? 0 : (lo < cap ? lo : cap);
        hi = hi < lo ? lo : (hi < cap ? hi : cap);
        if (hi - lo > most) hi = lo + most;
        g.row[e] = (int)(d * cap + lo);
        g.count[e] = descends ? -1 : (int)(hi - lo);
        if constexpr (kSort) g.order[e] = e;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        constexpr int kTries = kMost - kLeast + 1;
        const int lane = threadIdx.x, per = (E + 31) / 32, e0 = lane * per, e1 = min(E, e0 + per);
        int sums[kTries] = {}, shift = kMost, sorted = 0;
        int signs = 0;
        for (int e = e0; e < e1; ++e) {
            const int c = g.count[e];
            signs |= c;
#pragma unroll
            for (int i = 0; i < kTries; ++i) {
                sums[i] += tiles(c, kMost - i);
                if (i > 0) sums[i] = min(sums[i], 1 << 25);  // too many anyway; 32 lanes' do not overflow
            }
        }
        if (__any_sync(0xffffffffu, signs < 0)) {  // no rows
            for (int e = e0; e < e1; ++e) g.count[e] = 0;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kTries; ++i) sums[i] = max(0, e1 - e0) * tiles(0, kMost - i);
        }
        int sum = sums[0];
        if constexpr (kTries > 1) {
            int all[kTries];  // does not get less with the shift
#pragma unroll
            for (int i = 1; i < kTries; ++i) all[i] = __reduce_add_sync(0xffffffffu, sums[i]);
#pragma unroll
            for (int i = 1; i < kTries; ++i) {
                if (all[i] <= units) shift = kMost - i, sum = sums[i];
            }
        }
        if constexpr (kSort) {
            if (__reduce_add_sync(0xffffffffu, sum) > kRounds * units) {
                int at[kRanks] = {}, first = 0, kinds = 0;  // groups of a rank, then the next one's place
                for (int c0 = 0; c0 < E; c0 += 32) {
                    int r = -1;
                    if (c0 + lane < E) g.prefix[c0 + lane] = r = rank(g.count[c0 + lane]);
#pragma unroll
                    for (int i = 0; i < kRanks; ++i) at[i] += __popc(__ballot_sync(0xffffffffu, r == i));
                }
#pragma unroll
                for (int i = 0; i < kRanks; ++i) {
                    const int n = at[i];
                    at[i] = first;
                    first += n;
                    kinds += i < kRanks - 1 && n > 0;
                }
                if (kinds > 1) {
                    sorted = 1;
                    for (int c0 = 0; c0 < E; c0 += 32) {
                        const int r = c0 + lane < E ? g.prefix[c0 + lane] : -1;
#pragma unroll
                        for (int i = 0; i < kRanks; ++i) {
                            const uint32_t alike = __ballot_sync(0xffffffffu, r == i);
                            if (r == i) g.order[at[i] + __popc(alike & ((1u << lane) - 1))] = c0 + lane;
                            at[i] += __popc(alike);
                        }
                    }
                    __syncwarp();  // the order is complete
                    sum = 0;
                    for (int i = e0; i < e1; ++i) sum += tiles(g.count[g.order[i]], shift);
                }
                __syncwarp();  // prefix is written again
            }
        }
        int before = scan(sum, lane);
        if (lane == 31) g.prefix[E] = before;
        if (lane == 0) s_shift = shift, s_sorted = sorted;
        before -= sum;
        for (int i = e0; i < e1; ++i) {
            g.prefix[i] = before;
            before += tiles(g.count[kSort ? g.order[i] : i], shift);
        }
    }
    __syncthreads();
    if constexpr (kLeast < kMost) g.shift = same(s_shift);
    if constexpr (kSort) g.sorted = same(s_sorted);
    return g;
}

// Rows of each of a group's `tiles` equal tiles (count > 0): count + tiles - 1 need
// not fit 32 bits.
__host__ __device__ constexpr int tile_rows(int count, int tiles) { return (count - 1) / tiles + 1; }

// The group that holds tile t (prefix[e] <= t < prefix[e + 1]), searched
// from group e on: tiles are taken in ascending order, so e only grows.
__device__ __forceinline__ int find_group(const Groups &g, int E, int e, int t) {
    int step = 1;
    while (e + step < E && g.prefix[e + step] <= t) {
        e += step;
        step <<= 1;
    }
    for (step >>= 1; step > 0; step >>= 1)
        if (e + step < E && g.prefix[e + step] <= t) e += step;
    return e;
}

// ---- host side ------------------------------------------------------------------

// Reads and clears this unit's error word (the stream has been waited for).
static inline cudaError_t take_tc_error(int *err) {
    cudaError_t e = cudaMemcpyFromSymbol(err, g_tc_error, sizeof(int));
    if (e != cudaSuccess || *err == 0) return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_tc_error, &zero, sizeof(int));
}

// Whether a kernel's dynamic shared memory limit has been raised in the
// current device and context (one object per kernel and host thread).
struct AttrCache {
    int dev = -1;
    unsigned long long ctx = 0;
    cudaError_t allow_smem(const void *kernel, int bytes) {
        int now = 0;
        cudaError_t e = cudaGetDevice(&now);
        if (e != cudaSuccess) return e;
        const unsigned long long key = context_key();
        if (now == dev && key != 0 && key == ctx) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        dev = now;
        ctx = context_key();
        return cudaSuccess;
    }
};

// Launch of a persistent kernel in clusters of two blocks.
struct PairLaunch {
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};
    PairLaunch(int threads, int smem, cudaStream_t stream) {
        attr[0] = pdl_attribute();
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 2;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
    }
    PairLaunch(const PairLaunch &) = delete;
};

// Such a kernel's shared memory limit, as above, and the number of its blocks
// that fit the device at once.
struct PairCache {
    AttrCache attr;
    int dev = -1, blocks = 0;
    unsigned long long ctx = 0;
    cudaError_t prepare(const void *kernel, const cudaLaunchConfig_t &cfg) {  // cfg with the most shared memory
        cudaError_t e = attr.allow_smem(kernel, (int)cfg.dynamicSmemBytes);
        if (e != cudaSuccess || (blocks > 0 && dev == attr.dev && ctx == attr.ctx && ctx != 0)) return e;
        int clusters = 0;
        e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
        if (e != cudaSuccess) return e;
        if (clusters < 1) return cudaErrorLaunchOutOfResources;
        blocks = 2 * clusters;
        dev = attr.dev;
        ctx = attr.ctx;
        return cudaSuccess;
    }
};

// Tiled tensor map with 128-byte swizzle and zero fill out of bounds;
// strides in bytes for dimensions 1.. (false: the driver refused it).
bool encode_map(CUtensorMap *m, int fp8, int rank, const void *base, const uint64_t *dims, const uint64_t *strides,
                const uint32_t *box);

// The maps of load_rows over rows of `cols` elements (16-bit, or 8-bit: fp8),
// of which no tile takes more than `most` at once.
inline bool encode_rows(RowMaps *maps, int fp8, const void *base, int cols, int64_t rows, int64_t most) {
    const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, stride = (uint64_t)cols * (fp8 ? 1 : 2);
    maps->first = most > 96 ? 0 : most > 32 ? 1 : 2;  // by rows_loaded(most)
    for (int i = maps->first; i < 3; ++i) {
        const uint32_t box[2] = {fp8 ? 128u : 64u, 128u >> i};
        if (!encode_map(&maps->m[i], fp8, 2, base, dims, &stride, box)) return false;
    }
    return true;
}

}  // namespace moe
