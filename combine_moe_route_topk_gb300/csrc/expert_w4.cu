// Product of the experts' rows with matrices of 4-bit weights, on the layout
// that dispatch writes:
//
//   y[p][f] = r[e][f] sum_k x[p][k] (s[e][k/group][f] q[e][f][k])
//
// q has 4 bits, s (e4m3) four significant ones: q s has at most seven and is
// exact in bf16, which has eight.  So the weights become bf16 on the way and
// the tensor core multiplies them exactly; r multiplies the f32 sum.
//
// The matrix is the operand with 128 rows of tcgen05.mma (M), read from TMEM;
// the expert's tokens are its columns (N).  A block's warps: one loads codes
// (TMA) and group scales, one loads the tokens (TMA), one issues mma, 16 turn
// codes into bf16 (a thread has one matrix row) and write them to TMEM, eight
// store results.  Dequantised weights never see shared memory: there they
// would cost 2 x 2 bytes a weight for writing and reading where the codes
// come in at 44 a cycle from HBM, 176 bytes a cycle of the 128 it has.
//
// An mma of 128 rows and 16 elements takes 33 cycles with up to 32 tokens, 44 with
// 64, 72 with 128, 80 with 144 (measured, A in TMEM); to issue one takes some 25,
// a commit 87, a wait for a barrier that is complete 40 to 60.  So a unit has
// eight mma: with four, 256 tokens of 64 experts (K = 7168, F = 2048 gated) took
// 356 us, with eight 226.  There instructions bound it, 30 weights a cycle and SM: 75 % of
// the issue slots are in use, by 1650 instructions a unit, 704 of which take codes apart
// (the others wait, arrive, convert scales, compute addresses and store results); HBM, at
// 57 %, would bring 44.  With 8192 rows (K = 2048, F = 7168) the mma, 127 us of
// 169, and what keeps them waiting: with half the tokens' bytes loaded (for
// timing alone) it took 6 us less, without the arithmetic on the codes 14, without either 18;
// call after call the clock comes down and it takes 168 to 198, by the box.  Three slots of tokens
// and two stages of codes more: 185 us alone; pairs of blocks that load half the tokens
// each for both: the same.
#include <cuda_bf16.h>

#include "expert_w4_internal.cuh"
#include "pdl.cuh"
#include "tc_ops.cuh"
#include "w4_ops.cuh"
#include "w4_rule.cuh"

namespace moe {
namespace {

using namespace w4_tile;
constexpr int kCodes = kM * 128, kScales = 8 * kM;  // bytes of a stage
constexpr int kDequantWarps = 16;  // in sets, which turn units into bf16 by turns
constexpr int kStoreWarps = 8;
constexpr int kPartUnits = 512 / kK;  // units of a part of an f32 result's sum

// TMEM holds two accumulators of kTok columns, so that a tile's results leave
// while the next one is computed, and kSlots slots of 64 columns for weights.
// kTok = 64 for few tokens, 160 beyond (with 128, experts of a little more have
// their weights turned into bf16 twice: 8192 rows of 64 experts 199 us against
// 183; with 192 there is room for three slots of tokens only).
// For sums in parts the storing warps hold kTok / 2 sums a thread in registers:
// 896 threads are launched with 72 each, the storing ones take 104 or 120, the
// dequantising ones keep 64 or 56, the others (with an idle warp, so that they
// are four) 40.
template <int kTok, bool kParts, bool kF32, bool kSplit>
struct Shape {
    static constexpr int kSlots = (512 - 2 * kTok) / (kK / 2);
    static constexpr int kRowSlots = kTok == 64 ? 6 : 4;
    // Dequantising warps work in sets of four, which take units by turns.  A unit's barriers are those of its slot of
    // rows; its slot in TMEM is free once the unit kSlots before is done.  Its set waits for that one's barrier: the
    // barrier's use before is complete then (the set has waited for a unit kSets before that one), and its next use
    // is this unit or a later one.  Four sets in 8192 rows, call after call: 187 us, two of eight warps 196 (each warp
    // does what there is besides the codes for half as many of them); two, with barriers for weights and rows apart, 193.
    static constexpr int kSets = 4;
    static_assert(kSlots <= kRowSlots && kSets <= kRowSlots && kSets * 4 == kDequantWarps);
    static constexpr int kHalf = kTok * 128, kRows = 2 * kHalf;  // bytes of half a unit's token rows, of a slot of them
    static constexpr int kCodeStages = kSplit ? (kF32 ? 3 : 4) : kTok == 64 ? 5 : kParts ? 3 : 2;
    static constexpr int kJoin = kSplit ? 24 << 10 : 0;  // other blocks' sums: 8 / S warps, S - 1 blocks, 4 KB
    static constexpr int kThreads = 32 * (kDequantWarps + kStoreWarps + (kParts ? 4 : 3));
    static constexpr int kStoreRegs = kTok == 64 ? 104 : 120, kDequantRegs = kTok == 64 ? 64 : 56;
    static_assert(!kParts || 32 * (kStoreWarps * kStoreRegs + kDequantWarps * kDequantRegs + 4 * 40) <= kThreads * 72);
    static constexpr int kBuf = kF32 ? 4096 : 2048;  // a storing warp's: 32 tokens' results, to be written as whole sectors
    // Barriers: full and empty of the rings, of the two accumulators, the end, and of the storing warps' joins.
    static constexpr int kBars = 2 * kCodeStages + 2 * kRowSlots + 5 + (kSplit ? 2 * kStoreWarps : 0);
    static constexpr int kSmem = 1024 + kCodeStages * (kCodes + kScales) + kRowSlots * kRows + kStoreWarps * kBuf + kJoin;
};

// Token rows by boxes of 128, 64, 32 and 16 rows of 128 bytes.
struct TokenMaps {
    CUtensorMap m[4];
    int first;  // the largest box that any tile of the batch can need
};

struct Args {
    const int32_t *offsets;
    const uint8_t *group_scales;
    const float *row_scales;
    void *y;
    int64_t cap, most, pairs;
    int E, L, K, F, wide, groups, group_shift;
    int split;  // blocks that share a tile's reduction
};

__host__ __device__ constexpr int mma_tokens(int n) { return (n + 15) & ~15; }
template <int kTok>
__device__ __forceinline__ int token_tiles(int count) {
    return count > 0 ? (count - 1) / kTok + 1 : 0;  // count + kTok need not fit 32 bits
}

struct Tile {
    int e, m0, row, n;  // group, first matrix row (or feature), first token row, tokens
};

// Tiles of a group: its token tiles (of equal size) run fastest, so that
// blocks working at the same time share the matrix rows through L2.
template <int kTok>
__device__ __forceinline__ Tile get_tile(const Groups &g, int E, int e, int t, int m_step) {
    Tile r;
    r.e = same(find_group(g, E, e, t));
    const int c = same(g.count[r.e]), nt = token_tiles<kTok>(c), at = t - same(g.prefix[r.e]);
    int m = at, first = 0, size = c;
    if (nt > 1) {  // three divisions, 0.2 us before a block's first load
        m = at / nt;
        size = mma_tokens(tile_rows(c, nt));
        first = (at - m * nt) * size;
    }
    r.m0 = m * m_step;
    r.row = same(g.row[r.e]) + first;
    r.n = min(size, c - first);
    return r;
}

// 32 lanes x 16 columns of 32 bits; done after tmem_store_wait.
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D += A B, A in TMEM: lane i holds row i, a column two elements of the reduction.
__device__ __forceinline__ void mma_bf16_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t desc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(desc), "r"((uint32_t)accumulate)
        : "memory");
}

// kSplit: a cluster of a.split blocks (two or four) takes a tile, each a part of
// the reduction.  Block q % S stores the rows of the tile's quarter q, and gets
// the other blocks' sums of them in its shared memory: 32 rows by 32 tokens
// of a storing warp at a time, added to its own in the blocks' order.
template <int kTok, bool kGated, bool kParts, bool kF32, bool kSplit>
__global__ void __launch_bounds__(Shape<kTok, kParts, kF32, kSplit>::kThreads, 1)
expert_w4_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ TokenMaps map_x, const Args a) {
    using S = Shape<kTok, kParts, kF32, kSplit>;
    static_assert(!kSplit || kTok == 64);  // one piece of 32 tokens a storing warp
    constexpr int kSlots = S::kSlots, kRows = S::kRows, kRowSlots = S::kRowSlots, kCodeStages = S::kCodeStages, kBuf = S::kBuf;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long bars[S::kBars];
    __shared__ uint32_t s_tmem;
    __shared__ int s_gave_up;
    const int tid = threadIdx.x, warp = same(tid / 32), lane = tid % 32;
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t rows_at = smem + kCodeStages * kCodes, scales_at = rows_at + kRowSlots * kRows,
                   bufs_at = scales_at + kCodeStages * kScales, join_at = bufs_at + kStoreWarps * kBuf,
                   tables_at = join_at + S::kJoin;
    int *tables = reinterpret_cast<int *>(smem_raw + (tables_at - smem_u32(smem_raw)));
    // A unit has one pair of barriers, of its rows' slot: `full` counts the rows' bytes and the weights' warps,
    // `empty` is the mma's one commit for both.
    const uint32_t cfull = smem_u32(bars), cempty = cfull + 8 * kCodeStages, full = cempty + 8 * kCodeStages,
                   empty = full + 8 * kRowSlots, tfull = empty + 8 * kRowSlots, tempty = tfull + 16, done = tempty + 16, jfull = done + 8, jfree = jfull + 8 * kStoreWarps;
    volatile int *gave_up = &s_gave_up;
    constexpr int kStoreFirst = kDequantWarps, kCodeWarp = kDequantWarps + kStoreWarps, kRowWarp = kCodeWarp + 1,
                  kMmaWarp = kCodeWarp + 2;

    if (warp == kMmaWarp) tmem_alloc(smem_u32(&s_tmem), 512);
    if (tid == 0) {
        for (int i = 0; i < kCodeStages; ++i) {
            mb_init(cfull + 8 * i, 1 + 32);  // the loads' bytes, and the lanes that copy scales
            mb_init(cempty + 8 * i, kDequantWarps);
        }
        for (int i = 0; i < kRowSlots; ++i) {
            mb_init(full + 8 * i, 1 + 4);
            mb_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mb_init(tfull + 8 * i, 1);
            mb_init(tempty + 8 * i, kStoreWarps);
        }
        mb_init(done, 1);
        for (int i = 0; kSplit && i < kStoreWarps; ++i) {
            mb_init(jfull + 8 * i, 1);  // the other blocks' sums are here: their bytes
            mb_init(jfree + 8 * i, 1);  // this block's have been read
        }
        s_gave_up = 0;
        mb_init_fence();
        tma_prefetch_map(&map_w);
        for (int i = map_x.first; i < 4; ++i) tma_prefetch_map(&map_x.m[i]);
    }
    const int rank = kSplit ? same((int)cluster_rank()) : 0, split = kSplit ? a.split : 1, shift = split >> 1;  // its log2
    tc_fence_before();
    if constexpr (kSplit) cluster_arrive();  // waited for by those who reach the other blocks, and by the others at the end
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)same((int)s_tmem), a_at = tmem + 2 * kTok;
    grid_dependency_wait();  // offsets and rows come from earlier kernels
    grid_launch_dependents();
    constexpr int kStep = kGated ? kM / 2 : kM;  // result columns of a tile
    const int m_tiles = (a.F + kStep - 1) / kStep, tile0 = blockIdx.x >> shift, tile_step = gridDim.x >> shift;
    const Groups g = make_groups<0, 0, 1>(
        tables, a.offsets, a.E, a.L, a.cap, a.most, a.pairs, tile_step,
        [&](int c, int) { return token_tiles<kTok>(c) * m_tiles; }, [](int) { return 0; });  // syncs the block
    const int tiles = same(g.prefix[a.E]);
    // this block's units of a tile: whole stages of codes
    const int all = (a.K + kK - 1) / kK, stages = (all + kUnits - 1) / kUnits;
    const int first = kSplit ? (stages * rank >> shift) * kUnits : 0;
    const int units = kSplit ? min(all, (stages * (rank + 1) >> shift) * kUnits) : all;
    const int part = kParts ? kPartUnits : units - first;  // units that are summed in TMEM

    if constexpr (kParts) {
        if (warp < kDequantWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kDequantRegs));
        else if (warp >= kCodeWarp) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    }

    if (warp == kCodeWarp) {
        Ring<kCodeStages> r;
        int e = 0;
        bool ok = true;
        const int per_stage = 256 >> a.group_shift;
        for (int t = tile0; t < tiles && ok; t += tile_step) {
            const Tile w = get_tile<kTok>(g, a.E, e, t, kStep);
            e = w.e;
            // lanes copy the scales of four matrix rows each
            int f = w.m0 + lane * 4;
            bool inside = f < a.F;
            if constexpr (kGated) {  // rows run in groups of 8 gate rows and their 8 up rows
                f = w.m0 + lane / 4 * 8 + lane % 2 * 4;
                inside = f < a.F;
                f += (lane & 2) ? a.F : 0;
            }
            const uint8_t *scales = a.group_scales + (int64_t)w.e * a.groups * a.wide + (inside ? f : 0);
            for (int u = first, b = first / kUnits * per_stage; u < units; u += kUnits) {
                ok = mb_wait_warp(cempty + 8 * r.slot, r.phase ^ 1u, gave_up);
                if (!ok) break;
                const uint32_t bar = cfull + 8 * r.slot;
                if (elect_one()) {
                    mb_expect_tx(bar, kCodes);
                    if constexpr (kGated)
                        tma_load_5d(smem + r.slot * kCodes, &map_w, bar, u * (kK / 2), 0, 0, w.m0 / 8, w.e);
                    else
                        tma_load_3d(smem + r.slot * kCodes, &map_w, bar, u * (kK / 2), w.m0, w.e);
                }
                __syncwarp();
                const uint32_t to = scales_at + r.slot * kScales + lane * 4;
                for (int i = 0; i < per_stage; ++i, ++b) {
                    const bool there = inside && b < a.groups;
                    copy_async<4>(to + i * kM, scales + (there ? (int64_t)b * a.wide : 0), there ? 4 : 0);
                }
                copy_arrive(bar);
                r.next();
            }
        }
        drain_ring(cfull, r);  // nothing may still be landing here when the block ends
    } else if (warp == kRowWarp) {
        Ring<kRowSlots> r;
        int e = 0;
        bool ok = true;
        for (int t = tile0; t < tiles && ok; t += tile_step) {
            const Tile w = get_tile<kTok>(g, a.E, e, t, kStep);
            e = w.e;
            const int n = mma_tokens(w.n);
            for (int u = first; u < units; ++u) {
                ok = mb_wait_warp(empty + 8 * r.slot, r.phase ^ 1u, gave_up);
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t bar = full + 8 * r.slot;
                    mb_expect_tx(bar, 2 * n * 128);
                    uint32_t dst = rows_at + r.slot * kRows;
                    int row = w.row;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int box = 128 >> i;
                        if (n & box) {
                            tma_load_2d(dst, &map_x.m[i], bar, u * kK, row);
                            tma_load_2d(dst + S::kHalf, &map_x.m[i], bar, u * kK + kK / 2, row);
                            dst += box * 128;
                            row += box;
                        }
                    }
                }
                __syncwarp();
                r.next();
            }
        }
        drain_ring(full, r);
    } else if (warp == kMmaWarp) {
        // An mma of few tokens takes 33 cycles, a commit 87 to issue and a wait some 60: what is
        // between the eight mma of a unit is kept short.
        Ring<kSlots> r;  // of weights in TMEM
        Ring<kRowSlots> x;
        Ring<2> acc;
        int e = 0;
        bool ok = true;
        for (int t = tile0; t < tiles && ok; t += tile_step) {
            const Tile w = get_tile<kTok>(g, a.E, e, t, kStep);
            e = w.e;
            const uint32_t desc = mma_desc(1, false, false, kM, mma_tokens(w.n));
            for (int u0 = first; u0 < units && ok; u0 += part) {
                const uint32_t d = tmem + acc.slot * kTok;
                ok = mb_wait_warp(tempty + 8 * acc.slot, acc.phase ^ 1u, gave_up);
                for (int u = u0; u < min(u0 + part, units) && ok; ++u) {
                    ok = mb_wait_warp(full + 8 * x.slot, x.phase, gave_up);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t db = smem_operand(rows_at + x.slot * kRows, 16, 1024);
                        const uint32_t da = a_at + r.slot * (kK / 2);
#pragma unroll
                        for (int i = 0; i < kK / 16; ++i)
                            mma_bf16_tmem(d, da + i * 8, db + (i / 4 * (S::kHalf / 16) + i % 4 * 2), desc, u != u0 || i != 0);
                        tc_commit(empty + 8 * x.slot);
                    }
                    __syncwarp();
                    r.next();
                    x.next();
                }
                if (elect_one()) tc_commit(tfull + 8 * acc.slot);
                __syncwarp();
                acc.next();
            }
        }
        if (elect_one()) tc_commit(done);  // after every arrival before it
        __syncwarp();
        mb_drain(done, 0);
    } else if (warp < kDequantWarps) {
        // A thread has one matrix row; the sets take units by turns.
        constexpr int kSets = S::kSets, kChunks = kK / 32;
        const int quarter = warp & 3, set = warp >> 2, row = quarter * 32 + lane;
        const uint32_t magic = w4_magic(), line = smem + row * 128, at = a_at + ((uint32_t)(quarter * 32) << 16);
        Ring<kCodeStages> c;
        Ring<kSlots> r;     // of the next unit: its slot of TMEM
        Ring<kRowSlots> x;  // and its barriers, where they are not the same
        constexpr bool kSame = kSlots == kRowSlots;
        auto next_unit = [&] {
            r.next();
            if constexpr (!kSame) x.next();
        };
        bool ok = true;
        int turn = 0;       // the set that takes it
        for (int t = tile0; t < tiles && ok; t += tile_step) {
            for (int u0 = first; u0 < units && ok; u0 += kUnits) {
                const int n = min(kUnits, units - u0);
                const int mine = (set - turn) & (kSets - 1);  // this set's unit of the stage, if below n
                turn = (turn + n) & (kSets - 1);
                // a set without a unit waits as well: its arrival must not run ahead into the slot's next use
                ok = mb_wait_warp(cfull + 8 * c.slot, c.phase, gave_up);
                if (!ok) break;
                if (mine < n) {
                    if (mine) next_unit();
                    const uint32_t codes = line + c.slot * kCodes, scales = scales_at + c.slot * kScales + row;
                    const uint32_t to = at + r.slot * (kK / 2);
                    uint4 q[kChunks];
                    uint32_t code[kChunks];
#pragma unroll
                    for (int h = 0; h < kChunks; ++h) {  // 32 codes: 16 bytes, of one group
                        const int chunk = mine * kChunks + h;
                        q[h] = ld_shared128(codes + ((chunk ^ (row & 7)) << 4));
                        code[h] = ld_shared8(scales + (chunk >> (a.group_shift - 5)) * kM);
                    }
                    W4Scales two(0);
                    static_assert(kChunks % 2 == 0);
                    uint32_t loaded = 0;
#pragma unroll
                    for (int h = 0; h < kChunks; ++h) loaded ^= q[h].x ^ code[h];
                    if (lane == reader_lane(loaded)) mb_arrive(cempty + 8 * c.slot);
#pragma unroll
                    for (int h = 0; h < kChunks; ++h) {
                        if (h % 2 == 0) two = W4Scales(code[h] | code[h + 1] << 8);
                        const W4Scale s = h % 2 == 0 ? two.first : two.second;
                        uint32_t out[16];
                        dequant8(q[h].x, s, magic, out);
                        dequant8(q[h].y, s, magic, out + 4);
                        dequant8(q[h].z, s, magic, out + 8);
                        dequant8(q[h].w, s, magic, out + 12);
                        if (h == 0) {
                            // the unit that had the slot before: kSlots units ago
                            if constexpr (kSame) {
                                ok = mb_wait_warp(empty + 8 * r.slot, r.phase ^ 1u, gave_up);
                            } else {
                                const int b = x.slot - kSlots;
                                ok = mb_wait_warp(empty + 8 * (b < 0 ? b + kRowSlots : b), x.phase ^ (b < 0), gave_up);
                            }
                            if (!ok) break;
                            tc_fence_after();
                        }
                        tmem_store16(to + h * 16, out);
                    }
                    if (!ok) break;
                    tmem_store_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mb_arrive(full + 8 * (kSame ? r.slot : x.slot));
                    if (mine == 0 && n == 2) next_unit();
                    next_unit();
                } else {
                    if (lane == 0) mb_arrive(cempty + 8 * c.slot);
                    if (n == 2) next_unit();
                    next_unit();
                }
                c.next();
            }
        }
    } else if (warp < kCodeWarp) {
        // Results: warp w holds matrix rows 32 (w % 4).. of the tile, one per lane, and every other 32 tokens.
        if constexpr (kParts) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kStoreRegs));
        if constexpr (kSplit) cluster_wait();
        const int quarter = warp & 3, half = (warp - kStoreFirst) >> 2;
        const uint32_t buf = bufs_at + (warp - kStoreFirst) * kBuf;
        const int fl = kGated ? (lane >> 4) * 8 + (lane & 7) : lane, up = (lane >> 3) & 1;
        auto store = [&](const Tile &w, int c0, float scale, auto v) {
            const int left = w.n - c0;
            if constexpr (kF32) {  // one token's 32 features are 128 bytes
#pragma unroll
                for (int j = 0; j < 32; ++j) st_shared32(buf + j * 128 + lane * 4, __float_as_uint(v(j) * scale));
                __syncwarp();
                const int f = w.m0 + quarter * 32 + lane % 8 * 4;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int tok = q * 4 + lane / 8;
                    const uint4 o = ld_shared128(buf + q * 512 + lane * 16);
                    if (tok < left && f < a.F)
                        *reinterpret_cast<uint4 *>(static_cast<float *>(a.y) + (int64_t)(w.row + c0 + tok) * a.F + f) = o;
                }
            } else if constexpr (kGated) {
                // lanes with bit 3 clear hold gate rows, the others the up
                // rows of the same features; of a pair of tokens each half of
                // the lanes finishes one
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float one = v(j) * scale, two = v(j + 1) * scale;
                    const float got = __shfl_xor_sync(0xffffffffu, up ? one : two, 8);
                    const float h = silu_mul(up ? got : one, up ? two : got);
                    st_shared16(buf + (j + up) * 32 + fl * 2, bf16x2(__float_as_uint(h), 0u));
                }
                __syncwarp();
                const int f = w.m0 + quarter * 16 + (lane & 1) * 8;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int tok = i * 16 + lane / 2;
                    const uint4 o = ld_shared128(buf + i * 512 + lane * 16);
                    if (tok < left && f < a.F)
                        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.y) + (int64_t)(w.row + c0 + tok) * a.F + f) = o;
                }
            } else {  // one token's 32 features are 64 bytes
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const uint32_t two = bf16x2(__float_as_uint(v(j) * scale), __float_as_uint(v(j + 1) * scale));
                    st_shared16(buf + j * 64 + lane * 2, two);
                    st_shared16(buf + (j + 1) * 64 + lane * 2, two >> 16);
                }
                __syncwarp();
                const int f = w.m0 + quarter * 32 + lane % 4 * 8;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = i * 8 + lane / 4;
                    const uint4 o = ld_shared128(buf + i * 512 + lane * 16);
                    if (tok < left && f < a.F)
                        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.y) + (int64_t)(w.row + c0 + tok) * a.F + f) = o;
                }
            }
            __syncwarp();
        };
        // Joins the blocks' sums of 32 tokens, v(0) to v(31): the owner of the quarter gets them all, the others give
        // theirs.  A block's sums leave for the owner's memory once what it gave before has been read.
        const int me = warp - kStoreFirst, owner = quarter & (split - 1);
        uint32_t given = 0;  // parity of the next join
        auto join = [&](float (&v)[32]) {
            const uint32_t slot = join_at + ((quarter >> shift) * 2 + half) * (split - 1) * 4096 + lane * 16;
            if (rank != owner) {
                if (!mb_wait_warp_pair(jfree + 8 * me, given ^ 1u, gave_up, kPolls + all * kStepPolls)) return false;
                const uint32_t to = at_rank(slot + (rank - (rank > owner)) * 4096, owner), bar = at_rank(jfull + 8 * me, owner);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    st_async128(to + j * 512, make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]), bar);
            } else {
                if (lane == 0) mb_expect_tx(jfull + 8 * me, (split - 1) * 4096);
                __syncwarp();
                if (!mb_wait_warp_pair(jfull + 8 * me, given, gave_up, kPolls + all * kStepPolls)) return false;
                for (int b = 0; b < split - 1; ++b) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint4 o = ld_shared128(slot + b * 4096 + j * 512);
                        v[4 * j] += __uint_as_float(o.x);
                        v[4 * j + 1] += __uint_as_float(o.y);
                        v[4 * j + 2] += __uint_as_float(o.z);
                        v[4 * j + 3] += __uint_as_float(o.w);
                    }
                }
            }
            given ^= 1u;
            return true;
        };
        auto joined = [&] {  // what the others gave is stored: they may give again
            if (rank == owner && lane < split && lane != rank) mb_arrive_remote_relaxed(at_rank(jfree + 8 * me, lane));
        };
        Ring<2> acc;
        int e = 0;
        bool ok = true;
        for (int t = tile0; t < tiles && ok; t += tile_step) {
            const Tile w = get_tile<kTok>(g, a.E, e, t, kStep);
            e = w.e;
            const int f = w.m0 + quarter * (kGated ? 16 : 32) + fl;
            const float scale =
                f < a.F ? __ldg(a.row_scales + (int64_t)w.e * a.wide + f + (kGated && up ? a.F : 0)) : 0.f;
            const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + 32 * half;
            if constexpr (kParts) {
                float sum[kTok / 64][32];
#pragma unroll
                for (int i = 0; i < kTok / 64; ++i)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[i][j] = 0.f;
                for (int u0 = first; u0 < units; u0 += part) {
                    ok = mb_wait_warp(tfull + 8 * acc.slot, acc.phase, gave_up, kPolls + part * kStepPolls);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < kTok / 64; ++i) {
                        if (64 * i + 32 * half < w.n) {
                            uint32_t v[32];
                            tmem_load32(src + acc.slot * kTok + 64 * i, v);
#pragma unroll
                            for (int j = 0; j < 32; ++j) sum[i][j] += __uint_as_float(v[j]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mb_arrive(tempty + 8 * acc.slot);
                    acc.next();
                }
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < kTok / 64; ++i) {
                    if (64 * i + 32 * half >= w.n) continue;
                    if constexpr (kSplit) {
                        ok = join(sum[i]);
                        if (!ok || rank != owner) break;
                    }
                    store(w, 64 * i + 32 * half, scale, [&](int j) { return sum[i][j]; });
                    if constexpr (kSplit) joined();
                }
            } else {  // straight from TMEM
                ok = mb_wait_warp(tfull + 8 * acc.slot, acc.phase, gave_up, kPolls + units * kStepPolls);
                if (!ok) break;
                tc_fence_after();
                if constexpr (kSplit) {
                    float v[32];
                    const bool some = 32 * half < w.n;
                    if (some) tmem_load32(src + acc.slot * kTok, reinterpret_cast<uint32_t *>(v));
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mb_arrive(tempty + 8 * acc.slot);
                    acc.next();
                    if (!some) continue;
                    ok = join(v);
                    if (!ok) break;
                    if (rank == owner) {
                        store(w, 32 * half, scale, [&](int j) { return v[j]; });
                        joined();
                    }
                } else {
                    for (int c0 = 0; 32 * half + c0 < w.n; c0 += 64) {
                        uint32_t v[32];
                        tmem_load32(src + acc.slot * kTok + c0, v);
                        store(w, c0 + 32 * half, scale, [&](int j) { return __uint_as_float(v[j]); });
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mb_arrive(tempty + 8 * acc.slot);
                    acc.next();
                }
            }
        }
        // The owner's last arrival must not come after this block is gone, nor this block's sums after the owner is.
        if (kSplit && ok && rank != owner) mb_wait_warp(jfree + 8 * me, given ^ 1u, gave_up, kPolls + all * kStepPolls);
    }
    __syncwarp();
    tc_fence_before();
    if constexpr (kSplit) {
        if (*gave_up) __nanosleep(100000);  // sums that left before it did have landed by then
        __syncwarp();
        if (warp < kStoreFirst || warp >= kCodeWarp) cluster_wait();
        cluster_sync();  // no block leaves while another may reach it
    } else {
        __syncthreads();
    }
    tc_fence_after();
    if (tid == 0 && s_gave_up) record_timeout();
    if (warp == kMmaWarp) tmem_free(tmem, 512);
}

template <int kTok, bool kGated, bool kParts, bool kF32>
cudaError_t launch(const CUtensorMap &map_w, const TokenMaps &map_x, const Args &a, cudaStream_t stream) {
    auto kern = expert_w4_kernel<kTok, kGated, kParts, kF32, false>;
    using S = Shape<kTok, kParts, kF32, false>;
    static_assert(S::kSmem + groups_bytes(1024) <= most_shared_w4(S::kBars));
    static thread_local AttrCache attr;
    cudaError_t e = attr.allow_smem(reinterpret_cast<const void *>(kern), S::kSmem + groups_bytes(1024));
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute pdl[1] = {pdl_attribute()};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)sm_count());
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem + groups_bytes(a.E);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, map_w, map_x, a);
}

template <bool kGated, bool kParts, bool kF32>
cudaError_t launch_split(const CUtensorMap &map_w, const TokenMaps &map_x, const Args &a, cudaStream_t stream) {
    auto kern = expert_w4_kernel<64, kGated, kParts, kF32, true>;
    using S = Shape<64, kParts, kF32, true>;
    static_assert(S::kSmem + groups_bytes(1024) <= most_shared_w4(S::kBars));
    static thread_local PairCache caches[2];
    PairLaunch l(S::kThreads, S::kSmem + groups_bytes(1024), stream);
    l.attr[1].val.clusterDim.x = a.split;
    l.cfg.gridDim = dim3(a.split);
    PairCache &cache = caches[a.split == 4];
    cudaError_t e = cache.prepare(reinterpret_cast<const void *>(kern), l.cfg);
    if (e != cudaSuccess) return e;
    l.cfg.gridDim = dim3((unsigned)(cache.blocks / 2 * a.split));  // it counts two blocks a cluster
    l.cfg.dynamicSmemBytes = S::kSmem + groups_bytes(a.E);
    return cudaLaunchKernelEx(&l.cfg, kern, map_w, map_x, a);
}

// kTok = 64 (alone or split), or the most that TMEM and the registers hold.
template <bool kGated, bool kParts, bool kF32>
cudaError_t launch_any(bool small, const CUtensorMap &map_w, const TokenMaps &map_x, const Args &a, cudaStream_t stream) {
    if (a.split > 1) return launch_split<kGated, kParts, kF32>(map_w, map_x, a, stream);
    return small ? launch<64, kGated, kParts, kF32>(map_w, map_x, a, stream)
                 : launch<kParts ? 128 : 160, kGated, kParts, kF32>(map_w, map_x, a, stream);
}

}  // namespace

cudaError_t launch_expert_gemm_w4(const ExpertRows &r, int K, int F, int gated, int group, const void *x,
                                  const void *wq, const void *group_scales, const float *row_scales, void *y, int y_f32,
                                  cudaStream_t stream) {
    const int sms = sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    const W4Form form = w4_form(r, K, F, gated, y_f32, sms);
    if (form.tokens == w4_few::kTok)
        return launch_expert_w4_few(r, K, F, gated, group, x, wq, group_scales, row_scales, y, y_f32, stream);
    const bool parts = w4_parts(K, gated, y_f32), small = form.tokens == 64;
    const int most = form.tokens;
    CUtensorMap map_w;
    TokenMaps map_x;
    if (!encode_w4(&map_w, wq, r.E, K, F, gated, kM)) return cudaErrorInvalidValue;
    const int64_t tok = r.most < most ? mma_tokens((int)r.most) : most;
    map_x.first = tok >= 128 ? 0 : tok >= 64 ? 1 : tok >= 32 ? 2 : 3;
    const uint64_t dims[2] = {(uint64_t)K, (uint64_t)r.rows_total}, stride = (uint64_t)K * 2;
    for (int i = map_x.first; i < 4; ++i) {
        const uint32_t box[2] = {kK / 2, 128u >> i};
        if (!encode_map(&map_x.m[i], 0, 2, x, dims, &stride, box)) return cudaErrorInvalidValue;
    }
    int shift = 5;
    while ((1 << shift) < group) ++shift;
    const Args a{r.offsets, static_cast<const uint8_t *>(group_scales), row_scales, y, r.cap, r.most, r.pairs,
                 r.E, r.L, K, F, gated ? 2 * F : F, K / group, shift, form.split};
    if (gated) return parts ? launch_any<true, true, false>(small, map_w, map_x, a, stream) : launch_any<true, false, false>(small, map_w, map_x, a, stream);
    if (y_f32) return launch_any<false, true, true>(small, map_w, map_x, a, stream);
    return parts ? launch_any<false, true, false>(small, map_w, map_x, a, stream) : launch_any<false, false, false>(small, map_w, map_x, a, stream);
}

cudaError_t take_expert_w4_error(int *err) { return take_tc_error(err); }

}  // namespace moe
