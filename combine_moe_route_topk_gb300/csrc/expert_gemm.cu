// Products of the experts in bf16, on the layout that dispatch writes: rows
// of expert e in its rank's receive region times the expert's matrix, and the
// gradient with respect to the rows.
//
//   linear   y[p][f]  = sum_k x[p][k] w[e][f][k]
//   gated    h[p][f]  = silu(g) u, g|u = sum_k x[p][k] w[e][f | F + f][k]
//   dgrad    dx[p][k] = sum_f dy[p][f] w[e][f][k]
//
// The matrix is the operand with 128 fixed rows of tcgen05.mma (M) and the
// expert's tokens are its columns (N), so a tile takes as many tokens as the
// expert has, rounded up to 32, up to 256: an expert with 20 rows pays for
// 32, and its matrix is read once.  Accumulators are f32 in TMEM, two of
// 128 x 256 so that a tile's results leave while the next one is computed.
// Blocks work in pairs: one tcgen05.mma of the pair multiplies 256 matrix
// rows by the tile's tokens, each block loading its 128 rows and half the
// tokens, which halves what the tokens cost in L2 and shared memory.
//
// The tensor core cuts what it adds off below the accumulator's last place, so
// a long sum comes out small, the more the longer it is.  For f32 results the sum
// is taken in parts of 512, which the storing warps add up in registers,
// rounding to nearest: 3e-7 off for any length where one accumulator was 3.5e-6
// off after 6144 elements.  bf16 results, which are off by up to 3.9e-3 from
// their rounding alone, are summed in one go up to kWhole elements and in parts
// of 2048 beyond (K = 28672, 4096 rows: 1145 us either way; 512 cost the gated
// form 4 %).
#include <cuda_bf16.h>

#include "expert_internal.cuh"
#include "pdl.cuh"
#include "tc_ops.cuh"

namespace moe {
namespace {

constexpr int kM = 128;        // matrix rows of a block's half of a tile
// Most tokens of a tile: 256, or 128 or 64 where all tiles then still run at
// once (E = 1, K = 7168, F = 4096: 256 rows 25.2 us against 36.3 with 256, 512
// rows 27.4 against 36.5; 32 never gained).
constexpr int kTokShift = 8, kLeastShift = 6, kTok = 1 << kTokShift;
constexpr int kK = 64;         // reduction elements of a stage: one 128-byte line
constexpr int kBytesA = kM * kK * 2;
constexpr int kBytesB = kTok / 2 * kK * 2;
constexpr int kStage = kBytesA + kBytesB;
constexpr int kStoreWarps = 8;
// Stages of a part of a sum: 512 elements for f32 results, 2048 for bf16.
constexpr int part_stages(bool f32) { return (f32 ? 512 : 2048) / kK; }

// Warps: those that store results, one that loads, one that issues mma; for
// sums in parts two more that only give their registers away (384 threads are
// launched with 168 each, the storing ones take 216, the others keep 72).
template <bool kParts, bool kF32>
struct Shape {
    static_assert(kParts || !kF32, "f32 results are summed in parts");
    static constexpr int kThreads = 32 * (kStoreWarps + (kParts ? 4 : 2)), kStages = kF32 ? 5 : 6;
    static constexpr int kBuf = kF32 ? 4096 : 2048;  // each storing warp's: 32 tokens' results, to be written as whole sectors
    static constexpr int kSmem = 1024 + kStages * kStage + kStoreWarps * kBuf;
};

enum Form { kLinear, kGated, kDgrad };

struct Args {
    const int32_t *offsets;
    void *y;
    __nv_bfloat16 *pre;
    int64_t cap, most, pairs;
    int E, L, K, F;  // reduction length, result columns
};

__device__ __forceinline__ int token_tiles(int count, int shift) { return (count + (1 << shift) - 1) >> shift; }

// N of a pair's mma is a multiple of 32.
__host__ __device__ inline int mma_tokens(int n) { return (n + 31) & ~31; }

__device__ __forceinline__ int tile_tokens(int count, int shift) {
    return mma_tokens(tile_rows(count, token_tiles(count, shift)));
}

// Larger tiles come first (make_groups sorts by the size), so that a round's
// tiles are alike and the last round has the smallest: 32 experts of 440 to
// 560 rows, tiles of 192 or 256 tokens, K = 2048, F = 4096, take 195 us against
// 204 in the experts' own order (197 without the turns).  64 experts of 128
// rows, bound by HBM, lose 0.3 %.
//
// The tiles of a pair: one of each round of all pairs, which take them in
// ascending order or, where the tiles get smaller from round to round, in
// ascending and descending order by turns.
struct Turns {
    int t, step;
    __device__ __forceinline__ explicit Turns(const Groups &g)
        : t(blockIdx.x / 2), step(g.sorted ? gridDim.x - 1 - 2 * t : gridDim.x / 2) {}
    __device__ __forceinline__ operator int() const { return t; }
    __device__ __forceinline__ void next() {
        t += step;
        step = gridDim.x - step;
    }
};

struct Tile {
    int i, e, m0, row, n;  // place of the group, group, first matrix row (or feature), first token row, tokens
};

// Tiles of a group: its token tiles (of equal size, so that no tile is left
// with a few rows) run fastest, so that blocks working at the same time share
// the matrix rows through L2.
__device__ __forceinline__ Tile get_tile(const Groups &g, int E, int i, int t, int m_step) {
    Tile r;
    r.i = same(find_group(g, E, i, t));
    r.e = same(g.order[r.i]);
    const int c = same(g.count[r.e]), nt = token_tiles(c, g.shift), at = t - same(g.prefix[r.i]);
    const int size = tile_tokens(c, g.shift);
    const int tt = at % nt;
    r.m0 = at / nt * m_step;
    r.row = same(g.row[r.e]) + tt * size;
    r.n = min(size, c - tt * size);
    return r;
}

template <int kForm, bool kParts, bool kF32, bool kSave>
__global__ void __launch_bounds__(Shape<kParts, kF32>::kThreads, 1)
expert_gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ RowMaps map_x, const Args a) {
    constexpr int kStages = Shape<kParts, kF32>::kStages, kBuf = Shape<kParts, kF32>::kBuf;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long bars[2 * kStages + 5];
    __shared__ uint32_t s_tmem;
    __shared__ int s_gave_up;
    const int tid = threadIdx.x, warp = same(tid / 32), lane = tid % 32;
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t buf = smem + kStages * kStage + (warp & (kStoreWarps - 1)) * kBuf;
    int *tables = reinterpret_cast<int *>(smem_raw + (smem - smem_u32(smem_raw)) + kStages * kStage + kStoreWarps * kBuf);
    const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, tfull = empty + 8 * kStages,
                   tempty = tfull + 16, done = tempty + 16;
    volatile int *gave_up = &s_gave_up;

    const int rank = same((int)cluster_rank());
    if (warp == kStoreWarps) tmem_alloc_pair(smem_u32(&s_tmem), 512);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mb_init(full + 8 * i, 1);
            mb_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mb_init(tfull + 8 * i, 1);
            mb_init(tempty + 8 * i, 2 * kStoreWarps);  // the storing warps of both blocks
        }
        mb_init(done, 1);
        s_gave_up = 0;
        mb_init_fence();
        tma_prefetch_map(&map_w);
        prefetch_maps(map_x);
    }
    tc_fence_before();
    cluster_sync();  // barriers and TMEM of both blocks are ready
    tc_fence_after();
    const uint32_t tmem = (uint32_t)same((int)s_tmem);
    grid_dependency_wait();  // offsets and rows come from earlier kernels
    grid_launch_dependents();
    constexpr int kHalf = kForm == kGated ? kM / 2 : kM;  // result columns of a block
    constexpr int kStep = 2 * kHalf;
    const int m_tiles = (a.F + kStep - 1) / kStep;
    const Groups g = make_groups<kTokShift, kLeastShift, kTok / 32 + 1>(
        tables, a.offsets, a.E, a.L, a.cap, a.most, a.pairs, gridDim.x / 2,
        [&](int c, int shift) { return token_tiles(c, shift) * m_tiles; },
        [](int c) { return c == 0 ? kTok / 32 : (kTok - tile_tokens(c, kTokShift)) / 32; });  // syncs the block
    const int tiles = same(g.prefix[a.E]), steps = (a.K + kK - 1) / kK;
    const int part = kParts ? part_stages(kF32) : steps;  // stages that are summed in TMEM
    if constexpr (kParts) {
        if (warp >= kStoreWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    }

    if (warp == kStoreWarps) {  // loads
        Ring<kStages> r;
        int i = 0;
        bool ok = true;
        for (Turns t(g); t < tiles && ok; t.next()) {
            const Tile w = get_tile(g, a.E, i, t, kStep);
            i = w.i;
            const int m0 = w.m0 + rank * kHalf, half = mma_tokens(w.n) / 2;  // this block's share
            const int row = w.row + rank * half;
            for (int k = 0; k < steps; ++k) {
                ok = mb_wait_warp(empty + 8 * r.slot, r.phase ^ 1u, gave_up);
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t bar = at_leader(full + 8 * r.slot), sa = smem + r.slot * kStage, sb = sa + kBytesA;
                    if (rank == 0) mb_expect_tx(full + 8 * r.slot, 2 * (kBytesA + rows_loaded(half) * 128));
                    if constexpr (kForm == kLinear) {
                        tma_load_3d_pair(sa, &map_w, bar, k * kK, m0, w.e);
                    } else if constexpr (kForm == kGated) {
                        tma_load_5d_pair(sa, &map_w, bar, k * kK, 0, 0, m0 / 8, w.e);
                    } else {
                        tma_load_3d_pair(sa, &map_w, bar, m0, k * kK, w.e);
                        tma_load_3d_pair(sa + kBytesA / 2, &map_w, bar, m0 + 64, k * kK, w.e);
                    }
                    load_rows_pair(sb, map_x, bar, k * kK, row, half);
                }
                __syncwarp();
                r.next();
            }
        }
        if (rank == 0) drain_ring(full, r);  // of both blocks
        drain_ring(empty, r);  // in each block: its loads, and the leader's arrivals, the last of them `done`
        mb_drain(done, 0);
    } else if (warp == kStoreWarps + 1) {  // mma
        if (rank == 0) {
            Ring<kStages> r;
            Ring<2> acc;
            int i = 0;
            bool ok = true;
            for (Turns t(g); t < tiles && ok; t.next()) {
                const Tile w = get_tile(g, a.E, i, t, kStep);
                i = w.i;
                const uint32_t desc = mma_desc(1, kForm == kDgrad, false, 2 * kM, mma_tokens(w.n));
                for (int k0 = 0; k0 < steps && ok; k0 += part) {
                    const uint32_t d = tmem + acc.slot * kTok;
                    ok = mb_wait_warp(tempty + 8 * acc.slot, acc.phase ^ 1u, gave_up);
                    tc_fence_after();
                    for (int k = k0; k < min(k0 + part, steps) && ok; ++k) {
                        ok = mb_wait_warp(full + 8 * r.slot, r.phase, gave_up);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint32_t sa = smem + r.slot * kStage;
                            // reduction contiguous: 16 elements are 32 bytes
                            // of the line; else they are 16 lines
                            const uint64_t da = kForm == kDgrad ? smem_operand(sa, kBytesA / 2, 1024)
                                                                : smem_operand(sa, 16, 1024);
                            const uint64_t db = smem_operand(sa + kBytesA, 16, 1024);
                            constexpr int kStepA = kForm == kDgrad ? 2048 / 16 : 32 / 16;
#pragma unroll
                            for (int i = 0; i < kK / 16; ++i)
                                mma_bf16_pair(d, da + i * kStepA, db + i * 2, desc, k != k0 || i != 0);
                            tc_commit_pair(empty + 8 * r.slot);
                        }
                        __syncwarp();
                        r.next();
                    }
                    if (elect_one()) tc_commit_pair(tfull + 8 * acc.slot);
                    __syncwarp();
                    acc.next();
                }
            }
            if (elect_one()) tc_commit_pair(done);
            __syncwarp();
            mb_drain(done, 0);
        }
    } else if (warp < kStoreWarps) {
        // results: warp w holds matrix rows 32 (w % 4).. of the block's half,
        // one per lane, and every other 32 tokens, 2 i + w / 4.  (Four warps,
        // each with all tokens, took 8.7 us for 222 rows of K = 1000, F = 776
        // with pre kept, eight take 8.4.)
        if constexpr (kParts) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int quarter = warp & 3, half = warp >> 2;
        // The lane's sums of tokens c0.. of a tile, v(0) to v(31) as bits, are
        // finished, turned in shared memory and stored.
        auto store = [&](const Tile &w, int c0, auto v) {
            const int left = w.n - c0;
            if constexpr (kF32) {  // one token's 32 features are 128 bytes
#pragma unroll
                for (int j = 0; j < 32; ++j) st_shared32(buf + j * 128 + lane * 4, v(j));
                __syncwarp();
                const int f = w.m0 + rank * kHalf + quarter * 32 + lane % 8 * 4;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int tok = q * 4 + lane / 8;
                    const uint4 r = ld_shared128(buf + q * 512 + lane * 16);
                    if (tok < left && f < a.F)
                        *reinterpret_cast<uint4 *>(static_cast<float *>(a.y) + (int64_t)(w.row + c0 + tok) * a.F + f) = r;
                }
            } else if constexpr (kForm == kGated) {
                // lanes with bit 3 clear hold gate rows, the others the
                // up rows of the same features; of a pair of tokens each
                // half of the lanes finishes one
                const int fl = (lane >> 4) * 8 + (lane & 7), up = (lane >> 3) & 1;
                const int f0 = w.m0 + rank * kHalf + quarter * 16;
                if constexpr (kSave) {
                    const uint32_t to = buf + up * 32 + fl * 2;
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const uint32_t two = bf16x2(v(j), v(j + 1));
                        st_shared16(to + j * 64, two);
                        st_shared16(to + j * 64 + 64, two >> 16);
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = i * 8 + lane / 4, which = (lane >> 1) & 1, f = f0 + (lane & 1) * 8;
                        const uint4 q = ld_shared128(buf + i * 512 + lane * 16);
                        if (tok < left && f < a.F)
                            *reinterpret_cast<uint4 *>(a.pre + ((int64_t)(w.row + c0 + tok) * 2 + which) * a.F + f) = q;
                    }
                    __syncwarp();
                }
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? v(j) : v(j + 1), 8);
                    const float gate = __uint_as_float(up ? got : v(j)), lin = __uint_as_float(up ? v(j + 1) : got);
                    const float h = silu_mul(gate, lin);
                    st_shared16(buf + (j + up) * 32 + fl * 2, bf16x2(__float_as_uint(h), 0u));
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int tok = i * 16 + lane / 2, f = f0 + (lane & 1) * 8;
                    const uint4 q = ld_shared128(buf + i * 512 + lane * 16);
                    if (tok < left && f < a.F)
                        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.y) + (int64_t)(w.row + c0 + tok) * a.F + f) = q;
                }
            } else {  // one token's 32 features are 64 bytes
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const uint32_t two = bf16x2(v(j), v(j + 1));
                    st_shared16(buf + j * 64 + lane * 2, two);
                    st_shared16(buf + (j + 1) * 64 + lane * 2, two >> 16);
                }
                __syncwarp();
                const int f = w.m0 + rank * kHalf + quarter * 32 + lane % 4 * 8;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = i * 8 + lane / 4;
                    const uint4 q = ld_shared128(buf + i * 512 + lane * 16);
                    if (tok < left && f < a.F)
                        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.y) + (int64_t)(w.row + c0 + tok) * a.F + f) = q;
                }
            }
            __syncwarp();
        };
        Ring<2> acc;
        int i = 0;
        bool ok = true;
        for (Turns t(g); t < tiles && ok; t.next()) {
            const Tile w = get_tile(g, a.E, i, t, kStep);
            i = w.i;
            if constexpr (kParts) {
                float sum[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[i][j] = 0.f;
                for (int k0 = 0; k0 < steps; k0 += part) {
                    ok = mb_wait_warp(tfull + 8 * acc.slot, acc.phase, gave_up, kPolls + part * kStepPolls);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t src = tmem + acc.slot * kTok + ((uint32_t)(quarter * 32) << 16) + 32 * half;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (64 * i + 32 * half < w.n) {
                            uint32_t v[32];
                            tmem_load32(src + 64 * i, v);
#pragma unroll
                            for (int j = 0; j < 32; ++j) sum[i][j] += __uint_as_float(v[j]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mb_arrive_remote_relaxed(at_leader(tempty + 8 * acc.slot));
                    acc.next();
                }
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (64 * i + 32 * half < w.n)
                        store(w, 64 * i + 32 * half, [&](int j) { return __float_as_uint(sum[i][j]); });
                }
            } else {  // straight from TMEM
                ok = mb_wait_warp(tfull + 8 * acc.slot, acc.phase, gave_up, kPolls + steps * kStepPolls);
                if (!ok) break;
                tc_fence_after();
                const uint32_t src = tmem + acc.slot * kTok + ((uint32_t)(quarter * 32) << 16);
                for (int c0 = 32 * half; c0 < w.n; c0 += 64) {
                    uint32_t v[32];
                    tmem_load32(src + c0, v);
                    store(w, c0, [&](int j) { return v[j]; });
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mb_arrive_remote_relaxed(at_leader(tempty + 8 * acc.slot));
                acc.next();
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();  // neither block leaves, or frees TMEM, while the other may reach it
    tc_fence_after();
    if (tid == 0 && s_gave_up) record_timeout();
    if (warp == kStoreWarps) tmem_free_pair(tmem, 512);
}

template <int kForm, bool kParts, bool kF32 = false, bool kSave = false>
cudaError_t launch(const CUtensorMap &map_w, const RowMaps &map_x, const Args &a, cudaStream_t stream) {
    auto kern = expert_gemm_kernel<kForm, kParts, kF32, kSave>;
    static thread_local PairCache cache;
    using S = Shape<kParts, kF32>;
    PairLaunch l(S::kThreads, S::kSmem + groups_bytes(1024, true), stream);
    cudaError_t e = cache.prepare(reinterpret_cast<const void *>(kern), l.cfg);
    if (e != cudaSuccess) return e;
    l.cfg.gridDim = dim3((unsigned)cache.blocks);
    l.cfg.dynamicSmemBytes = S::kSmem + groups_bytes(a.E, true);
    return cudaLaunchKernelEx(&l.cfg, kern, map_w, map_x, a);
}

// Most tokens that a block loads: half a pair's.
int64_t half_tile(const ExpertRows &r) { return (r.most < kTok ? mma_tokens((int)r.most) : kTok) / 2; }

}  // namespace

cudaError_t launch_expert_gemm(const ExpertRows &r, int K, int F, int gated, const void *x, const void *w, void *y,
                               int y_f32, void *pre, cudaStream_t stream) {
    CUtensorMap map_w;
    RowMaps map_x;
    const uint64_t row = (uint64_t)K * 2;
    if (gated) {  // per feature block of 8: 8 gate rows, then its 8 up rows
        const uint64_t dims[5] = {(uint64_t)K, 8, 2, (uint64_t)F / 8, (uint64_t)r.E};
        const uint64_t strides[4] = {row, row * F, row * 8, row * F * 2};
        const uint32_t box[5] = {kK, 8, 2, kM / 16, 1};
        if (!encode_map(&map_w, 0, 5, w, dims, strides, box)) return cudaErrorInvalidValue;
    } else {
        const uint64_t dims[3] = {(uint64_t)K, (uint64_t)F, (uint64_t)r.E};
        const uint64_t strides[2] = {row, row * F};
        const uint32_t box[3] = {kK, kM, 1};
        if (!encode_map(&map_w, 0, 3, w, dims, strides, box)) return cudaErrorInvalidValue;
    }
    if (!encode_rows(&map_x, 0, x, K, r.rows_total, half_tile(r))) return cudaErrorInvalidValue;
    const Args a{r.offsets, y, static_cast<__nv_bfloat16 *>(pre), r.cap, r.most, r.pairs, r.E, r.L, K, F};
    const bool parts = K > kWhole;
    if (gated && pre) return parts ? launch<kGated, true, false, true>(map_w, map_x, a, stream)
                                   : launch<kGated, false, false, true>(map_w, map_x, a, stream);
    if (gated) return parts ? launch<kGated, true>(map_w, map_x, a, stream) : launch<kGated, false>(map_w, map_x, a, stream);
    if (y_f32) return launch<kLinear, true, true>(map_w, map_x, a, stream);
    return parts ? launch<kLinear, true>(map_w, map_x, a, stream) : launch<kLinear, false>(map_w, map_x, a, stream);
}

cudaError_t launch_expert_dgrad(const ExpertRows &r, int K, int F, const void *dy, const void *w, void *dx,
                                cudaStream_t stream) {
    CUtensorMap map_w;
    RowMaps map_x;
    const uint64_t wdims[3] = {(uint64_t)K, (uint64_t)F, (uint64_t)r.E};
    const uint64_t strides[2] = {(uint64_t)K * 2, (uint64_t)K * 2 * F};
    const uint32_t wbox[3] = {64, kK, 1};
    if (!encode_map(&map_w, 0, 3, w, wdims, strides, wbox)) return cudaErrorInvalidValue;
    if (!encode_rows(&map_x, 0, dy, F, r.rows_total, half_tile(r))) return cudaErrorInvalidValue;
    const Args a{r.offsets, dx, nullptr, r.cap, r.most, r.pairs, r.E, r.L, F, K};
    return F > kWhole ? launch<kDgrad, true>(map_w, map_x, a, stream) : launch<kDgrad, false>(map_w, map_x, a, stream);
}

cudaError_t take_expert_gemm_error(int *err) { return take_tc_error(err); }

}  // namespace moe
