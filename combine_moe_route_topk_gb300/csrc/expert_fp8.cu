// Products of the experts in fp8 with block scales, on the rows that the
// quantising dispatch writes:
//
//   y[p][f] = sum_b sx[p][b] sw[e][f / 128][b] sum_{k in block b} xq[p][k] wq[e][f][k]
//
// or the gated pair silu(g) u of two such products, quantised again (per 128
// features of a row: scale = amax / 448, code = e4m3(h / scale), the format
// the next product reads).
//
// The scales are arbitrary f32 numbers, so the tensor core sums one block of
// 128 at a time (four tcgen05.mma of 32, f32 in TMEM, two buffers) and eight
// warps add the blocks up in f32 registers: acc += (sx sw) * block.  Here the
// tokens are M, unlike in the bf16 product: a TMEM lane, hence a thread, is
// then one token, its factor is one register per block of the matrix, and
// the largest magnitude of a requantised row needs no exchange between lanes.
// With the matrix rows as M the factors of 16 columns came from shared
// memory for every 16 sums, which cost as much as the sums (2048 tokens, K =
// F = 2048, gated: 143 us against 103 without those loads).  A tile is up to
// 128 tokens by two blocks of 128 matrix rows: the gate and the up rows of
// the same features, or neighbours.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "expert_internal.cuh"
#include "pdl.cuh"
#include "tc_ops.cuh"

namespace moe {
namespace {

constexpr int kTok = 128;   // tokens of a tile (M)
constexpr int kBlk = 128;   // matrix rows of a block: one scale
constexpr int kN = 2 * kBlk;
constexpr int kK = 128;     // reduction elements of a stage: one scale block, one 128-byte line
constexpr int kStages = 4;
constexpr int kBytesA = kTok * kK;
constexpr int kBytesB = kN * kK;
constexpr int kStage = kBytesA + kBytesB;
constexpr int kGroup = 4;   // blocks whose scales are loaded together
constexpr int kSumWarps = 8;
constexpr int kThreads = 32 * (kSumWarps + 4);  // one warp loads, one issues mma, two bring the scales
// 384 threads are launched with 168 registers each; the summing warps take
// 216 (linear form: 224), the others keep 72 (56): 256 * 216 + 128 * 72 = 256 *
// 224 + 128 * 56 = 384 * 168.  With these splits neither form spills; with the
// other's it does (linear at 216: 86 us where 224 takes 72).
constexpr int sum_regs(bool gated) { return gated ? 216 : 224; }
constexpr int other_regs(bool gated) { return gated ? 72 : 56; }
constexpr int kBuf = 2048;  // each summing warp's: 64 bytes of its 32 tokens' results
constexpr int kSmem = 1024 + kStages * kStage + kSumWarps * kBuf;

struct Args {
    const int32_t *offsets;
    const float *x_scales, *w_scales;
    void *y;
    float *y_scales;
    int64_t cap, most, pairs;
    int E, L, K, F, w_rows;  // reduction length, result columns, matrix rows of an expert
};

__host__ __device__ inline int token_tiles(int count) { return (count + kTok - 1) / kTok; }

struct Tile {
    int e, f0, row, n;  // group, first result column, first token row, tokens
};

// Token tiles of a group (of equal size) run fastest: blocks working at the
// same time share the matrix rows through L2.
__device__ __forceinline__ Tile get_tile(const Groups &g, int E, int e, int t, int f_step) {
    Tile r;
    r.e = same(find_group(g, E, e, t));
    const int c = same(g.count[r.e]), nt = token_tiles(c), at = t - same(g.prefix[r.e]);
    const int size = tile_rows(c, nt), tt = at % nt;
    r.f0 = at / nt * f_step;
    r.row = same(g.row[r.e]) + tt * size;
    r.n = min(size, c - tt * size);
    return r;
}

__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {  // two f32 fma
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {  // a in the low byte
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

template <bool kGated, bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
expert_fp8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ RowMaps map_x, const Args a) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long bars[2 * kStages + 11];
    __shared__ float s_x[2][kTok];     // the tokens' scales of a block, per accumulator
    __shared__ float2 s_w[2];          // the two blocks of matrix rows' scales
    __shared__ float s_amax[2][2][kTok];  // largest |h| of a token in each half of the features, for two tiles by turns
    __shared__ uint32_t s_tmem;
    __shared__ int s_gave_up;
    const int tid = threadIdx.x, warp = same(tid / 32), lane = tid % 32;
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t buf = smem + kStages * kStage + (warp & (kSumWarps - 1)) * kBuf;
    int *tables = reinterpret_cast<int *>(smem_raw + (smem - smem_u32(smem_raw)) + kStages * kStage + kSumWarps * kBuf);
    const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, tfull = empty + 8 * kStages, tempty = tfull + 16,
                   sempty = tempty + 16, done = sempty + 16, met = done + 8;
    volatile int *gave_up = &s_gave_up;

    if (warp == kSumWarps) tmem_alloc(smem_u32(&s_tmem), 512);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mb_init(full + 8 * i, 1);
            mb_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mb_init(tfull + 8 * i, 3);  // the block's sums, and its scales by two warps
            mb_init(tempty + 8 * i, kSumWarps);
            mb_init(sempty + 8 * i, kSumWarps);
        }
        mb_init(done, 1);
        for (int i = 0; i < 4; ++i) mb_init(met + 8 * i, 2);  // the two warps that share 32 tokens
        s_gave_up = 0;
        mb_init_fence();
        tma_prefetch_map(&map_w);
        prefetch_maps(map_x);
    }
    tc_fence_before();
    __syncthreads();  // barriers and TMEM are ready
    tc_fence_after();
    const uint32_t tmem = (uint32_t)same((int)s_tmem);
    grid_dependency_wait();  // offsets, rows and scales come from earlier kernels
    grid_launch_dependents();
    // Result columns of a tile: 256, or 128 where all tiles then still run at
    // once (8 experts of 128 rows, K = 7168, F = 2048: 27.3 us against 30.0).
    const Groups g = make_groups<kGated ? 7 : 8, 7, 1>(
        tables, a.offsets, a.E, a.L, a.cap, a.most, a.pairs, gridDim.x,
        [&](int c, int shift) { return token_tiles(c) * ((a.F + (1 << shift) - 1) >> shift); },
        [](int) { return 0; });  // syncs the block
    const int width = 1 << g.shift;
    const int tiles = same(g.prefix[a.E]), steps = a.K / kK;
    int e = 0;

    if (warp >= kSumWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(other_regs(kGated)));
    if (warp == kSumWarps) {  // loads
        Ring<kStages> r;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const Tile w = get_tile(g, a.E, e, t, width);
            e = w.e;
            const bool two = kGated || (width == kN && w.f0 + kBlk < a.F);  // the second block of matrix rows exists
            const int second = w.f0 + (kGated ? a.F : kBlk);
            for (int k = 0; k < steps; ++k) {
                ok = mb_wait_warp(empty + 8 * r.slot, r.phase ^ 1u, gave_up);
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t bar = full + 8 * r.slot, sa = smem + r.slot * kStage, sb = sa + kBytesA;
                    mb_expect_tx(bar, (two ? 2 : 1) * kBlk * kK + rows_loaded(w.n) * 128);
                    tma_load_3d(sb, &map_w, bar, k * kK, w.f0, w.e);
                    if (two) tma_load_3d(sb + kBlk * kK, &map_w, bar, k * kK, second, w.e);
                    load_rows(sa, map_x, bar, k * kK, w.row, w.n);
                }
                __syncwarp();
                r.next();
            }
        }
        drain_ring(full, r);
        drain_ring(empty, r);
        mb_drain(done, 0);
    } else if (warp == kSumWarps + 1) {  // mma
        Ring<kStages> r;
        Ring<2> acc;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const Tile w = get_tile(g, a.E, e, t, width);
            e = w.e;
            const uint32_t desc = mma_desc(0, false, false, kTok, kGated ? kN : min(width, (a.F - w.f0 + 15) & ~15));
            for (int k = 0; k < steps; ++k) {
                ok = mb_wait_warp(full + 8 * r.slot, r.phase, gave_up) &&
                     mb_wait_warp(tempty + 8 * acc.slot, acc.phase ^ 1u, gave_up);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t sa = smem + r.slot * kStage;
                    const uint64_t da = smem_operand(sa, 16, 1024), db = smem_operand(sa + kBytesA, 16, 1024);
                    const uint32_t d = tmem + acc.slot * kN;
#pragma unroll
                    for (int i = 0; i < kK / 32; ++i) mma_fp8(d, da + i * 2, db + i * 2, desc, i != 0);
                    tc_commit(tfull + 8 * acc.slot);
                    tc_commit(empty + 8 * r.slot);
                }
                __syncwarp();
                r.next();
                acc.next();
            }
        }
        if (elect_one()) tc_commit(done);
        __syncwarp();
        mb_drain(done, 0);
    } else if (warp >= kSumWarps + 2) {
        // scales: each of two warps takes 64 tokens, two a lane; the next
        // blocks' are on their way while these wait for their accumulator
        const int t0 = (warp - kSumWarps - 2) * 64 + lane;
        const int fb = (a.w_rows + kBlk - 1) / kBlk;  // blocks of matrix rows
        const bool first = t0 == 0;
        Ring<2> acc;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const Tile w = get_tile(g, a.E, e, t, width);
            e = w.e;
            const bool in0 = t0 < w.n, in1 = t0 + 32 < w.n, two = kGated || (width == kN && w.f0 + kBlk < a.F);
            const float *sx = a.x_scales + (int64_t)(w.row + t0) * steps, *sx1 = sx + (int64_t)32 * steps;
            const float *sw0 = a.w_scales + ((int64_t)w.e * fb + w.f0 / kBlk) * steps;
            const float *sw1 = sw0 + (kGated ? (int64_t)(a.F / kBlk) * steps : steps);
            float next[kGroup][4];
            auto load = [&](int k0) {
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    const bool in = k0 + i < steps;
                    next[i][0] = in && in0 ? __ldg(sx + k0 + i) : 0.f;
                    next[i][1] = in && in1 ? __ldg(sx1 + k0 + i) : 0.f;
                    next[i][2] = in && first ? __ldg(sw0 + k0 + i) : 0.f;
                    next[i][3] = in && first && two ? __ldg(sw1 + k0 + i) : 0.f;
                }
            };
            load(0);
            for (int k0 = 0; k0 < steps && ok; k0 += kGroup) {
                float now[kGroup][4];
#pragma unroll
                for (int i = 0; i < kGroup; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) now[i][j] = next[i][j];
                load(k0 + kGroup);
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    if (k0 + i >= steps) break;
                    ok = mb_wait_warp(sempty + 8 * acc.slot, acc.phase ^ 1u, gave_up);
                    if (!ok) break;
                    s_x[acc.slot][t0] = now[i][0];
                    s_x[acc.slot][t0 + 32] = now[i][1];
                    if (first) s_w[acc.slot] = make_float2(now[i][2], now[i][3]);
                    __syncwarp();
                    if (lane == 0) mb_arrive(tfull + 8 * acc.slot);
                    acc.next();
                }
            }
        }
    } else if (warp < kSumWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(sum_regs(kGated)));
        // sums and results: warp w holds tokens 32 (w % 4).., one per lane,
        // and 64 columns of both blocks, 64 (w / 4)..
        const int quarter = warp & 3, half = warp >> 2;
        Ring<2> acc;
        int turn = 0;  // of the meetings at `met`
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const Tile w = get_tile(g, a.E, e, t, width);
            e = w.e;
            const bool some = quarter * 32 < w.n, mine = quarter * 32 + lane < w.n;
            uint64_t sum[2][4][8];  // [block][16 columns][pair]
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[b][i][j] = 0;
            for (int k = 0; k < steps; ++k) {
                ok = mb_wait_warp(tfull + 8 * acc.slot, acc.phase, gave_up);
                if (!ok) break;
                tc_fence_after();
                if (some) {
                    const uint32_t src = tmem + acc.slot * kN + ((uint32_t)(quarter * 32) << 16) + 64 * half;
                    // the next 32 columns are on their way while these are added
                    uint32_t v[2][32];
                    tmem_load32_async(src, v[0]);
                    const float x = s_x[acc.slot][quarter * 32 + lane];
                    const float2 sw = s_w[acc.slot];
                    const uint32_t x0 = __float_as_uint(x * sw.x), x1 = __float_as_uint(x * sw.y);
                    const uint64_t f0 = pair(x0, x0), f1 = pair(x1, x1);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        tmem_wait32(v[u & 1]);
                        if (u < 3) {
                            tmem_load32_async(src + (u + 1) / 2 * kBlk + (u + 1) % 2 * 32, v[(u + 1) & 1]);
                        } else {  // everything is in registers: the accumulator is free
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) {
                                mb_arrive(tempty + 8 * acc.slot);
                                mb_arrive(sempty + 8 * acc.slot);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            sum[u / 2][u % 2 * 2 + j / 8][j % 8] = fma2(pair(v[u & 1][2 * j], v[u & 1][2 * j + 1]),
                                                                        u < 2 ? f0 : f1, sum[u / 2][u % 2 * 2 + j / 8][j % 8]);
                    }
                } else if (lane == 0) {
                    mb_arrive(tempty + 8 * acc.slot);
                    mb_arrive(sempty + 8 * acc.slot);
                }
                acc.next();
            }
            if (!ok) break;
            if (!some) continue;
            if constexpr (!kGated) {
                // 64 bytes of each token's row at a time, turned in shared
                // memory so that four lanes write them (chunks of 16 bytes
                // swapped by token against bank conflicts)
                constexpr int kElem = kF32 ? 4 : 2, kCols = 64 / kElem;
                const int t0 = lane / 4, left = w.n - quarter * 32 - t0;  // first token that this lane writes
                const int cols = a.F - (w.f0 + 64 * half) - (lane & 3) * (16 / kElem);
                unsigned char *to = static_cast<unsigned char *>(a.y) +
                                    ((int64_t)(w.row + quarter * 32 + t0) * a.F + (a.F - cols)) * kElem;
                const int64_t step = (int64_t)8 * a.F * kElem;
                const uint32_t put = buf + lane * 64, get = buf + t0 * 64 + (((lane & 3) ^ ((t0 >> 1) & 3)) * 16);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if (b == 1 && width < kN) break;
#pragma unroll
                    for (int c0 = 0; c0 < 64; c0 += kCols) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint4 v;
                            if constexpr (kF32) {
                                const float2 x = unpair(sum[b][(c0 + 4 * q) / 16][(c0 + 4 * q) % 16 / 2]),
                                             y = unpair(sum[b][(c0 + 4 * q) / 16][(c0 + 4 * q) % 16 / 2 + 1]);
                                v = make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x),
                                               __float_as_uint(y.y));
                            } else {
                                uint32_t p[4];
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const float2 x = unpair(sum[b][(c0 + 8 * q) / 16][(c0 + 8 * q) % 16 / 2 + j]);
                                    p[j] = bf16x2(__float_as_uint(x.x), __float_as_uint(x.y));
                                }
                                v = make_uint4(p[0], p[1], p[2], p[3]);
                            }
                            st_shared128(put + ((q ^ ((lane >> 1) & 3)) * 16), v);
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {  // tokens t0 + 8 i: the same swap, 8 tokens being 512 bytes
                            const uint4 v = ld_shared128(get + i * 512);
                            if (8 * i < left && b * kBlk + c0 < cols)
                                *reinterpret_cast<uint4 *>(to + i * step + (b * kBlk + c0) * kElem) = v;
                        }
                        __syncwarp();
                    }
                }
            } else {
                // h takes the place of the gate's sums; its largest magnitude
                // over the token's 128 features joins two warps
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 gt = unpair(sum[0][i][j]), up = unpair(sum[1][i][j]);
                        const float h0 = silu_mul(gt.x, up.x), h1 = silu_mul(gt.y, up.y);
                        sum[0][i][j] = pair(__float_as_uint(h0), __float_as_uint(h1));
                        top = fmaxf(top, fmaxf(fabsf(h0), fabsf(h1)));
                    }
                // (a wait like the others: the other warp may have given
                // up.  One meeting a tile: what is written here is written
                // again after the next one, which the other warp reaches
                // after reading it.)
                s_amax[turn][half][quarter * 32 + lane] = top;
                __syncwarp();
                if (lane == 0) mb_arrive(met + 8 * quarter);
                ok = mb_wait_warp(met + 8 * quarter, turn, gave_up);
                if (!ok) break;
                top = fmaxf(top, s_amax[turn][half ^ 1][quarter * 32 + lane]);
                turn ^= 1;
                // h / scale as (h up) (1 / (scale up)): the reciprocal of a
                // scale below 2^-126 would overflow
                const float scale = __fdiv_rn(top, 448.f), up = scale < 0x1p-100f ? 0x1p100f : 1.f;
                const float inv = scale == 0.f ? 0.f : __fdiv_rn(1.f, scale * up);
                if (mine) {
                    const int64_t row = w.row + quarter * 32 + lane;
                    uint8_t *y = static_cast<uint8_t *>(a.y) + row * a.F + w.f0 + 64 * half;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t p[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 h0 = unpair(sum[0][i][2 * j]), h1 = unpair(sum[0][i][2 * j + 1]);
                            p[j] = e4m3x2(h0.x * up * inv, h0.y * up * inv) | (e4m3x2(h1.x * up * inv, h1.y * up * inv) << 16);
                        }
                        reinterpret_cast<uint4 *>(y)[i] = make_uint4(p[0], p[1], p[2], p[3]);
                    }
                    if (half == 0) a.y_scales[row * (a.F / kBlk) + w.f0 / kBlk] = scale;
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && s_gave_up) record_timeout();
    if (warp == kSumWarps) tmem_free(tmem, 512);
}

template <bool kGated, bool kF32>
cudaError_t launch(const CUtensorMap &map_w, const RowMaps &map_x, const Args &a, cudaStream_t stream) {
    auto kern = expert_fp8_kernel<kGated, kF32>;
    static thread_local AttrCache cache;
    cudaError_t e = cache.allow_smem(reinterpret_cast<const void *>(kern), kSmem + groups_bytes(1024));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)sm_count());
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem + groups_bytes(a.E);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, map_w, map_x, a);
}

}  // namespace

cudaError_t launch_expert_gemm_fp8(const ExpertRows &r, int K, int F, int gated, const void *xq, const float *x_scales,
                                   const void *wq, const float *w_scales, void *y, int y_f32, float *y_scales,
                                   cudaStream_t stream) {
    CUtensorMap map_w;
    RowMaps map_x;
    const int w_rows = gated ? 2 * F : F;
    const uint64_t wdims[3] = {(uint64_t)K, (uint64_t)w_rows, (uint64_t)r.E};
    const uint64_t strides[2] = {(uint64_t)K, (uint64_t)K * w_rows};
    const uint32_t wbox[3] = {kK, kBlk, 1};
    if (!encode_map(&map_w, 1, 3, wq, wdims, strides, wbox)) return cudaErrorInvalidValue;
    if (!encode_rows(&map_x, 1, xq, K, r.rows_total, r.most < kTok ? r.most : kTok)) return cudaErrorInvalidValue;
    const Args a{r.offsets, x_scales, w_scales, y, y_scales, r.cap, r.most, r.pairs, r.E, r.L, K, F, w_rows};
    if (gated) return launch<true, false>(map_w, map_x, a, stream);
    return y_f32 ? launch<false, true>(map_w, map_x, a, stream) : launch<false, false>(map_w, map_x, a, stream);
}

cudaError_t take_expert_fp8_error(int *err) { return take_tc_error(err); }

}  // namespace moe
