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
// 128 at a time (four tcgen05.mma of 32, f32 in TMEM) and eight warps add the
// blocks up in f32 registers: acc += (sx sw) * block.  As in the bf16 product
// the matrix rows are M; a tile is two blocks of 128 of them (the gate and
// the up rows of the same features, or neighbours) by up to 128 tokens.  A
// ninth warp loads, a tenth issues mma, an eleventh multiplies the scales of
// the coming blocks.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "expert_internal.cuh"
#include "pdl.cuh"
#include "tc_ops.cuh"

namespace moe {
namespace {

constexpr int kM = 128;     // matrix rows of a block; a tile has two
constexpr int kTok = 128;   // most tokens of a tile
constexpr int kK = 128;     // reduction elements of a stage: one scale block, one 128-byte line
constexpr int kBox = 32;    // token rows of one TMA load
constexpr int kStages = 4;
constexpr int kBytesA = kM * kK;  // one block
constexpr int kBytesB = kTok * kK;
constexpr int kStage = 2 * kBytesA + kBytesB;
constexpr int kSlots = 8;   // blocks whose scale products are ready
constexpr int kThreads = 352;
constexpr int kGroup = 4;   // blocks whose scales are loaded together

struct Args {
    const int32_t *offsets;
    const float *x_scales, *w_scales;
    void *y;
    float *y_scales;
    int64_t cap;
    int E, L, K, F, w_rows;  // reduction length, result columns, matrix rows of an expert
};

__host__ __device__ inline int token_tiles(int count) { return (count + kTok - 1) / kTok; }

struct Tile {
    int e, m0, row, n;  // group, first result column, first token row, tokens
};

__device__ __forceinline__ Tile get_tile(const Groups &g, int E, int e, int t, int m_step) {
    Tile r;
    r.e = find_group(g, E, e, t);
    const int c = g.count[r.e], nt = token_tiles(c), at = t - g.prefix[r.e];
    const int size = ((c + nt - 1) / nt + 15) & ~15;
    const int tt = at % nt;
    r.m0 = at / nt * m_step;
    r.row = g.row[r.e] + tt * size;
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
__device__ __forceinline__ uint8_t e4m3(float v) {
    return (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

template <bool kGated, bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
expert_fp8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const Args a) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long bars[2 * kStages + 2 * kSlots + 5];
    __shared__ __align__(16) float s_fac[kSlots][2][kTok];  // sx * sw of each token, per block of rows
    __shared__ __align__(16) float s_amax[kTok][4];         // largest |h| of a token in each warp's features
    __shared__ uint32_t s_tmem;
    __shared__ int s_gave_up;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    int *tables = reinterpret_cast<int *>(smem_raw + (smem - smem_u32(smem_raw)) + kStages * kStage);
    const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, sfull = empty + 8 * kStages,
                   sempty = sfull + 8 * kSlots, tfull = sempty + 8 * kSlots, tempty = tfull + 16, done = tempty + 16;
    volatile int *gave_up = &s_gave_up;

    if (warp == 8) tmem_alloc(smem_u32(&s_tmem), 512);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mb_init(full + 8 * i, 1);
            mb_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < kSlots; ++i) {
            mb_init(sfull + 8 * i, 1);
            mb_init(sempty + 8 * i, 8);
        }
        for (int i = 0; i < 2; ++i) {
            mb_init(tfull + 8 * i, 1);
            mb_init(tempty + 8 * i, 8);
        }
        mb_init(done, 1);
        s_gave_up = 0;
        mb_init_fence();
        tma_prefetch_map(&map_w);
        tma_prefetch_map(&map_x);
    }
    grid_dependency_wait();  // offsets, rows and scales come from earlier kernels
    grid_launch_dependents();
    constexpr int kStep = kGated ? kM : 2 * kM;  // result columns of a tile
    const int m_tiles = (a.F + kStep - 1) / kStep;
    const Groups g = make_groups(tables, a.offsets, a.E, a.L, a.cap,
                                 [&](int c) { return token_tiles(c) * m_tiles; });  // syncs the block
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int tiles = g.prefix[a.E], steps = a.K / kK;
    int e = 0;

    if (warp == 8) {  // loads
        if (lane == 0) {
            Ring<kStages> r;
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const Tile w = get_tile(g, a.E, e, t, kStep);
                e = w.e;
                const int boxes = (w.n + kBox - 1) / kBox;
                const bool two = kGated || w.m0 + kM < a.F;  // the second block of rows exists
                for (int k = 0; k < steps; ++k) {
                    ok = mb_wait(empty + 8 * r.slot, r.phase ^ 1u, gave_up);
                    if (!ok) break;
                    const uint32_t bar = full + 8 * r.slot, sa = smem + r.slot * kStage, sb = sa + 2 * kBytesA;
                    mb_expect_tx(bar, (two ? 2 : 1) * kBytesA + boxes * kBox * kK);
                    tma_load_3d(sa, &map_w, bar, k * kK, w.m0, w.e);
                    if (two) tma_load_3d(sa + kBytesA, &map_w, bar, k * kK, w.m0 + (kGated ? a.F : kM), w.e);
                    for (int b = 0; b < boxes; ++b)
                        tma_load_2d(sb + b * kBox * kK, &map_x, bar, k * kK, w.row + b * kBox);
                    r.next();
                }
            }
            drain_loads(full, r);
        }
    } else if (warp == 9) {  // mma
        if (lane == 0) {
            Ring<kStages> r;
            Ring<2> acc;
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const Tile w = get_tile(g, a.E, e, t, kStep);
                e = w.e;
                const uint32_t desc = mma_desc(0, false, false, kM, (w.n + 15) & ~15);
                const int blocks = kGated || w.m0 + kM < a.F ? 2 : 1;
                for (int k = 0; k < steps; ++k) {
                    ok = mb_wait(tempty + 8 * acc.slot, acc.phase ^ 1u, gave_up) &&
                         mb_wait(full + 8 * r.slot, r.phase, gave_up);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t sa = smem + r.slot * kStage;
                    const uint64_t db = smem_operand(sa + 2 * kBytesA, 16, 1024);
                    for (int b = 0; b < blocks; ++b) {
                        const uint64_t da = smem_operand(sa + b * kBytesA, 16, 1024);
                        const uint32_t d = tmem + acc.slot * 2 * kTok + b * kTok;
#pragma unroll
                        for (int i = 0; i < kK / 32; ++i) mma_fp8(d, da + i * 2, db + i * 2, desc, i != 0);
                    }
                    tc_commit(empty + 8 * r.slot);
                    tc_commit(tfull + 8 * acc.slot);
                    r.next();
                    acc.next();
                }
            }
            tc_commit(done);
            mb_drain(done, 0);
        }
    } else if (warp == 10) {  // scale products; lane l takes tokens l, l + 32, ...
        Ring<kSlots> s;
        bool ok = true;
        const int fb = (a.w_rows + kM - 1) / kM;  // blocks of matrix rows
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const Tile w = get_tile(g, a.E, e, t, kStep);
            e = w.e;
            const float *sx = a.x_scales + (int64_t)w.row * steps;
            const float *sw0 = a.w_scales + ((int64_t)w.e * fb + w.m0 / kM) * steps;
            const float *sw1 = sw0 + (kGated ? (int64_t)(a.F / kM) * steps : steps);
            const bool two = kGated || w.m0 + kM < a.F;
            for (int k0 = 0; k0 < steps && ok; k0 += kGroup) {
                float fx[kGroup][kTok / 32], f0[kGroup], f1[kGroup];
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    const bool in = k0 + i < steps;
                    f0[i] = in ? __ldg(sw0 + k0 + i) : 0.f;
                    f1[i] = in && two ? __ldg(sw1 + k0 + i) : 0.f;
#pragma unroll
                    for (int j = 0; j < kTok / 32; ++j)
                        fx[i][j] = in && lane + 32 * j < w.n ? __ldg(sx + (int64_t)(lane + 32 * j) * steps + k0 + i) : 0.f;
                }
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    if (k0 + i >= steps || !ok) break;
                    ok = __all_sync(0xffffffffu, mb_wait(sempty + 8 * s.slot, s.phase ^ 1u, gave_up));
                    if (!ok) break;
#pragma unroll
                    for (int j = 0; j < kTok / 32; ++j) {
                        s_fac[s.slot][0][lane + 32 * j] = fx[i][j] * f0[i];
                        s_fac[s.slot][1][lane + 32 * j] = fx[i][j] * f1[i];
                    }
                    __syncwarp();
                    if (lane == 0) mb_arrive(sfull + 8 * s.slot);
                    s.next();
                }
            }
        }
    } else {
        // sums and results: warp w holds the lanes (matrix rows) 32 (w % 4)..
        // of both blocks and the chunks of 16 tokens 2 i + w / 4
        const int quarter = warp & 3, half = warp >> 2;
        Ring<kSlots> s;
        Ring<2> acc;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const Tile w = get_tile(g, a.E, e, t, kStep);
            e = w.e;
            uint64_t sum[2][4][8];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[b][i][j] = 0;
            for (int k = 0; k < steps; ++k) {
                ok = mb_wait(sfull + 8 * s.slot, s.phase, gave_up) && mb_wait(tfull + 8 * acc.slot, acc.phase, gave_up);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t src = tmem + acc.slot * 2 * kTok + ((uint32_t)(quarter * 32) << 16);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c0 = 16 * (2 * i + half);
                    if (c0 < w.n) {
                        uint32_t v[2][16];
                        tmem_load16x2(src + c0, v[0], src + kTok + c0, v[1]);
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const ulonglong2 *f = reinterpret_cast<const ulonglong2 *>(&s_fac[s.slot][b][c0]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const ulonglong2 ff = f[j];
                                sum[b][i][2 * j] = fma2(pair(v[b][4 * j], v[b][4 * j + 1]), ff.x, sum[b][i][2 * j]);
                                sum[b][i][2 * j + 1] =
                                    fma2(pair(v[b][4 * j + 2], v[b][4 * j + 3]), ff.y, sum[b][i][2 * j + 1]);
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mb_arrive(tempty + 8 * acc.slot);
                    mb_arrive(sempty + 8 * s.slot);
                }
                s.next();
                acc.next();
            }
            if (!ok) break;
            if constexpr (!kGated) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int f = w.m0 + b * kM + quarter * 32 + lane;
                    if (f >= a.F) continue;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c0 = 16 * (2 * i + half);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float2 v = unpair(sum[b][i][j]);
                            const int64_t at = (int64_t)(w.row + c0 + 2 * j) * a.F + f;
                            if constexpr (kF32) {
                                float *y = static_cast<float *>(a.y);
                                if (c0 + 2 * j < w.n) y[at] = v.x;
                                if (c0 + 2 * j + 1 < w.n) y[at + a.F] = v.y;
                            } else {
                                __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(a.y);
                                if (c0 + 2 * j < w.n) y[at] = __float2bfloat16_rn(v.x);
                                if (c0 + 2 * j + 1 < w.n) y[at + a.F] = __float2bfloat16_rn(v.y);
                            }
                        }
                    }
                }
            } else {
                // h replaces the gate's sums; its largest magnitude over the
                // 128 features of a token: over the warp's 32 by a warp
                // maximum of the (non-negative) float's bits, then over the
                // four warps that hold the same tokens
                float h[4][16];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c0 = 16 * (2 * i + half);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 gt = unpair(sum[0][i][j]), up = unpair(sum[1][i][j]);
                        h[i][2 * j] = gt.x / (1.f + expf(-gt.x)) * up.x;
                        h[i][2 * j + 1] = gt.y / (1.f + expf(-gt.y)) * up.y;
                    }
                    if (c0 < w.n) {
                        uint32_t mine = 0;
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(h[i][j]) & 0x7fffffffu);
                            if (lane == j) mine = m;
                        }
                        if (lane < 16) s_amax[c0 + lane][quarter] = __uint_as_float(mine);
                    }
                }
                asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c0 = 16 * (2 * i + half);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        if (c0 + j < w.n) {
                            const float4 m = *reinterpret_cast<const float4 *>(s_amax[c0 + j]);
                            const float top = fmaxf(fmaxf(m.x, m.y), fmaxf(m.z, m.w));
                            const float scale = __fdiv_rn(top, 448.f);
                            const int64_t row = w.row + c0 + j;
                            uint8_t code = 0;
                            if (scale != 0.f) code = e4m3(__fdiv_rn(h[i][j], scale));
                            static_cast<uint8_t *>(a.y)[row * a.F + w.m0 + quarter * 32 + lane] = code;
                            if (quarter == 0 && lane == 0) a.y_scales[row * (a.F / kM) + w.m0 / kM] = scale;
                        }
                    }
                }
                asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");  // s_amax is written again
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && s_gave_up) record_timeout();
    if (warp == 8) tmem_free(tmem, 512);
}

template <bool kGated, bool kF32>
cudaError_t launch(const CUtensorMap &map_w, const CUtensorMap &map_x, const Args &a, cudaStream_t stream) {
    auto kern = expert_fp8_kernel<kGated, kF32>;
    const int smem = 1024 + kStages * kStage + groups_bytes(a.E);
    static thread_local AttrCache cache;
    cudaError_t e = cache.allow_smem(reinterpret_cast<const void *>(kern), 1024 + kStages * kStage + groups_bytes(1024));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)sm_count());
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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
    CUtensorMap map_w, map_x;
    const int w_rows = gated ? 2 * F : F;
    const uint64_t wdims[3] = {(uint64_t)K, (uint64_t)w_rows, (uint64_t)r.E};
    const uint64_t strides[2] = {(uint64_t)K, (uint64_t)K * w_rows};
    const uint32_t wbox[3] = {kK, kM, 1};
    if (!encode_map(&map_w, 1, 3, wq, wdims, strides, wbox)) return cudaErrorInvalidValue;
    const uint64_t xdims[2] = {(uint64_t)K, (uint64_t)r.rows_total}, row = (uint64_t)K;
    const uint32_t xbox[2] = {kK, kBox};
    if (!encode_map(&map_x, 1, 2, xq, xdims, &row, xbox)) return cudaErrorInvalidValue;
    const Args a{r.offsets, x_scales, w_scales, y, y_scales, r.cap, r.E, r.L, K, F, w_rows};
    if (gated) return launch<true, false>(map_w, map_x, a, stream);
    return y_f32 ? launch<false, true>(map_w, map_x, a, stream) : launch<false, false>(map_w, map_x, a, stream);
}

cudaError_t take_expert_fp8_error(int *err) { return take_tc_error(err); }

}  // namespace moe
