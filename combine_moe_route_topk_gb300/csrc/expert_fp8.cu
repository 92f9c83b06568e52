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
// 128 at a time (four tcgen05.mma of 32, f32 in TMEM) and eight warps add
// the blocks up in f32 registers: acc += (sx sw) * block.  As in the bf16
// product the matrix rows are M; a tile is two blocks of 128 of them (the gate
// and the up rows of the same features, or neighbours) by up to 128 tokens.
// Of the last four warps one loads, one issues mma and two multiply the
// scales of the coming blocks.
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
constexpr int kGroup = 4;   // blocks whose scales are loaded together
constexpr int kSumWarps = 8;
constexpr int kThreads = 32 * (kSumWarps + 4);
constexpr int kBuf = 1024;  // each summing warp's: 16 tokens' bf16 (8 tokens' f32) results of 32 features
constexpr int kSmem = 1024 + kStages * kStage + kSumWarps * kBuf;
// Registers: 384 threads are launched with 168 each; the summing warps take
// 208, the others give back to 88 (256 * 208 + 128 * 88 = 384 * 168).
constexpr int kSumRegs = 208, kOtherRegs = 88;

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
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {  // a in the low byte
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ void st_shared8(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

template <bool kGated, bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
expert_fp8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const Args a) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long bars[2 * kStages + 2 * kSlots + 5];
    __shared__ __align__(16) float s_fac[kSlots][2][kTok];  // sx * sw of each token, per block of rows
    __shared__ __align__(16) float s_amax[kTok][4];         // largest |h| of a token in each warp's features
    __shared__ __align__(16) float s_inv[kTok];             // 1 / scale of its 128 features
    __shared__ uint32_t s_tmem;
    __shared__ int s_gave_up;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t buf = smem + kStages * kStage + (warp & (kSumWarps - 1)) * kBuf;
    int *tables = reinterpret_cast<int *>(smem_raw + (smem - smem_u32(smem_raw)) + kStages * kStage + kSumWarps * kBuf);
    const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, sfull = empty + 8 * kStages,
                   sempty = sfull + 8 * kSlots, tfull = sempty + 8 * kSlots, tempty = tfull + 16, done = tempty + 16;
    volatile int *gave_up = &s_gave_up;

    if (warp == kSumWarps) tmem_alloc(smem_u32(&s_tmem), 512);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mb_init(full + 8 * i, 1);
            mb_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < kSlots; ++i) {
            mb_init(sfull + 8 * i, 2);
            mb_init(sempty + 8 * i, kSumWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mb_init(tfull + 8 * i, 1);
            mb_init(tempty + 8 * i, kSumWarps);
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

    if (warp >= kSumWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kSumWarps) {  // loads
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
    } else if (warp == kSumWarps + 1) {  // mma
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
    } else if (warp >= kSumWarps + 2) {
        // scale products; the two warps take 64 tokens each, two a lane.  The
        // next blocks' scales are on their way while these wait for slots.
        const int t0 = (warp - kSumWarps - 2) * 64 + lane;
        const int fb = (a.w_rows + kM - 1) / kM;  // blocks of matrix rows
        Ring<kSlots> s;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const Tile w = get_tile(g, a.E, e, t, kStep);
            e = w.e;
            const bool in0 = t0 < w.n, in1 = t0 + 32 < w.n, two = kGated || w.m0 + kM < a.F;
            const float *sx = a.x_scales + (int64_t)(w.row + t0) * steps, *sx1 = sx + (int64_t)32 * steps;
            const float *sw0 = a.w_scales + ((int64_t)w.e * fb + w.m0 / kM) * steps;
            const float *sw1 = sw0 + (kGated ? (int64_t)(a.F / kM) * steps : steps);
            float next[kGroup][4];
            auto load = [&](int k0) {
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    const bool in = k0 + i < steps;
                    next[i][0] = in && in0 ? __ldg(sx + k0 + i) : 0.f;
                    next[i][1] = in && in1 ? __ldg(sx1 + k0 + i) : 0.f;
                    next[i][2] = in ? __ldg(sw0 + k0 + i) : 0.f;
                    next[i][3] = in && two ? __ldg(sw1 + k0 + i) : 0.f;
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
                    if (k0 + i >= steps || !ok) break;
                    ok = __all_sync(0xffffffffu, mb_wait(sempty + 8 * s.slot, s.phase ^ 1u, gave_up));
                    if (!ok) break;
                    s_fac[s.slot][0][t0] = now[i][0] * now[i][2];
                    s_fac[s.slot][1][t0] = now[i][0] * now[i][3];
                    s_fac[s.slot][0][t0 + 32] = now[i][1] * now[i][2];
                    s_fac[s.slot][1][t0 + 32] = now[i][1] * now[i][3];
                    __syncwarp();
                    if (lane == 0) mb_arrive(sfull + 8 * s.slot);
                    s.next();
                }
            }
        }
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
        // sums and results: warp w holds the lanes (matrix rows) 32 (w % 4)..
        // of both blocks and every other chunk of 16 tokens, 2 i + w / 4
        const int quarter = warp & 3, half = warp >> 2;
        Ring<kSlots> s;
        Ring<2> acc;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const Tile w = get_tile(g, a.E, e, t, kStep);
            e = w.e;
            const int chunks = (w.n + 31 - 16 * half) / 32;  // this warp's
            uint64_t sum[4][2][8];  // [chunk][block][pair of tokens]
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[i][b][j] = 0;
            for (int k = 0; k < steps; ++k) {
                ok = mb_wait(sfull + 8 * s.slot, s.phase, gave_up) && mb_wait(tfull + 8 * acc.slot, acc.phase, gave_up);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t src = tmem + acc.slot * 2 * kTok + ((uint32_t)(quarter * 32) << 16) + 16 * half;
                const uint32_t fac = smem_u32(&s_fac[s.slot][0][16 * half]);
                // the next 16 columns are on their way while these are added
                uint32_t v[2][16];
                if (chunks > 0) tmem_load16_async(src, v[0]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i < chunks) {
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            tmem_wait16(v[b]);
                            if (b == 0) tmem_load16_async(src + 32 * i + kTok, v[1]);
                            else if (i + 1 < chunks) tmem_load16_async(src + 32 * (i + 1), v[0]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint4 f = ld_shared128(fac + (b * kTok + 32 * i + 4 * j) * 4);
                                sum[i][b][2 * j] = fma2(pair(v[b][4 * j], v[b][4 * j + 1]), pair(f.x, f.y), sum[i][b][2 * j]);
                                sum[i][b][2 * j + 1] =
                                    fma2(pair(v[b][4 * j + 2], v[b][4 * j + 3]), pair(f.z, f.w), sum[i][b][2 * j + 1]);
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
                // 16 (f32: 8) tokens at a time through the warp's buffer, to
                // write whole sectors
                constexpr int kRow = kF32 ? 128 : 64, kElem = kF32 ? 4 : 2, kPass = kBuf / kRow, kPer = kRow / 16;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
#pragma unroll
                        for (int j0 = 0; j0 < 16; j0 += kPass) {
                            const int c0 = 16 * (2 * i + half) + j0;
                            if (c0 < w.n) {
#pragma unroll
                                for (int j = 0; j < kPass; j += 2) {
                                    const float2 v = unpair(sum[i][b][(j0 + j) / 2]);
                                    if constexpr (kF32) {
                                        st_shared32(buf + j * kRow + lane * 4, __float_as_uint(v.x));
                                        st_shared32(buf + (j + 1) * kRow + lane * 4, __float_as_uint(v.y));
                                    } else {
                                        const uint32_t two = bf16x2(__float_as_uint(v.x), __float_as_uint(v.y));
                                        st_shared16(buf + j * kRow + lane * 2, two);
                                        st_shared16(buf + (j + 1) * kRow + lane * 2, two >> 16);
                                    }
                                }
                                __syncwarp();
                                const int f = w.m0 + b * kM + quarter * 32 + lane % kPer * (16 / kElem);
#pragma unroll
                                for (int i2 = 0; i2 < kBuf / 512; ++i2) {
                                    const int tok = i2 * (32 / kPer) + lane / kPer;
                                    const uint4 q = ld_shared128(buf + i2 * 512 + lane * 16);
                                    if (c0 + tok < w.n && f < a.F)
                                        *reinterpret_cast<uint4 *>(static_cast<unsigned char *>(a.y) +
                                                                   ((int64_t)(w.row + c0 + tok) * a.F + f) * kElem) = q;
                                }
                                __syncwarp();
                            }
                        }
                    }
                }
            } else {
                // h takes the place of the gate's sums; its largest magnitude
                // over the 128 features of a token: over the warp's 32 by a
                // warp maximum of the (non-negative) float's bits, then over
                // the four warps that hold the same tokens
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c0 = 16 * (2 * i + half);
                    if (c0 < w.n) {
                        uint32_t mine = 0;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float2 gt = unpair(sum[i][0][j]), up = unpair(sum[i][1][j]);
                            const uint32_t h0 = __float_as_uint(silu_mul(gt.x, up.x)),
                                           h1 = __float_as_uint(silu_mul(gt.y, up.y));
                            sum[i][0][j] = pair(h0, h1);
                            const uint32_t m0 = __reduce_max_sync(0xffffffffu, h0 & 0x7fffffffu),
                                           m1 = __reduce_max_sync(0xffffffffu, h1 & 0x7fffffffu);
                            if (lane == 2 * j) mine = m0;
                            if (lane == 2 * j + 1) mine = m1;
                        }
                        if (lane < 16) s_amax[c0 + lane][quarter] = __uint_as_float(mine);
                    }
                }
                asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
                if (lane < 16) {  // a warp for each of their chunks
                    const int c = 16 * (2 * quarter + half) + lane;
                    if (c < w.n) {
                        const float4 m = *reinterpret_cast<const float4 *>(s_amax[c]);
                        const float scale = __fdiv_rn(fmaxf(fmaxf(m.x, m.y), fmaxf(m.z, m.w)), 448.f);
                        s_inv[c] = scale == 0.f ? 0.f : __fdiv_rn(1.f, scale);
                        a.y_scales[(int64_t)(w.row + c) * (a.F / kM) + w.m0 / kM] = scale;
                    }
                }
                asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c0 = 16 * (2 * i + half);
                    if (c0 < w.n) {  // 16 tokens by 32 features: 512 bytes
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float2 h = unpair(sum[i][0][j]);
                            const uint32_t two = e4m3x2(h.x * s_inv[c0 + 2 * j], h.y * s_inv[c0 + 2 * j + 1]);
                            st_shared8(buf + 64 * j + lane, two);
                            st_shared8(buf + 64 * j + 32 + lane, two >> 8);
                        }
                        __syncwarp();
                        const uint4 q = ld_shared128(buf + lane * 16);
                        if (c0 + lane / 2 < w.n)
                            *reinterpret_cast<uint4 *>(static_cast<unsigned char *>(a.y) +
                                                       (int64_t)(w.row + c0 + lane / 2) * a.F + w.m0 + quarter * 32 +
                                                       (lane & 1) * 16) = q;
                        __syncwarp();
                    }
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
cudaError_t launch(const CUtensorMap &map_w, const CUtensorMap &map_x, const Args &a, cudaStream_t stream) {
    auto kern = expert_fp8_kernel<kGated, kF32>;
    const int smem = kSmem + groups_bytes(a.E);
    static thread_local AttrCache cache;
    cudaError_t e = cache.allow_smem(reinterpret_cast<const void *>(kern), kSmem + groups_bytes(1024));
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
