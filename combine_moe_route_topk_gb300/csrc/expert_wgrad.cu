// Gradient of the experts' matrices: dw[e][f][k] = sum over e's rows p of
// dy[p][f] x[p][k], zero for an expert without rows.
//
// Both operands have the reduction (the rows) as their outer dimension, so
// TMA boxes of 64 columns by 64 rows are handed to tcgen05.mma as transposed
// operands: M = 128 columns of dy, N = 256 columns of x, f32 sums in TMEM.  An
// expert's rows end anywhere; rows behind them belong to the next expert or
// hold anything (NaN too), so the mma warp zeroes them in shared memory, in
// the last block of 64 only and up to the next multiple of 16.
#include <cuda_bf16.h>

#include "expert_internal.cuh"
#include "pdl.cuh"
#include "tc_ops.cuh"

namespace moe {
namespace {

constexpr int kM = 128;  // columns of dy (rows of dw) of a tile
constexpr int kN = 256;  // columns of x
constexpr int kP = 64;   // rows of a stage
constexpr int kBlock = kP * 128;  // bytes of 64 columns of a stage
constexpr int kStages = 4;
constexpr int kStage = (kM + kN) / 64 * kBlock;
constexpr int kBuf = 4096;  // each storing warp's: 128 bytes of its 32 rows
constexpr int kThreads = 192;
constexpr int kSmem = 1024 + kStages * kStage + 4 * kBuf;

// An operand's columns: whole blocks of 64 are the third dimension of `blocks`,
// so that one load takes all blocks of a tile; `cols` takes one block and
// zero-fills behind the last column, for tiles that reach it.
struct ColumnMaps {
    CUtensorMap blocks, cols;
};

struct Args {
    const int32_t *offsets;
    void *dw;
    int64_t cap;
    int E, L, K, F;
};

template <bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
expert_wgrad_kernel(const __grid_constant__ ColumnMaps map_dy, const __grid_constant__ ColumnMaps map_x, const Args a) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long bars[2 * kStages + 5];
    __shared__ uint32_t s_tmem;
    __shared__ int s_gave_up;
    const int tid = threadIdx.x, warp = same(tid / 32), lane = tid % 32;
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char *stages = smem_raw + (smem - smem_u32(smem_raw));
    const uint32_t buf = smem + kStages * kStage + (warp & 3) * kBuf;
    int *tables = reinterpret_cast<int *>(stages + kStages * kStage + 4 * kBuf);
    const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, tfull = empty + 8 * kStages, tempty = tfull + 16,
                   done = tempty + 16;
    volatile int *gave_up = &s_gave_up;

    if (warp == 4) tmem_alloc(smem_u32(&s_tmem), 512);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mb_init(full + 8 * i, 1);
            mb_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mb_init(tfull + 8 * i, 1);
            mb_init(tempty + 8 * i, 4);
        }
        mb_init(done, 1);
        s_gave_up = 0;
        mb_init_fence();
        tma_prefetch_map(&map_dy.blocks);
        tma_prefetch_map(&map_x.blocks);
    }
    grid_dependency_wait();  // offsets and rows come from earlier kernels
    grid_launch_dependents();
    const int mt = (a.F + kM - 1) / kM, per = mt * ((a.K + kN - 1) / kN);  // tiles of an expert
    const Groups g = make_groups(tables, a.offsets, a.E, a.L, a.cap, [&](int) { return per; });  // syncs the block
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)same((int)s_tmem);
    const int tiles = a.E * per;

    if (warp == 4) {  // loads
        {
            Ring<kStages> r;
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const int e = t / per, at = t % per, m0 = at % mt * kM, n0 = at / mt * kN;
                const int row = same(g.row[e]), steps = (same(g.count[e]) + kP - 1) / kP;
                const bool whole_m = m0 + kM <= a.F, whole_n = n0 + kN <= a.K;
                const int mb = min(kM, a.F - m0) > 64 ? 2 : 1, nb = (min(kN, a.K - n0) + 63) / 64;
                for (int k = 0; k < steps; ++k) {
                    ok = mb_wait_warp(empty + 8 * r.slot, r.phase ^ 1u, gave_up);
                    if (!ok) break;
                    if (elect_one()) {
                    const uint32_t bar = full + 8 * r.slot, sa = smem + r.slot * kStage, sb = sa + kM / 64 * kBlock;
                    mb_expect_tx(bar, (mb + nb) * kBlock);
                    if (whole_m) {
                        tma_load_3d(sa, &map_dy.blocks, bar, 0, row + k * kP, m0 / 64);
                    } else {
                        for (int i = 0; i < mb; ++i)
                            tma_load_2d(sa + i * kBlock, &map_dy.cols, bar, m0 + i * 64, row + k * kP);
                    }
                    if (whole_n) {
                        tma_load_3d(sb, &map_x.blocks, bar, 0, row + k * kP, n0 / 64);
                    } else {
                        for (int i = 0; i < nb; ++i)
                            tma_load_2d(sb + i * kBlock, &map_x.cols, bar, n0 + i * 64, row + k * kP);
                    }
                    }
                    __syncwarp();
                    r.next();
                }
            }
            drain_loads(full, r);
        }
    } else if (warp == 5) {  // mma (the whole warp runs the loop, lane 0 issues)
        Ring<kStages> r;
        Ring<2> acc;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const int e = t / per, at = t % per, n0 = at / mt * kN;
            const int count = same(g.count[e]), steps = (count + kP - 1) / kP;
            if (steps == 0) continue;  // nothing to sum: the results are zeros
            const uint32_t desc = mma_desc(1, true, true, kM, (min(kN, a.K - n0) + 15) & ~15);
            const uint32_t d = tmem + acc.slot * kN;
            ok = mb_wait_warp(tempty + 8 * acc.slot, acc.phase ^ 1u, gave_up);
            tc_fence_after();
            for (int k = 0; k < steps && ok; ++k) {
                ok = mb_wait_warp(full + 8 * r.slot, r.phase, gave_up);
                if (!ok) break;
                const int left = min(kP, count - k * kP), slices = (left + 15) / 16;
                if (left % 16 != 0) {
                    const int words = (slices * 16 - left) * 8;  // 16-byte words of the lines behind the last row
                    for (int i = 0; i < (kM + kN) / 64; ++i) {
                        uint4 *line = reinterpret_cast<uint4 *>(stages + r.slot * kStage + i * kBlock + left * 128);
                        for (int j = lane; j < words; j += 32) line[j] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t sa = smem + r.slot * kStage;
                    const uint64_t da = smem_operand(sa, kBlock, 1024), db = smem_operand(sa + kM / 64 * kBlock, kBlock, 1024);
                    for (int i = 0; i < slices; ++i)  // 16 rows are 16 lines of 128 bytes
                        mma_bf16(d, da + i * 128, db + i * 128, desc, (k | i) != 0);
                    tc_commit(empty + 8 * r.slot);
                }
                __syncwarp();
                r.next();
            }
            if (elect_one()) tc_commit(tfull + 8 * acc.slot);
            __syncwarp();
            acc.next();
        }
        if (elect_one()) tc_commit(done);
        __syncwarp();
        mb_drain(done, 0);
    } else {  // results: warp w holds rows 32w.. of the tile, one per lane
        Ring<2> acc;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
            const int e = t / per, at = t % per, m0 = at % mt * kM, n0 = at / mt * kN;
            const bool some = same(g.count[e]) > 0;
            if (some) {
                if (!mb_wait_warp(tfull + 8 * acc.slot, acc.phase, gave_up)) break;
                tc_fence_after();
            }
            const uint32_t src = tmem + acc.slot * kN + ((uint32_t)(warp * 32) << 16);
            const int f0 = m0 + warp * 32, n = min(kN, a.K - n0);
            // 128 bytes of each row at a time, turned in shared memory so that
            // eight lanes write a row's 128 bytes (chunks of 16 bytes swapped
            // by row against bank conflicts)
            constexpr int kCols = kF32 ? 32 : 64, kElem = kF32 ? 4 : 2;
            for (int c0 = 0; c0 < n; c0 += kCols) {
#pragma unroll
                for (int h = 0; h < kCols / 32; ++h) {
                    uint32_t v[32];
                    if (some) {
                        tmem_load32(src + c0 + 32 * h, v);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0u;
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 16 / kElem) {
                        uint4 q;
                        if constexpr (kF32)
                            q = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                        else
                            q = make_uint4(bf16x2(v[j], v[j + 1]), bf16x2(v[j + 2], v[j + 3]),
                                           bf16x2(v[j + 4], v[j + 5]), bf16x2(v[j + 6], v[j + 7]));
                        const int chunk = (32 * h + j) * kElem / 16;
                        st_shared128(buf + lane * 128 + ((chunk ^ (lane & 7)) * 16), q);
                    }
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = i * 4 + lane / 8, chunk = lane & 7;
                    const uint4 q = ld_shared128(buf + r * 128 + ((chunk ^ (r & 7)) * 16));
                    const int k = c0 + chunk * 16 / kElem;
                    if (f0 + r < a.F && k < n)
                        *reinterpret_cast<uint4 *>(static_cast<unsigned char *>(a.dw) +
                                                   (((int64_t)e * a.F + f0 + r) * a.K + n0 + k) * kElem) = q;
                }
                __syncwarp();
            }
            if (some) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mb_arrive(tempty + 8 * acc.slot);
                acc.next();
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && s_gave_up) record_timeout();
    if (warp == 4) tmem_free(tmem, 512);
}

template <bool kF32>
cudaError_t launch(const ColumnMaps &map_dy, const ColumnMaps &map_x, const Args &a, cudaStream_t stream) {
    auto kern = expert_wgrad_kernel<kF32>;
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
    return cudaLaunchKernelEx(&cfg, kern, map_dy, map_x, a);
}

// `tile`: columns of a tile.  Rows of less than one tile use `cols` alone.
bool encode_columns(ColumnMaps *m, const void *base, int cols, int64_t rows, int tile) {
    const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, stride = (uint64_t)cols * 2;
    const uint32_t box[2] = {64, kP};
    if (!encode_map(&m->cols, 0, 2, base, dims, &stride, box)) return false;
    m->blocks = m->cols;
    if (cols < tile) return true;
    const uint64_t dims3[3] = {64, (uint64_t)rows, (uint64_t)cols / 64}, strides3[2] = {stride, 128};
    const uint32_t box3[3] = {64, kP, (uint32_t)tile / 64};
    return encode_map(&m->blocks, 0, 3, base, dims3, strides3, box3);
}

}  // namespace

cudaError_t launch_expert_wgrad(const ExpertRows &r, int K, int F, const void *dy, const void *x, void *dw, int dw_f32,
                                cudaStream_t stream) {
    ColumnMaps map_dy, map_x;
    if (!encode_columns(&map_dy, dy, F, r.rows_total, kM) || !encode_columns(&map_x, x, K, r.rows_total, kN))
        return cudaErrorInvalidValue;
    const Args a{r.offsets, dw, r.cap, r.E, r.L, K, F};
    return dw_f32 ? launch<true>(map_dy, map_x, a, stream) : launch<false>(map_dy, map_x, a, stream);
}

cudaError_t take_expert_wgrad_error(int *err) { return take_tc_error(err); }

}  // namespace moe
