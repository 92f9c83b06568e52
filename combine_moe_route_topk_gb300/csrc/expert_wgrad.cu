// Gradient of the experts' matrices: dw[e][f][k] = sum over e's rows p of
// dy[p][f] x[p][k], zero for an expert without rows.
//
// Both operands have the reduction (the rows) as their outer dimension, so
// TMA boxes of 64 columns by 64 rows are handed to tcgen05.mma as transposed
// operands, f32 sums in TMEM.  Blocks work in pairs: a tile is 256 columns of
// dy (M) by 256 of x (N), each block holding 128 of both and 128 rows of the
// result.  An expert's rows end anywhere; rows behind them belong to the next
// expert or hold anything (NaN too), so they are zeroed in shared memory, up
// to the next multiple of 16: a warp of each block does so with its part of
// the expert's last 64 rows, which are counted on barriers of their own, and
// tells the leader.  (With the mma warp itself doing so, a tile of 512 rows
// spent 2600 to 4000 of its 10000 cycles on it.)
//
// f32 results are summed in parts of 512 rows, added up in registers: the
// tensor core's sums come out small, by 8e-7 of their value after 1024 rows,
// 1.6e-5 after 16384 (expert_gemm.cu says why).  So are bf16 ones, in parts of
// 2048, where an expert can have more than kWhole rows (at most 1.5 % slower; with
// parts of 512 one expert of 65536 rows, K = F = 1024, took 248 us instead of 236,
// now 239).
#include <cuda_bf16.h>

#include <type_traits>

#include "expert_internal.cuh"
#include "pdl.cuh"
#include "tc_ops.cuh"

namespace moe {
namespace {

constexpr int kM = 128;  // columns of dy (rows of dw) of a block's half of a tile
constexpr int kN = 256;  // most columns of x of a tile
constexpr int kP = 64;   // rows of a stage
constexpr int kCols = kP * 128;  // bytes of 64 columns of a stage
constexpr int kStage = (kM + kN / 2) / 64 * kCols;
constexpr int kStages = 6;
// Stages of a part of a sum: 512 rows for f32 results, 2048 for bf16.
constexpr int part_stages(bool f32) { return (f32 ? 512 : 2048) / kP; }

// Warps: those that store results, one that loads, one that issues mma, one
// that zeroes; for sums in parts one more that only gives its registers away
// (384 threads are launched with 168 each, the storing ones take 216, the
// others keep 72).
template <bool kParts>
struct Shape {
    static constexpr int kStoreWarps = kParts ? 8 : 4, kThreads = kParts ? 384 : 224;
    static constexpr int kBuf = kParts ? 2048 : 4096;  // each storing warp's: 64 (or 128) bytes of its 32 rows
    static constexpr int kSmem = 1024 + kStages * kStage + kStoreWarps * kBuf;
};

// An operand's columns: whole blocks of 64 are the third dimension of `blocks`,
// so that one load takes all blocks of a tile; `cols` takes one block and
// zero-fills behind the last column, for tiles that reach it.
struct ColumnMaps {
    CUtensorMap blocks, cols;
};

struct Args {
    const int32_t *offsets;
    void *dw;
    int64_t cap, most, pairs;
    int E, L, K, F;
    int width;  // columns of x of a tile
};

// Tile `at` of an expert, and what block `rank` of the pair has of it.
struct Part {
    int m0, n0, n;  // first row and column of the tile's results, N of its mma
    int m_cols0, m_cols1;  // columns of dy that block 0 and 1 load, in blocks of 64 (0, 1 or 2)
    int n_cols;            // columns of x that each loads, in blocks of 64
};
__device__ __forceinline__ Part get_part(const Args &a, int mt, int at) {
    Part p;
    p.m0 = at % mt * 2 * kM;
    p.n0 = at / mt * a.width;
    p.n = min(a.width, (a.K - p.n0 + 31) & ~31);  // a pair's N is a multiple of 32
    p.m_cols0 = min(2, (a.F - p.m0 + 63) / 64);
    p.m_cols1 = max(0, min(2, (a.F - p.m0 - kM + 63) / 64));
    p.n_cols = (p.n / 2 + 63) / 64;
    return p;
}

template <bool kParts, bool kF32>
__global__ void __launch_bounds__(Shape<kParts>::kThreads, 1)
expert_wgrad_kernel(const __grid_constant__ ColumnMaps map_dy, const __grid_constant__ ColumnMaps map_x, const Args a) {
    static_assert(kParts || !kF32, "f32 results are summed in parts");
    constexpr int kStoreWarps = Shape<kParts>::kStoreWarps, kBuf = Shape<kParts>::kBuf;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long bars[4 * kStages + 5];
    __shared__ uint32_t s_tmem;
    __shared__ int s_gave_up;
    const int tid = threadIdx.x, warp = same(tid / 32), lane = tid % 32, rank = same((int)cluster_rank());
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char *stages = smem_raw + (smem - smem_u32(smem_raw));
    const uint32_t buf = smem + kStages * kStage + (warp & (kStoreWarps - 1)) * kBuf;
    int *tables = reinterpret_cast<int *>(stages + kStages * kStage + kStoreWarps * kBuf);
    const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, tfull = empty + 8 * kStages, tempty = tfull + 16,
                   done = tempty + 16, end_full = done + 8, end_peer = end_full + 8 * kStages;
    volatile int *gave_up = &s_gave_up;

    if (warp == kStoreWarps) tmem_alloc_pair(smem_u32(&s_tmem), 512);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mb_init(full + 8 * i, 1);
            mb_init(empty + 8 * i, 1);
            mb_init(end_full + 8 * i, 1);
            mb_init(end_peer + 8 * i, 2);  // both blocks have zeroed
        }
        for (int i = 0; i < 2; ++i) {
            mb_init(tfull + 8 * i, 1);
            mb_init(tempty + 8 * i, 2 * kStoreWarps);  // the storing warps of both blocks
        }
        mb_init(done, 1);
        s_gave_up = 0;
        mb_init_fence();
        tma_prefetch_map(&map_dy.blocks);
        tma_prefetch_map(&map_x.blocks);
    }
    tc_fence_before();
    cluster_sync();  // barriers and TMEM of both blocks are ready
    tc_fence_after();
    const uint32_t tmem = (uint32_t)same((int)s_tmem);
    grid_dependency_wait();  // offsets and rows come from earlier kernels
    grid_launch_dependents();
    const int mt = (a.F + 2 * kM - 1) / (2 * kM), per = mt * ((a.K + a.width - 1) / a.width);  // tiles of an expert
    const Groups g = make_groups<0, 0, 1>(tables, a.offsets, a.E, a.L, a.cap, a.most, a.pairs, 0,
                                       [&](int, int) { return per; }, [](int) { return 0; });  // syncs the block
    const int tiles = a.E * per;

    if constexpr (kParts) {
        if (warp >= kStoreWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    }
    if (warp == kStoreWarps) {  // loads
        Ring<kStages> r;
        uint32_t end_phase = 0;  // a bit per slot: the end barriers' next phases
        WaitLimit limit;
        bool ok = true;
        for (int t = blockIdx.x / 2; t < tiles && ok; t += gridDim.x / 2) {
            const int e = t / per;
            const Part p = get_part(a, mt, t % per);
            const int row = same(g.row[e]), count = same(g.count[e]), steps = (count + kP - 1) / kP;
            const int m0 = p.m0 + rank * kM, n0 = p.n0 + rank * (p.n / 2), m_cols = rank == 0 ? p.m_cols0 : p.m_cols1;
            const bool whole_m = m0 + kM <= a.F, whole_n = a.width == kN && p.n0 + kN <= a.K;
            limit.tile(steps);
            for (int k = 0; k < steps; ++k) {
                ok = mb_wait_warp(empty + 8 * r.slot, r.phase ^ 1u, gave_up, limit.polls());
                if (!ok) break;
                limit.waited();
                const bool ends = k + 1 == steps && count % 16 != 0;  // rows to be zeroed
                if (elect_one()) {
                    const uint32_t sa = smem + r.slot * kStage, sb = sa + kM / 64 * kCols;
                    const uint32_t bar = ends ? end_full + 8 * r.slot : at_leader(full + 8 * r.slot);
                    if (ends) mb_expect_tx(bar, (m_cols + p.n_cols) * kCols);
                    if (rank == 0) {
                        if (ends) mb_arrive(full + 8 * r.slot);
                        else mb_expect_tx(full + 8 * r.slot, (p.m_cols0 + p.m_cols1 + 2 * p.n_cols) * kCols);
                    }
                    if (whole_m) {
                        tma_load_3d_pair(sa, &map_dy.blocks, bar, 0, row + k * kP, m0 / 64);
                    } else {
                        for (int i = 0; i < m_cols; ++i)
                            tma_load_2d_pair(sa + i * kCols, &map_dy.cols, bar, m0 + i * 64, row + k * kP);
                    }
                    if (whole_n) {
                        tma_load_3d_pair(sb, &map_x.blocks, bar, 0, row + k * kP, n0 / 64);
                    } else {
                        for (int i = 0; i < p.n_cols; ++i)
                            tma_load_2d_pair(sb + i * kCols, &map_x.cols, bar, n0 + i * 64, row + k * kP);
                    }
                }
                __syncwarp();
                if (ends) end_phase ^= 1u << r.slot;
                r.next();
            }
        }
        if (rank == 0) drain_ring(full, r);  // of both blocks
        drain_ring(empty, r, limit.polls());  // in each block: its loads, and the leader's arrivals, the last of them `done`
        mb_drain(done, 0);
        for (int i = 0; i < kStages; ++i) mb_drain(end_full + 8 * i, (end_phase >> i & 1u) ^ 1u);
    } else if (warp == kStoreWarps + 1) {  // the leader's mma
        if (rank == 0) {
            Ring<kStages> r;
            Ring<2> acc;
            uint32_t end_phase = 0;
            WaitLimit limit;
            bool ok = true;
            for (int t = blockIdx.x / 2; t < tiles && ok; t += gridDim.x / 2) {
                const int e = t / per;
                const Part p = get_part(a, mt, t % per);
                const int count = same(g.count[e]), steps = (count + kP - 1) / kP;
                limit.tile(steps);
                if (steps == 0) continue;  // nothing to sum: the results are zeros
                const uint32_t desc = mma_desc(1, true, true, 2 * kM, p.n);
                const int part = kParts ? part_stages(kF32) : steps;  // stages that are summed in TMEM
                for (int k0 = 0; k0 < steps && ok; k0 += part) {
                    const uint32_t d = tmem + acc.slot * kN;
                    ok = mb_wait_warp(tempty + 8 * acc.slot, acc.phase ^ 1u, gave_up, limit.polls());
                    tc_fence_after();
                    limit.waited();
                    for (int k = k0; k < min(k0 + part, steps) && ok; ++k) {
                        const int left = min(kP, count - k * kP), slices = (left + 15) / 16;
                        ok = mb_wait_warp(full + 8 * r.slot, r.phase, gave_up, limit.polls());
                        if (left % 16 != 0 && ok) {
                            ok = mb_wait_warp_pair(end_peer + 8 * r.slot, end_phase >> r.slot & 1u, gave_up, limit.polls());
                            end_phase ^= 1u << r.slot;
                        }
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint32_t sa = smem + r.slot * kStage;
                            const uint64_t da = smem_operand(sa, kCols, 1024),
                                           db = smem_operand(sa + kM / 64 * kCols, kCols, 1024);
                            for (int i = 0; i < slices; ++i)  // 16 rows are 16 lines of 128 bytes
                                mma_bf16_pair(d, da + i * 128, db + i * 128, desc, k != k0 || i != 0);
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
    } else if (warp == kStoreWarps + 2) {  // zeroes behind the experts' last rows
        int slot = 0;
        uint32_t end_phase = 0;
        WaitLimit limit;
        bool ok = true;
        for (int t = blockIdx.x / 2; t < tiles && ok; t += gridDim.x / 2) {
            const int count = same(g.count[t / per]), steps = (count + kP - 1) / kP, left = count % kP;
            limit.tile(steps);
            if (count % 16 != 0) {
                const int last = (slot + steps - 1) % kStages;
                // the first wait since the last such tile
                ok = mb_wait_warp(end_full + 8 * last, end_phase >> last & 1u, gave_up, limit.polls());
                limit.waited();
                end_phase ^= 1u << last;
                const int words = (((left + 15) & ~15) - left) * 8;  // 16-byte words of the lines behind the last row
                for (int i = 0; i < (kM + kN / 2) / 64; ++i) {
                    uint4 *line = reinterpret_cast<uint4 *>(stages + last * kStage + i * kCols + left * 128);
                    for (int j = lane; j < words; j += 32) line[j] = make_uint4(0u, 0u, 0u, 0u);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mb_arrive_remote(at_leader(end_peer + 8 * last));
            }
            slot = (slot + steps) % kStages;
        }
    } else if constexpr (kParts) {
        if (warp < kStoreWarps) {
            // results: warp w holds rows 32 (w % 4).. of the block's half, one
            // per lane, and every other 32 columns, 2 i + w / 4
            asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
            const int quarter = warp & 3, half = warp >> 2;
            Ring<2> acc;
            WaitLimit limit;
            bool ok = true;
            for (int t = blockIdx.x / 2; t < tiles && ok; t += gridDim.x / 2) {
                const int e = t / per;
                const Part p = get_part(a, mt, t % per);
                const int steps = (same(g.count[e]) + kP - 1) / kP, n = min(a.width, a.K - p.n0);
                constexpr int kPart = part_stages(kF32);
                limit.tile(min(steps, kPart));
                float sum[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[i][j] = 0.f;
                for (int k0 = 0; k0 < steps; k0 += kPart) {
                    ok = mb_wait_warp(tfull + 8 * acc.slot, acc.phase, gave_up, limit.polls());
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t src = tmem + acc.slot * kN + ((uint32_t)(quarter * 32) << 16) + 32 * half;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (64 * i + 32 * half < n) {
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
                limit.waited();
                // 64 bytes of each row at a time, turned in shared memory so
                // that four lanes write them (chunks of 16 bytes swapped by
                // row against bank conflicts).  With 128 bytes at a time the
                // buffers take a stage's place: 324 us instead of 312 for 1 GB
                // of results.
                using Elem = std::conditional_t<kF32, float, __nv_bfloat16>;
                constexpr int kVec = 16 / sizeof(Elem), kPass = 64 / sizeof(Elem);
                const int r0 = lane / 4, chunk = lane & 3, f0 = p.m0 + rank * kM + quarter * 32;
                Elem *to = static_cast<Elem *>(a.dw) + ((int64_t)e * a.F + f0 + r0) * a.K + p.n0 + chunk * kVec;
                const int64_t step = (int64_t)8 * a.K;
                const int rows = a.F - f0 - r0, cols = n - chunk * kVec;
                const uint32_t put = buf + lane * 64, get = buf + r0 * 64 + ((chunk ^ ((r0 >> 1) & 3)) * 16);
#pragma unroll
                for (int i = 0; i < 128 / kPass; ++i) {
                    const int at = i * kPass, c0 = 64 * (at / 32) + 32 * half + at % 32;
                    if (c0 < n) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float *v = &sum[at / 32][at % 32 + kVec * q];
                            uint4 four;
                            if constexpr (kF32) {
                                four = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                                  __float_as_uint(v[3]));
                            } else {
                                uint32_t w[4];
#pragma unroll
                                for (int j = 0; j < 4; ++j) w[j] = bf16x2(__float_as_uint(v[2 * j]), __float_as_uint(v[2 * j + 1]));
                                four = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                            st_shared128(put + ((q ^ ((lane >> 1) & 3)) * 16), four);
                        }
                        __syncwarp();
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint4 v = ld_shared128(get + q * 512);
                            if (8 * q < rows && c0 < cols) *reinterpret_cast<uint4 *>(to + q * step + c0) = v;
                        }
                        __syncwarp();
                    }
                }
            }
        }
    } else {  // results: warp w holds rows 32w.. of the block's half, one per lane
        Ring<2> acc;
        WaitLimit limit;
        for (int t = blockIdx.x / 2; t < tiles; t += gridDim.x / 2) {
            const int e = t / per;
            const Part p = get_part(a, mt, t % per);
            const int steps = (same(g.count[e]) + kP - 1) / kP;
            const bool some = steps > 0;
            limit.tile(steps);
            if (some) {
                if (!mb_wait_warp(tfull + 8 * acc.slot, acc.phase, gave_up, limit.polls())) break;
                tc_fence_after();
                limit.waited();
            }
            const uint32_t src = tmem + acc.slot * kN + ((uint32_t)(warp * 32) << 16);
            const int f0 = p.m0 + rank * kM + warp * 32, n = min(a.width, a.K - p.n0);
            // 128 bytes of each row at a time, turned in shared memory so that
            // eight lanes write a row's 128 bytes (chunks of 16 bytes swapped
            // by row against bank conflicts)
            constexpr int kPass = 64, kElem = 2;
            const int r0 = lane / 8, chunk = lane & 7;
            unsigned char *to = static_cast<unsigned char *>(a.dw) +
                                (((int64_t)e * a.F + f0 + r0) * a.K + p.n0 + chunk * (16 / kElem)) * kElem;
            const int64_t step = (int64_t)4 * a.K * kElem;
            const int rows = a.F - f0 - r0, cols = n - chunk * (16 / kElem);
            for (int c0 = 0; c0 < n; c0 += kPass) {
#pragma unroll
                for (int h = 0; h < kPass / 32; ++h) {
                    uint32_t v[32];
                    if (some) {
                        tmem_load32(src + c0 + 32 * h, v);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0u;
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 16 / kElem) {
                        const uint4 q = make_uint4(bf16x2(v[j], v[j + 1]), bf16x2(v[j + 2], v[j + 3]),
                                                   bf16x2(v[j + 4], v[j + 5]), bf16x2(v[j + 6], v[j + 7]));
                        st_shared128(buf + lane * 128 + ((((32 * h + j) * kElem / 16) ^ (lane & 7)) * 16), q);
                    }
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 q = ld_shared128(buf + (i * 4 + r0) * 128 + ((chunk ^ ((i * 4 + r0) & 7)) * 16));
                    if (4 * i < rows && c0 < cols) *reinterpret_cast<uint4 *>(to + i * step + c0 * kElem) = q;
                }
                __syncwarp();
            }
            if (some) {
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

template <bool kParts, bool kF32>
cudaError_t launch(const ColumnMaps &map_dy, const ColumnMaps &map_x, Args a, cudaStream_t stream) {
    auto kern = expert_wgrad_kernel<kParts, kF32>;
    static thread_local PairCache cache;
    using S = Shape<kParts>;
    PairLaunch l(S::kThreads, S::kSmem + groups_bytes(1024), stream);
    cudaError_t e = cache.prepare(reinterpret_cast<const void *>(kern), l.cfg);
    if (e != cudaSuccess) return e;
    l.cfg.gridDim = dim3((unsigned)cache.blocks);
    // 128 columns where all tiles then still run at once: one expert of 8192
    // rows, K = F = 1024, f32, takes 36 us against 41; 64 gain no more
    const int64_t narrow = (int64_t)a.E * ((a.F + 2 * kM - 1) / (2 * kM)) * ((a.K + kN / 2 - 1) / (kN / 2));
    a.width = narrow <= cache.blocks / 2 ? kN / 2 : kN;
    l.cfg.dynamicSmemBytes = S::kSmem + groups_bytes(a.E);
    return cudaLaunchKernelEx(&l.cfg, kern, map_dy, map_x, a);
}

// `tile`: columns that one block loads.  Rows of fewer columns use `cols` alone.
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
    if (!encode_columns(&map_dy, dy, F, r.rows_total, kM) || !encode_columns(&map_x, x, K, r.rows_total, kN / 2))
        return cudaErrorInvalidValue;
    const Args a{r.offsets, dw, r.cap, r.most, r.pairs, r.E, r.L, K, F, kN};
    if (dw_f32) return launch<true, true>(map_dy, map_x, a, stream);
    return r.most > kWhole ? launch<true, false>(map_dy, map_x, a, stream) : launch<false, false>(map_dy, map_x, a, stream);
}

cudaError_t take_expert_wgrad_error(int *err) { return take_tc_error(err); }

}  // namespace moe
