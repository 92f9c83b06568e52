// Product of the experts' rows with matrices of 4-bit weights where an expert
// has few rows: bound by the bytes of the codes.
//
//   y[p][f] = r[e][f] sum_k x[p][k] (s[e][k/group][f] q[e][f][k])
//
// Codes go from memory to registers (16 bytes a lane, three steps ahead), become
// bf16 there (w4_ops.cuh) and are the A fragments of mma.sync as they are: a
// lane's word of eight consecutive elements serves two products of 16, the
// order of the reduction being free as long as the tokens' fragments have
// the same one.  tcgen05 would have to read them from TMEM, 128 rows by 16
// elements at a time, which takes it 64 to 70 cycles whatever the number of
// tokens: 32 weights a cycle where HBM brings 47.  mma.sync takes 2 cycles for
// 16 x 16 weights and eight tokens (measured), 128 weights a cycle.
//
// A block holds one expert's tokens, at most eight, in shared memory, in the
// order in which lanes read them, and walks through a run of the matrix's
// rows, 32 a warp at a time.  kSplit warps take the same rows and share their
// reduction by blocks of 128; the sums are added up in shared memory in the
// warps' order.
#include "expert_w4_internal.cuh"
#include "mem_ops.cuh"
#include "pdl.cuh"
#include "tc_ops.cuh"
#include "w4_ops.cuh"

namespace moe {
namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kTokShift = 3, kTok = 1 << kTokShift;
constexpr int kRows = 32;        // matrix rows of a warp's step: two of mma's 16
constexpr int kK = 128;          // its reduction elements: 16 bytes of codes a lane and row
constexpr int kPartSteps = 4;    // steps of a part of a sum: 512 elements
constexpr int kSums = kRows * kTok;
constexpr int kRed = 2 * kWarps * kSums * 4;  // bytes of the warps' sums, twice

struct Args {
    const int32_t *offsets;
    const uint8_t *x, *wq, *group_scales;
    const float *row_scales;
    void *y;
    int64_t cap, most, pairs;
    int E, L, K, F, wide, groups, group_shift;
    int split_shift, units;  // log2 of the warps that share rows; units of (16 / split) * 32 rows in a matrix
};

// Bytes of a token's line in shared memory: two lines that are read together start 64 bytes apart.
__host__ __device__ constexpr int line_bytes(int K) { return (K + kK - 1) / kK * (kK * 2) + 64; }

__device__ __forceinline__ void mma_m16n8k16(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct Unit {
    int i, tt, m;    // group, token tile, first row (or feature) of this warp's rows
    int row, n;      // first token row, tokens
};

__device__ __forceinline__ Unit get_unit(const Groups &g, int E, int i, int u, int units) {
    Unit r;
    r.i = same(find_group(g, E, i, u));
    const int at = u - same(g.prefix[r.i]), c = same(g.count[r.i]);
    r.tt = at / units;
    r.m = at - r.tt * units;
    r.row = same(g.row[r.i]) + (r.tt << kTokShift);
    r.n = min(kTok, c - (r.tt << kTokShift));
    return r;
}

// A warp's step: what a lane loads for it.
struct Step {
    uint4 codes[4];
    uint32_t scales[4];
};

template <bool kGated, bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
expert_w4_few_kernel(const Args a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const int tid = threadIdx.x, warp = same(tid / 32), lane = tid % 32;
    const int line = line_bytes(a.K);
    float *red = reinterpret_cast<float *>(smem_raw);
    unsigned char *tokens = smem_raw + kRed;
    int *tables = reinterpret_cast<int *>(tokens + kTok * line);
    grid_dependency_wait();  // offsets and rows come from earlier kernels
    grid_launch_dependents();
    const Groups g = make_groups<kTokShift, kTokShift, 1>(
        tables, a.offsets, a.E, a.L, a.cap, a.most, a.pairs, gridDim.x,
        [&](int c, int shift) { return ((c + (1 << shift) - 1) >> shift) * a.units; }, [](int) { return 0; });
    const int total = same(g.prefix[a.E]);
    const int lo = (int)((int64_t)total * blockIdx.x / gridDim.x), hi = (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x);
    if (lo == hi) return;  // the whole block

    const int split = 1 << a.split_shift, part = warp & (split - 1), sub = warp >> a.split_shift;
    const int per_unit = (kWarps >> a.split_shift) * (kGated ? kRows / 2 : kRows);  // rows (or features) of a unit
    const int blocks = (a.K + kK - 1) / kK, rest = blocks & (split - 1);
    const int gr = lane >> 2, t = lane & 3;  // row of a fragment's eight, place in the four lanes of a row
    const int64_t pitch = a.K / 2;           // bytes of a row's codes

    // The warp's steps, in order: blocks part', part' + split, ... of every unit, part' turned from unit to unit
    // so that all warps get the same number in the long run.
    struct Cursor {
        int u, kb;
    };
    auto first_block = [&](int u) { return (int)((uint32_t)part + (uint32_t)u * (uint32_t)rest) & (split - 1); };
    Cursor next{lo, first_block(lo)};
    int next_group = 0;
    const uint8_t *base = nullptr, *sbase = nullptr;  // of the lane's first row
    uint32_t rows_ok = 0;                             // which of its four rows there are
    auto open = [&] {  // the unit of `next`
        const Unit w = get_unit(g, a.E, next_group, next.u, a.units);
        next_group = w.i;
        const int f = w.m * per_unit + sub * (kGated ? kRows / 2 : kRows) + gr;
        base = a.wq + ((int64_t)w.i * a.wide + f) * pitch + t * 16;
        sbase = a.group_scales + (int64_t)w.i * a.groups * a.wide + f;
        rows_ok = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) rows_ok |= (uint32_t)(f + (kGated ? (i & 1) * 8 : i * 8) < a.F) << i;
    };
    auto fetch = [&](Step &s) {
        if (next.u < hi) {
            const int k = next.kb * kK + t * 32;
            const int64_t group = (int64_t)(k >> a.group_shift) * a.wide;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t row = kGated ? (i & 1) * 8 + (i >> 1) * (int64_t)a.F : i * 8;
                const bool there = ((rows_ok >> i) & 1u) && k < a.K;
                s.codes[i] = there ? ld_stream(reinterpret_cast<const uint4 *>(base + row * pitch + next.kb * (kK / 2)))
                                   : make_uint4(0u, 0u, 0u, 0u);
                s.scales[i] = there ? __ldg(sbase + group + row) : 0u;
            }
            next.kb += split;
            if (next.kb >= blocks) {
                ++next.u;
                next.kb = first_block(next.u);
                if (next.u < hi) open();
            }
        }
    };
    open();
    Step s0, s1, s2;
    fetch(s0);
    fetch(s1);
    fetch(s2);

    float acc[8], sum[8];
    int u = lo, kb = first_block(lo), steps = 0, held_i = -1, held_tt = -1, buf = 0;
    Unit w = get_unit(g, a.E, 0, lo, a.units);
    // Sums of the finished unit: element j of a warp's 256 lies at (j / 32: fragment register, j % 32: lane).
    auto row_of = [&](int j) { return ((j >> 5 & 4) << 2) + ((j & 31) >> 2) + ((j >> 5 & 2) << 2); };
    auto begin = [&] {
        if (w.i != held_i || w.tt != held_tt) {  // other tokens
            __syncthreads();                     // nobody reads the old ones any more
            held_i = w.i, held_tt = w.tt;
            const int chunks = blocks * (kK / 8);
            for (int j = tid; j < kTok * chunks; j += kThreads) {
                const int tok = j / chunks, q = j - tok * chunks;
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (tok < w.n && q * 8 < a.K)
                    v = __ldg(reinterpret_cast<const uint4 *>(a.x + ((int64_t)(w.row + tok) * a.K + q * 8) * 2));
                // lane t reads chunk 4 t + i of a block of 16 in its i-th turn: stored in that order
                *reinterpret_cast<uint4 *>(tokens + tok * line + (q >> 4) * 256 + (q & 3) * 64 + (q >> 2 & 3) * 16) = v;
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = sum[i] = 0.f;
    };
    begin();
    const uint32_t mine = smem_u32(tokens) + gr * line + t * 16;
    bool more = true;
    auto step = [&](Step &s) {
        const W4Scale sc[4] = {W4Scale(s.scales[0]), W4Scale(s.scales[1]), W4Scale(s.scales[2]), W4Scale(s.scales[3])};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint4 b = ld_shared128(mine + kb * 256 + j * 64);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                auto word = [&](const uint4 &v) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; };
                uint32_t p[4], q[4];
                dequant8(word(s.codes[2 * m]), sc[2 * m], p);
                dequant8(word(s.codes[2 * m + 1]), sc[2 * m + 1], q);
                mma_m16n8k16(acc + 4 * m, p[0], q[0], p[1], q[1], b.x, b.y);
                mma_m16n8k16(acc + 4 * m, p[2], q[2], p[3], q[3], b.z, b.w);
            }
        }
        fetch(s);
        kb += split;
        if (++steps == kPartSteps || kb >= blocks) {
            steps = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += acc[i], acc[i] = 0.f;
        }
        if (kb < blocks) return;
        // the unit is done: the warps' sums, in their order
        float *to = red + buf * (kWarps * kSums);
#pragma unroll
        for (int i = 0; i < 8; ++i) to[warp * kSums + i * 32 + lane] = sum[i];
        __syncthreads();
        constexpr int kOut = kGated ? kSums / 2 : kSums;
        for (int j = tid; j < (kWarps >> a.split_shift) * kOut; j += kThreads) {
            const int which = j / kOut, jj = j % kOut;
            const int f = w.m * per_unit + which * (kGated ? kRows / 2 : kRows) + row_of(jj);
            const int tok = 2 * (jj & 3) + (jj >> 5 & 1);
            if (tok >= w.n || f >= a.F) continue;
            const float *from = to + (which << a.split_shift) * kSums + jj;
            const float *rs = a.row_scales + (int64_t)w.i * a.wide + f;
            float v = 0.f;
            for (int i = 0; i < split; ++i) v += from[i * kSums];
            v *= __ldg(rs);
            const int64_t at = (int64_t)(w.row + tok) * a.F + f;
            if constexpr (kGated) {
                float up = 0.f;
                for (int i = 0; i < split; ++i) up += from[i * kSums + kSums / 2];
                static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(silu_mul(v, up * __ldg(rs + a.F)));
            } else if constexpr (kF32) {
                static_cast<float *>(a.y)[at] = v;
            } else {
                static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(v);
            }
        }
        buf ^= 1;
        if (++u == hi) {
            more = false;
            return;
        }
        kb = first_block(u);
        w = get_unit(g, a.E, w.i, u, a.units);
        begin();
    };
    while (more) {
        step(s0);
        if (more) step(s1);
        if (more) step(s2);
    }
}

template <bool kGated, bool kF32>
cudaError_t launch(const Args &a, cudaStream_t stream) {
    auto kern = expert_w4_few_kernel<kGated, kF32>;
    static thread_local AttrCache attr;
    const int smem = kRed + kTok * line_bytes(a.K) + groups_bytes(a.E);
    cudaError_t e = attr.allow_smem(reinterpret_cast<const void *>(kern), kMostSharedW4);
    if (e != cudaSuccess) return e;
    const int sms = sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    cudaLaunchAttribute pdl[1] = {pdl_attribute()};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

bool expert_w4_few(const ExpertRows &r, int K, int F, int gated) {
    const int64_t wide = gated ? 2 * (int64_t)F : F;
    return r.pairs <= 4 * (int64_t)r.E && kRed + kTok * line_bytes(K) + groups_bytes(r.E) <= kMostSharedW4 &&
           (r.E + r.pairs / kTok) * (wide / kRows + 1) < (1 << 30);  // units are counted in 32 bits
}

cudaError_t launch_expert_w4_few(const ExpertRows &r, int K, int F, int gated, int group, const void *x, const void *wq,
                                 const void *group_scales, const float *row_scales, void *y, int y_f32,
                                 cudaStream_t stream) {
    const int blocks = (K + kK - 1) / kK;
    int split = 0;
    while (split < 4 && (2 << split) <= blocks) ++split;
    const int per_unit = (kWarps >> split) * (gated ? kRows / 2 : kRows);
    int shift = 5;
    while ((1 << shift) < group) ++shift;
    const Args a{r.offsets, static_cast<const uint8_t *>(x), static_cast<const uint8_t *>(wq),
                 static_cast<const uint8_t *>(group_scales), row_scales, y, r.cap, r.most, r.pairs,
                 r.E, r.L, K, F, gated ? 2 * F : F, K / group, shift, split, (F + per_unit - 1) / per_unit};
    if (gated) return launch<true, false>(a, stream);
    return y_f32 ? launch<false, true>(a, stream) : launch<false, false>(a, stream);
}

}  // namespace moe
