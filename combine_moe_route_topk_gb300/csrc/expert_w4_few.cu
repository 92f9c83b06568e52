// Product of the experts' rows with matrices of 4-bit weights where an expert
// has few rows: bound by the bytes of the codes.
//
//   y[p][f] = r[e][f] sum_k x[p][k] (s[e][k/group][f] q[e][f][k])
//
// Codes come to shared memory by TMA, become bf16 in registers (w4_ops.cuh) and
// are the A fragments of mma.sync as they are: a lane's word of eight
// consecutive elements serves two products of 16, the order of the reduction
// being free as long as the tokens' fragments have the same one.  mma.sync takes
// 2 cycles of an SM for 16 x 16 weights and eight tokens (measured), 128 weights a
// cycle where HBM brings 44.  The kernel runs at 33 (32 of 64 experts, 7168 x 4096
// each, one token: 100 us, loads alone 82, floor 74; two stages of codes are as
// fast as five, half the mma 4 us less) and nothing is used up: a warp takes some 300
// instructions for 32 x 128 weights, 112 of them the shifts and logic that take nibbles
// apart (each two cycles of its pipe) and 16 mma, of which the SM could issue
// 54 weights' worth a cycle.  With 32 tokens of 64 experts (200 to 218 us, floor 148) 60 % of the
// issue slots are in use, 58 % of the integer and logic pipe, 25 % of the tensor pipe, 63 % of
// HBM.  What is left are waits: four warps a scheduler, of which 1.5 on average
// could issue, wait for that pipe, for the results of one another's instructions
// and for shared memory.  The tensor core proper
// would take the same bf16 from TMEM by tiles of 128 rows: more rows at once than
// a small call has for an SM.
//
// A block holds one expert's tokens, at most eight, in shared memory, in the
// order in which lanes read them, and walks through a run of the matrices'
// rows, in granules of 32, its share of all there are.  A unit is a few
// granules; the warps of one share its reduction by blocks of 128, and their
// sums are added up in shared memory in the warps' order.  Two more warps load, one of them the groups' scales: their copies in
// the same warp as the codes' loads held those up (loads alone 284 us against
// 187, 32 tokens of 64 experts, 7168 x 4096).
#include "expert_w4_internal.cuh"
#include "mem_ops.cuh"
#include "pdl.cuh"
#include "tc_ops.cuh"
#include "w4_ops.cuh"
#include "w4_rule.cuh"

namespace moe {
namespace {

using namespace w4_few;
constexpr int kThreads = 32 * (kWarps + 2);
constexpr int kPartSteps = 4;    // steps of a part of an f32 result's sum: 512 elements (bf16 ones: all of a warp's, at most 2^14)

struct Args {
    const int32_t *offsets;
    const uint8_t *x, *group_scales;
    const float *row_scales;
    void *y;
    int64_t cap, most, pairs;
    int E, L, K, F, wide, groups, group_shift;
    int least_shift, most_shift;  // log2 of the warps that share a granule: its limits
    int granules;            // of a matrix
    int stages, lines;       // stages of codes, lines of tokens in shared memory
    uint32_t grid_inverse;   // 2^32 / blocks, above
    int first_map;           // of the largest box that a unit can need
};

__device__ __forceinline__ void mma_m16n8k16(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Rows of codes by boxes of 128, 64 and 32.
struct CodeMaps {
    CUtensorMap m[3];
};

struct Unit {
    int i, tt;     // group, token tile
    int m, count;  // first granule in the matrix, granules
    int shift;     // log2 of the warps that share one of them
    int row, n;    // first token row, tokens
};

// How many granules of the next `left` a unit takes: as many as least_shift allows,
// or the power of two below, as long as every warp of a granule has work.  (7
// granules of 56 blocks of 128: 4, 2 and 1 take a warp 14 + 7 + 4 steps, 4 and 3 would 28.
// Two tokens of 8 of 64 experts, K = 7168, F = 2048 gated: 60 us, before 64.)
__device__ __forceinline__ void set_count(Unit &w, int left, int least_shift, int most_shift) {
    w.count = min(kWarps >> least_shift, left);
    w.shift = max(least_shift, min(most_shift, 4 - (31 - __clz(w.count))));
    if (w.count > kWarps >> most_shift) w.count = kWarps >> w.shift;
}

// The unit at place p of all granules, of which the block's end at hi.
__device__ __forceinline__ Unit get_unit(const Groups &g, int i, int p, int hi, const Args &a) {
    Unit r;
    r.i = same(find_group(g, a.E, i, p));
    const int at = p - same(g.prefix[r.i]), c = same(g.count[r.i]);
    r.tt = at < a.granules ? 0 : at / a.granules;
    r.m = at - r.tt * a.granules;
    set_count(r, min(a.granules - r.m, hi - p), a.least_shift, a.most_shift);
    r.row = same(g.row[r.i]) + (r.tt << kTokShift);
    r.n = min(kTok, c - (r.tt << kTokShift));
    return r;
}

template <bool kGated, bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
expert_w4_few_kernel(const __grid_constant__ CodeMaps maps, const Args a) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long bars[kBars];
    __shared__ int s_gave_up;
    const int tid = threadIdx.x, warp = same(tid / 32), lane = tid % 32;
    const int line = line_bytes(a.K);
    const uint32_t codes = (smem_u32(smem_raw) + 1023u) & ~1023u, scales_at = codes + a.stages * kCodes;
    unsigned char *behind = smem_raw + (scales_at + a.stages * kScales - smem_u32(smem_raw));
    float *red = reinterpret_cast<float *>(behind);
    unsigned char *tokens = behind + kRed + kZeros;
    int *tables = reinterpret_cast<int *>(tokens + a.lines * line);
    const uint32_t full = smem_u32(bars), empty = full + 8 * kMostStages, summed = empty + 8 * kMostStages,
                   placed = summed + 8;
    volatile int *gave_up = &s_gave_up;
    if (tid == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mb_init(full + 8 * i, 1 + 32);  // the codes' bytes, and the lanes that copy scales
            mb_init(empty + 8 * i, kWarps);
        }
        mb_init(summed, kWarps);
        mb_init(placed, kWarps);
        s_gave_up = 0;
        mb_init_fence();
        for (int i = a.first_map; i < 3; ++i) tma_prefetch_map(&maps.m[i]);
    }
    grid_dependency_wait();  // offsets and rows come from earlier kernels
    grid_launch_dependents();
    if (tid < kZeros / 4) reinterpret_cast<int *>(behind + kRed)[tid] = 0;
    const Groups g = make_groups<kTokShift, kTokShift, 1>(
        tables, a.offsets, a.E, a.L, a.cap, a.most, a.pairs, gridDim.x,
        [&](int c, int shift) { return ((c + (1 << shift) - 1) >> shift) * a.granules; }, [](int) { return 0; });
    // A block's granules are a run of all of them: it rarely changes the expert.
    const int total = same(g.prefix[a.E]);
    const int grid = gridDim.x, at = blockIdx.x;
    int each = (int)__umulhi(total, a.grid_inverse), rest = total - each * grid;
    if (rest < 0) --each, rest += grid;  // total < 2^30: one too many at most
    const int lo = at * each + (int)__umulhi(at * rest, a.grid_inverse);  // total * at / grid; products below grid^2 are exact
    const int hi = (at + 1) * each + (int)__umulhi((at + 1) * rest, a.grid_inverse);
    if (lo == hi) return;  // the whole block

    constexpr int kCols = kGated ? kRows / 2 : kRows;  // result columns of a granule
    const int blocks = (a.K + kK - 1) / kK;
    auto advance = [&](Unit &w, int p) {  // to the unit at p, the one behind it
        w.m += w.count;
        if (w.m == a.granules) w = get_unit(g, w.i, p, hi, a);
        else set_count(w, min(a.granules - w.m, hi - p), a.least_shift, a.most_shift);
    };
    Unit w = get_unit(g, 0, lo, hi, a);
    int slot = 0;
    uint32_t phase = 0;
    auto next_slot = [&] {
        if (++slot == a.stages) slot = 0, phase ^= 1u;
    };

    if (warp >= kWarps) {  // loads
        const bool scales = warp > kWarps;
        bool ok = true;
        for (int p = lo; p < hi && ok;) {
            const int split = 1 << w.shift, unit_rows = (kWarps * kRows) >> w.shift, rounds = (blocks + split - 1) >> w.shift;
            // A lane copies eight rows' scales of every `step`-th group.
            const int step = split / 2, first = lane >> (6 - w.shift), q = lane & ((64 >> w.shift) - 1);
            const int groups = (split * kK) >> a.group_shift;  // of a stage
            const int f0 = w.m * kCols, f = kGated ? f0 + (q >> 1) * 8 : f0 + q * 8;
            const uint8_t *from = a.group_scales + (int64_t)w.i * a.groups * a.wide + (int64_t)first * a.wide;
            if (f < a.F) from += f + (kGated && (q & 1) ? a.F : 0);
            for (int r = 0; r < rounds; ++r) {
                ok = mb_wait_warp(empty + 8 * slot, phase ^ 1u, gave_up);
                if (!ok) break;
                const uint32_t bar = full + 8 * slot;
                if (scales) {
                    const int left = a.groups - r * groups;
                    uint32_t to = scales_at + slot * kScales + first * unit_rows + q * 8;
                    for (int b = first; b < groups; b += step, to += step * unit_rows, from += (int64_t)step * a.wide) {
                        const bool there = f < a.F && b < left;
                        copy_async<8>(to, there ? from : a.group_scales, there ? 8 : 0);
                    }
                    copy_arrive(bar);
                } else if (elect_one()) {
                    // boxes of 256 elements (a line of 128 bytes) by up to 128 rows
                    const int b0 = r * split / 2, b1 = min(b0 + split / 2, (blocks + 1) / 2);
                    mb_expect_tx(bar, (b1 - b0) * w.count * kRows * 128);
                    for (int b = b0; b < b1; ++b) {
                        const uint32_t dst = codes + slot * kCodes + (b - b0) * unit_rows * 128;
                        for (int q = 0; q < w.count * kRows;) {
                            const int left = w.count * kRows - q, i = max(a.first_map, left >= 128 ? 0 : left >= 64 ? 1 : 2);
                            if constexpr (kGated) tma_load_5d(dst + q * 128, &maps.m[i], bar, b * 128, 0, 0, (f0 + q / 2) / 8, w.i);
                            else tma_load_3d(dst + q * 128, &maps.m[i], bar, b * 128, f0 + q, w.i);
                            q += 128 >> i;
                        }
                    }
                }
                __syncwarp();
                next_slot();
            }
            p += w.count;
            if (p < hi) advance(w, p);
        }
        // nothing may still be landing here when the block ends
        long long left = kPolls;
        for (int i = 0; i < a.stages; ++i, next_slot()) {
            while (!mb_try(full + 8 * slot, phase ^ 1u) && left > 0) --left;
        }
    } else {
        const int gr = lane >> 2, t = lane & 3;  // row of a fragment's eight, place in the four lanes of a row
        // A lane's four rows (of two fragments, eight rows apart in each) are four that follow one another in the
        // matrix: their scales are one word, and lanes that read codes at once read different places of the
        // swizzled lines.
        const uint32_t magic = w4_magic(), zeros = smem_u32(behind + kRed) + t * 16, held_at = smem_u32(tokens) + gr * line + t * 16;
        float acc[8], sum[8];
        int held_i = -1, held_tt = -1, buf = 0;
        uint32_t x_at = zeros, x_step = 0, summed_phase = 0, placed_phase = 0;  // the lane's token, from block to block
        Unit done = w;
        bool pending = false, ok = true;  // pending: `done` has sums that are not added up yet

        // The unit `done`: its warps' sums are added up in their order.  Element j of a warp's 256 lies at (j / 32: fragment register, j % 32: lane).
        auto finish = [&] {
            pending = false;
            ok = mb_wait_warp(summed, summed_phase, gave_up, kPolls + blocks * kStepPolls);
            summed_phase ^= 1u;
            if (!ok) return;
            const float *from = red + (buf ^ 1) * (kWarps * (kSumLine + kRows)), *scales = from + kWarps * kSumLine;
            const int split = 1 << done.shift, most = kWarps >> done.shift;
            for (int j = tid; j < most * kSumLine; j += 32 * kWarps) {
                int e = j;
                if constexpr (kGated) e = (e & ~15) + (e & 1) * 8 + (e >> 1 & 7);  // gate and up in neighbouring lanes
                const int which = e >> 8, i = e >> 5 & 7, l = e & 31;
                const float *at = from + (which << done.shift) * kSumLine + (e & 255);
                float v = 0.f;
                for (int k = 0; k < split; k += 2) v = v + at[k * kSumLine] + at[(k + 1) * kSumLine];
                // the row of the granule; of a gated one's, 8 are gate rows and the next 8 the same features' up rows
                const int row = 4 * (l >> 2) + (i >> 2) * 2 + (i >> 1 & 1);
                const int r = which * kCols + (kGated ? (row >> 4) * 8 + (row & 7) : row);
                const bool is_up = kGated && (row & 8);
                v *= scales[r + (is_up ? most * kCols : 0)];
                float up = 0.f;
                if constexpr (kGated) up = __shfl_xor_sync(0xffffffffu, v, 1);
                const int f = done.m * kCols + r, tok = 2 * (l & 3) + (i & 1);
                if (which >= done.count || tok >= done.n || f >= a.F || is_up) continue;
                const int64_t to = (int64_t)(done.row + tok) * a.F + f;
                if constexpr (kGated) static_cast<__nv_bfloat16 *>(a.y)[to] = __float2bfloat16_rn(silu_mul(v, up));
                else if constexpr (kF32) static_cast<float *>(a.y)[to] = v;
                else static_cast<__nv_bfloat16 *>(a.y)[to] = __float2bfloat16_rn(v);
            }
        };

        for (int p = lo; p < hi && ok;) {
            const int split = 1 << w.shift, most = kWarps >> w.shift, unit_rows = most * kRows, rounds = (blocks + split - 1) >> w.shift;
            const int part = warp & (split - 1), sub = warp >> w.shift;
            const bool fresh = w.i != held_i || w.tt != held_tt;
            if (fresh) {                             // other tokens
                if (pending) finish();               // nobody reads the old ones any more
                if (!ok) break;
                held_i = w.i, held_tt = w.tt;
                const int chunks = blocks * (kK / 8);
                const uint8_t *from = a.x + (int64_t)w.row * a.K * 2;
                for (int tok = 0; tok < w.n; ++tok, from += (int64_t)a.K * 2) {
                    for (int q = tid; q < chunks; q += 32 * kWarps) {
                        // lane t reads chunk 4 t + i of a block of 16 in its i-th turn: stored in that order
                        const int to = tok * line + (q >> 4) * 256 + (q & 3) * 64 + (q >> 2 & 3) * 16;
                        copy_async<16>(smem_u32(tokens) + to, q * 8 < a.K ? from + q * 16 : a.x, q * 8 < a.K ? 16 : 0);
                    }
                }
                x_at = gr < w.n ? held_at : zeros;
                x_step = gr < w.n ? 2 * kK : 0;
            }
            float scale = 0.f;  // of the thread's row of the unit, gate rows first
            {
                const int r = kGated && tid >= most * kCols ? tid - most * kCols : tid, f = w.m * kCols + r;
                if (r < w.count * kCols && f < a.F) scale = __ldg(a.row_scales + (int64_t)w.i * a.wide + f + (r != tid ? a.F : 0));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = sum[i] = 0.f;
            const int mine = sub < w.count ? (blocks - part + split - 1) >> w.shift : 0;  // blocks of this warp
            const int ch = ((part & 1) * 4 + t) ^ ((gr & 1) * 4);  // the lane's chunk of its first row's line
            uint32_t codes_at[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                codes_at[i] = codes + (part >> 1) * unit_rows * 128 + (sub * kRows + 4 * gr + i) * 128 + ((ch ^ i) << 4);
            const uint32_t scale_at = scales_at + ((part * kK + t * 32) >> a.group_shift) * unit_rows + sub * kRows + 4 * gr;
            uint32_t x = x_at + part * x_step;
            if (fresh) {  // what a unit needs besides was done while they were on their way
                asm volatile("cp.async.wait_all;" ::: "memory");
                __syncwarp();
                if (lane == 0) mb_arrive(placed);
                ok = mb_wait_warp(placed, placed_phase, gave_up);
                if (!ok) break;
                placed_phase ^= 1u;
            }
            for (int r = 0; r < mine; ++r, x += x_step << w.shift) {
                ok = mb_wait_warp(full + 8 * slot, phase, gave_up);
                if (!ok) break;
                uint4 c[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) c[i] = ld_shared128(codes_at[i] + slot * kCodes);
                const uint32_t sc = ld_shared32(scale_at + slot * kScales);
                if (lane == reader_lane(c[0].x ^ c[1].x ^ c[2].x ^ c[3].x ^ sc)) mb_arrive(empty + 8 * slot);
                next_slot();
                const W4Scales s01(sc & 0xffff), s23(sc >> 16);
                const W4Scale s[4] = {s01.first, s01.second, s23.first, s23.second};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 b = ld_shared128(x + j * 64);
                    auto word = [&](const uint4 &v) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; };
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        uint32_t top[4], low[4];  // the lane's row of the fragment's first eight, of its second
                        dequant8(word(c[2 * m]), s[2 * m], magic, top);
                        dequant8(word(c[2 * m + 1]), s[2 * m + 1], magic, low);
                        mma_m16n8k16(acc + 4 * m, top[0], low[0], top[1], low[1], b.x, b.y);
                        mma_m16n8k16(acc + 4 * m, top[2], low[2], top[3], low[3], b.z, b.w);
                    }
                }
                if (kF32 && ((r & (kPartSteps - 1)) == kPartSteps - 1 || r == mine - 1)) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum[i] += acc[i], acc[i] = 0.f;
                }
            }
            for (int r = mine; r < rounds && ok; ++r) {  // of others alone
                ok = mb_wait_warp(full + 8 * slot, phase, gave_up);
                if (ok && lane == 0) mb_arrive(empty + 8 * slot);
                next_slot();
            }
            // The unit before is finished only now: warps that got a block more or less than others need not wait.
            if (ok && pending) finish();
            if (!ok) break;
            float *to = red + buf * (kWarps * (kSumLine + kRows));
#pragma unroll
            for (int i = 0; i < 8; ++i) to[warp * kSumLine + i * 32 + lane] = kF32 ? sum[i] : acc[i];
            to[kWarps * kSumLine + tid] = scale;
            __syncwarp();
            if (lane == 0) mb_arrive(summed);
            buf ^= 1;
            pending = true;
            done = w;
            p += w.count;
            if (p < hi) advance(w, p);
        }
        if (ok && pending) finish();
    }
    __syncthreads();
    if (tid == 0 && s_gave_up) record_timeout();
}

template <bool kGated, bool kF32>
cudaError_t launch(const CodeMaps &maps, const Args &a, cudaStream_t stream) {
    auto kern = expert_w4_few_kernel<kGated, kF32>;
    static thread_local AttrCache attr;
    cudaError_t e = attr.allow_smem(reinterpret_cast<const void *>(kern), kMostShared);
    if (e != cudaSuccess) return e;
    const int sms = sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    cudaLaunchAttribute pdl[1] = {pdl_attribute()};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = 1024 + a.stages * (kCodes + kScales) + kRed + kZeros + a.lines * line_bytes(a.K) + groups_bytes(a.E);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, maps, a);
}

}  // namespace

cudaError_t launch_expert_w4_few(const ExpertRows &r, int K, int F, int gated, int group, const void *x, const void *wq,
                                 const void *group_scales, const float *row_scales, void *y, int y_f32,
                                 cudaStream_t stream) {
    const int blocks = (K + kK - 1) / kK;
    const int cols = gated ? kRows / 2 : kRows, granules = (F + cols - 1) / cols;
    // Four warps share a granule, so that a block's units are 128 rows: whole
    // boxes and lines of scales.  More, where a block has less than that to do
    // (one matrix of 4096 x 7168: 15 us with 16 warps a granule, 17 with four),
    // as long as each of them has two blocks of 128.
    const int least = blocks > 2 ? 2 : 1;  // two at least: a line of shared memory has two blocks
    int most = least;
    while (most < 4 && (4 << most) <= blocks) ++most;
    // A block's share bounds its units: of one granule, 32 rows, one map will do.
    const int64_t sms = sm_count(), share = sms > 0 ? (most_granules(r, F, gated) + sms - 1) / sms : 0;
    if (sms < 2) return cudaErrorInvalidDevice;
    const int first = share >= 4 ? 0 : share >= 2 ? 1 : 2;
    CodeMaps maps;
    for (int i = 0; i < 3; ++i)
        if (i >= first && !encode_w4(&maps.m[i], wq, r.E, K, F, gated, 128 >> i)) return cudaErrorInvalidValue;
    int shift = 5;
    while ((1 << shift) < group) ++shift;
    const int lines = lines_of(r);
    const Args a{r.offsets, static_cast<const uint8_t *>(x), static_cast<const uint8_t *>(group_scales), row_scales, y,
                 r.cap, r.most, r.pairs, r.E, r.L, K, F, gated ? 2 * F : F, K / group, shift, least,
                 most, granules, stages_of(r, K, lines), lines, (uint32_t)(0xffffffffu / sms + 1), first};
    if (gated) return launch<true, false>(maps, a, stream);
    return y_f32 ? launch<false, true>(maps, a, stream) : launch<false, false>(maps, a, stream);
}

cudaError_t take_expert_w4_few_error(int *err) { return take_tc_error(err); }

}  // namespace moe
