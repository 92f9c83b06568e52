// Which kernel takes a batch of the product with 4-bit weights, in tiles of how
// many tokens, by the dimensions and the number of SMs alone: host arithmetic,
// apart from the kernels so that tests can evaluate it for what they call.
#pragma once

#include "expert_internal.cuh"
#include "tc_ops.cuh"

namespace moe {

// Dynamic shared memory that a block may have beside its `bars` barriers and the
// other static words (two of the kernel's own, two of make_groups).
constexpr int most_shared_w4(int bars) { return 227 * 1024 - (8 * bars + 64); }

// The kernel for experts with few rows (expert_w4_few.cu).
namespace w4_few {
constexpr int kWarps = 16;       // that consume codes
constexpr int kTokShift = 3, kTok = 1 << kTokShift;
constexpr int kRows = 32;        // matrix rows of a granule, which a warp takes: two of mma's 16
constexpr int kK = 128;          // reduction elements of its step: 16 bytes of codes a lane and row
constexpr int kCodes = kWarps * kRows * kK / 2, kScales = kWarps * kRows * kK / 32;  // bytes of a stage: a step of every warp
constexpr int kMostStages = 6, kBars = 2 * kMostStages + 2;
constexpr int kMostShared = most_shared_w4(kBars);
constexpr int kSumLine = kRows * kTok;  // a warp's sums
constexpr int kRed = 2 * kWarps * (kSumLine + kRows) * 4;  // bytes of the warps' sums and of the rows' scales, twice
constexpr int kZeros = 256;           // bytes that stand for the tokens of a fragment that are not there

// Bytes of a token's line in shared memory: two lines that are read together start 64 bytes apart.
__host__ __device__ constexpr int line_bytes(int K) { return (K + kK - 1) / kK * (kK * 2) + 64; }
inline int lines_of(const ExpertRows &r) { return r.most < kTok ? (int)r.most : kTok; }
// Stages of codes that fit beside the tokens (fewer than two: the kernel does not take the batch).
inline int stages_of(const ExpertRows &r, int K, int lines) {
    const int left = kMostShared - 1024 - kRed - kZeros - groups_bytes(r.E) - lines * line_bytes(K);
    const int n = left / (kCodes + kScales);
    return n < kMostStages ? n : kMostStages;
}
// Granules of all token tiles, at most.
inline int64_t most_granules(const ExpertRows &r, int F, int gated) {
    const int64_t cols = gated ? kRows / 2 : kRows, active = r.pairs < r.E ? r.pairs : r.E;
    return (active + (r.pairs - active) / kTok) * ((F + cols - 1) / cols);
}
}  // namespace w4_few

// The kernel in tiles of 64 tokens or more (expert_w4.cu).
namespace w4_tile {
constexpr int kM = 128;            // matrix rows of a tile
constexpr int kK = 128;            // reduction elements of a unit: what one slot of TMEM and one of token rows hold
constexpr int kUnits = 2;          // units of a stage of codes: 256 codes, one 128-byte line of a row
}  // namespace w4_tile

// Whether sums are taken in parts.
inline bool w4_parts(int K, int gated, int y_f32) { return K > kWhole || (y_f32 && !gated); }

struct W4Form {
    int tokens;  // most tokens of a tile: 8 (the kernel for few rows), 64, or 160 (128 for sums in parts)
    int split;   // blocks that share a tile's reduction
};

// Where all tiles of 64 tokens leave half or more of the SMs idle, two or four blocks share one (one matrix of
// 4096 x 7168, 32, 64 and 128 tokens: 18, 21 and 21 us alone, 13, 15 and 15 in twos, 11, 12 and (not all at once) 16 in fours).
//
// The kernel for few rows where an SM has little to do at most: here `share`
// granules of 32 rows by eight tokens, there `rounds` of tiles of 128 rows by 64
// tokens, each in `split` blocks.  A tile takes as long as some five granules.
// Here against there, us (granules : tiles / split), K = 7168, F = 2048 gated, 8 of
// 64 experts a token: 1, 2, 4, 8 tokens 37 : 44 (7 : 2), 60 : 72 (14 : 4), 101 : 105
// (27 : 7), 148 : 166 (54 : 14), 16, 32, 48 179 : 187 (61 : 14), 212 : 218 (75 : 15), 246 : 232
// (88 : 15); K = 2048, F = 7168, 8, 24, 48 tokens 87 : 85 (95 : 24), 115 : 113 (118 : 25),
// 141 : 121 (154 : 26); one matrix of 4096 x 7168, 1, 8, 16, 32 tokens 13 : 17, 15 : 17,
// 17 : 17, 23 : 17 (1, 1, 2, 4 : 1 / 4); 2 of 8 experts of 2048 x 4096, 8 tokens 17 : 19 (4 : 1),
// of 4096 x 4096, 32 tokens 35 : 28 (13 : 2).
//
// Else tiles of 64 tokens up to 48 rows an expert, or where all of them run at once: 48 and 64 rows (64 experts, K = 7168,
// F = 2048 gated) take 232 and 330 us with them, 268 and 273 with tiles of 160; one matrix of 4096 x 7168, 160, 256 and
// 300 tokens 21, 21 and (160 tiles) 37 against 25, 23 and 25.
inline W4Form w4_form(const ExpertRows &r, int K, int F, int gated, int y_f32, int sms) {
    const int64_t active = r.pairs < r.E ? r.pairs : r.E, step = gated ? w4_tile::kM / 2 : w4_tile::kM;
    const int64_t tiles = (active + (r.pairs - active) / 64) * ((F + step - 1) / step);  // of 64 tokens, at most
    constexpr int kStage = w4_tile::kUnits * w4_tile::kK;
    const int stages = (K + kStage - 1) / kStage;
    const int split = tiles * 4 <= sms && stages >= 4 ? 4 : tiles * 2 <= sms && stages >= 2 ? 2 : 1;
    const int64_t granules = w4_few::most_granules(r, F, gated), share = (granules + sms - 1) / sms, rounds = (tiles + sms - 1) / sms;
    if (share * split <= 5 * rounds && K <= (1 << 15) && granules < (1 << 30) && w4_few::stages_of(r, K, w4_few::lines_of(r)) >= 2)
        return {w4_few::kTok, 1};
    if (split > 1 || r.pairs <= 48 * (int64_t)r.E || tiles <= sms) return {64, split};
    return {w4_parts(K, gated, y_f32) ? 128 : 160, 1};
}

}  // namespace moe
