// proj_plan.hpp -- which kernel a call of the projections or of rope takes: rules on
// its sizes alone, each with what both sides measured.  Host code without HIP, so
// that tests can ask which kernels a shape reaches.
#pragma once

#include <algorithm>

#include "sgmv.h"

namespace sgmv {

inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

inline int elem_size(int dtype) { return dtype == SGMV_F32 ? 4 : 2; }
inline int piece_elems(int dtype) { return dtype == SGMV_F32 ? 4 : 8; }
inline bool known_dtype(int dtype) {
    return dtype == SGMV_F32 || dtype == SGMV_F16 || dtype == SGMV_BF16;
}

// Rows and columns (of each matrix) of the output, in elements.
struct TileRange {
    long long m_first, m_end, n_first, n_end;
};

// ---- tiles of many rows ------------------------------------------------------
// Tiles of rows x features: big 256 x 256, wide 128 x 256, mid 128 x 128; of float32
// small 64 x 64 and tall 128 x 64; of 4-bit weights deep 256 x 128 and mid.
enum TileKind { kBigTiles, kWideTiles, kMidTiles, kSmallTiles, kTallTiles, kDeepTiles };

// Time of `tiles` tiles per 4096 of K, in microseconds, as rounds over the 256
// CUs (bf16, measured on whole rounds of products along K and across K): a round
// of 256 x 256 tiles takes 109 to 122, one of 128 x 256 tiles 62 to 79, two
// 128 x 128 tiles on each CU 67 to 83 and one on each 42 to 52.
inline double tiles_us(TileKind kind, long long tiles) {
    if (kind == kBigTiles) return 118. * ceil_div(tiles, 256);
    if (kind == kWideTiles) return 64. * ceil_div(tiles, 256);
    const long long rest = tiles % 512;
    return 78. * (tiles / 512) + (rest == 0 ? 0. : rest <= 256 ? 45. : 78.);
}

// The same of 4-bit weights' tiles, with 1, 2 or 4 scales per 128 K: a round of 256 x 128
// tiles 74 to 79, 82 to 86, 96 to 107; two 128 x 128 tiles on each CU 72 to 90, 84 to 97,
// 96 to 120, one on each 55 to 66, 65 to 73, 82 to 89.
inline double code_tiles_us(TileKind kind, long long tiles, int flushes) {
    if (kind == kDeepTiles)
        return (flushes == 4 ? 100. : flushes == 2 ? 84. : 76.) * ceil_div(tiles, 256);
    const double one = flushes == 4 ? 86. : flushes == 2 ? 68. : 61.;
    const double two = flushes == 4 ? 107. : flushes == 2 ? 90. : 82.;
    const long long rest = tiles % 512;
    return two * (tiles / 512) + (rest == 0 ? 0. : rest <= 256 ? one : two);
}

// A plan: the kind of tile for the whole output, or the largest tiles for the first rows
// or columns, as many as fill whole rounds, and `kind` for the rest.
struct TilePlan {
    TileKind kind, big_kind;
    TileRange big, rest;  // big: empty unless split
    double us;
};

// code_flushes: scales per 128 K of 4-bit weights, 0 of plain ones.
// 128 x 256 tiles: 2048 rows x 4096 from 2 x 11008, f16, 365 us, without them 470.
// 256 x 128 tiles of 4-bit weights: 1531 x 4096 -> 4096, bf16, 79 us, without them 91;
// 512 x 5120 -> 13824, 88 and 102.
inline TilePlan plan_tiles(long long M, long long N, int batches, bool gated, int code_flushes = 0) {
    const bool codes = code_flushes > 0;
    const TileKind large = codes ? kDeepTiles : kBigTiles;
    auto columns = [&](TileKind kind) {  // of each matrix
        return (kind == kBigTiles || kind == kWideTiles ? 256ll : 128ll) / (gated ? 2 : 1);
    };
    auto time = [&](TileKind kind, const TileRange& r) {
        const long long n = ceil_div(r.m_end - r.m_first, kind == large ? 256 : 128) *
                            ceil_div(r.n_end - r.n_first, columns(kind)) * batches;
        return codes ? code_tiles_us(kind, n, code_flushes) : tiles_us(kind, n);
    };
    const TileRange all{0, M, 0, N}, none{0, 0, 0, 0};
    TilePlan best{large, large, none, all, time(large, all)};
    auto offer = [&](TileKind kind, const TileRange& big, const TileRange& rest, double us) {
        if (codes && kind == kWideTiles) return;
        us += time(kind, rest);
        if (us < best.us) best = TilePlan{kind, large, big, rest, us};
    };
    offer(kWideTiles, none, all, 0.);
    offer(kMidTiles, none, all, 0.);
    // 4096 x 4096 -> 2 x 11008 is 1376 tiles, 5.4 rounds: 690 us as six rounds,
    // 676 as five and one of 128 x 256 tiles; its weights' gradients 625 and 606.
    // The second launch is priced at 4 us.
    const long long bn = columns(large), tm = ceil_div(M, 256), tn = ceil_div(N, bn);
    const long long rounds = tm * tn * batches / 256;
    if (rounds > 0) {
        const long long rows = 256 * rounds / (tn * batches), cols = 256 * rounds / (tm * batches);
        for (int by_rows = 0; by_rows < 2; ++by_rows) {
            TileRange big = all, rest = all;
            if (by_rows) big.m_end = rest.m_first = std::min(rows * 256, M);
            else big.n_end = rest.n_first = std::min(cols * bn, N);
            if (big.m_end == 0 || big.n_end == 0 || rest.m_first == M || rest.n_first == N) continue;
            const double us = 4. + time(large, big);
            offer(kWideTiles, big, rest, us);
            offer(kMidTiles, big, rest, us);
        }
    }
    return best;
}

// float32: the time of a step of 16 K, in microseconds, for the tiles a CU gets at
// most; several share it, so a round more costs little more than its products.
// Forward, 512 rows x 4096 -> 2 x 11008: 743 us by 128 x 64 tiles, 801 by 64 x 64;
// 333 x 2048 -> 2 x 5504: 198 and 182; 200 x 3968 -> 2 x 1504: 142 and 82 (by 128 x
// 128 tiles 800, 261 and 268).
inline double f32_step_us(TileKind kind, long long tiles) {
    const double each = (double)ceil_div(tiles, 256);
    if (kind == kTallTiles) return 0.1 + 0.475 * each;
    return each <= 1. ? 0.32 : 0.285 * each - 0.05;
}
inline long long f32_tiles(TileKind kind, long long M, long long N, bool gated) {
    return ceil_div(M, kind == kTallTiles ? 128 : 64) * ceil_div(N, gated ? 32 : 64);
}
inline TileKind f32_kind(long long M, long long N, int batches, bool gated) {
    const double tall = f32_step_us(kTallTiles, f32_tiles(kTallTiles, M, N, gated) * batches);
    const double small = f32_step_us(kSmallTiles, f32_tiles(kSmallTiles, M, N, gated) * batches);
    return tall < small ? kTallTiles : kSmallTiles;
}

// How the sum of `segments` products over K each is taken: by one workgroup per tile, or
// (ranges > 1) in ranges of K, each by a workgroup of its own that leaves its
// float32 sums, joined by a second kernel.  Outputs of a few tiles are worth it:
// their long K would run on a few CUs (1237 rows x 1000 from 2 x 2744, f16:
// 64 us in one range, 32 in three; 512 x 2048 from 2 x 5504, bf16: 105 and 38 in
// eight).
struct SumPlan {
    TileKind kind;
    int ranges, range_steps;
    long long stride;  // floats per range's sums
};

constexpr long long kMaxSumBytes = 64ll << 20;

inline SumPlan plan_sum(long long M, long long N, long long K, int segments, int dtype) {
    const bool f32 = dtype == SGMV_F32;
    const long long steps = ceil_div(segments * ceil_div(K, f32 ? 16 : 32), 4) * 4;
    // Microseconds per step of 32 (float32: 16) K; 128 of 32 are 4096.
    auto step_us = [&](TileKind kind, int ranges) {
        if (f32) return f32_step_us(kind, f32_tiles(kind, M, N, false) * ranges);
        return tiles_us(kind, ceil_div(M, 128) * ceil_div(N, kind == kMidTiles ? 128 : 256) * ranges) / 128.;
    };
    const long long stride = ceil_div(M * N, 64) * 64;
    SumPlan best{f32 ? f32_kind(M, N, 1, false) : kBigTiles, 1, (int)steps, stride};
    double best_us = steps * (f32 ? step_us(best.kind, 1) : plan_tiles(M, N, 1, false).us / 128.);
    if (stride > kMaxSumBytes / 8) return best;
    for (int ranges = 2; ranges <= 64; ++ranges) {
        const long long each = ceil_div(steps, 4ll * ranges) * 4;
        if (each < 16 || ranges * stride * 4 > kMaxSumBytes) break;
        if (ceil_div(steps, each) != ranges) continue;
        const double join = 5. + ranges * stride * 8 / 4e6;  // written and read at 4 TB/s
        for (const TileKind kind : {f32 ? kTallTiles : kWideTiles, f32 ? kSmallTiles : kMidTiles}) {
            const double us = join + each * step_us(kind, ranges);
            if (us < best_us) {
                best_us = us;
                best = SumPlan{kind, ranges, (int)each, stride};
            }
        }
    }
    return best;
}

// ---- 4-bit projections -------------------------------------------------------
// The largest block of rows and features that still gives about two of three
// CUs a workgroup.  Larger blocks read x and unpack weights less often; below
// that many workgroups the idle CUs cost more (5120 -> 13824, 4-bit, bf16, 64
// rows: 24.5 us on 216 workgroups of 64 x 64, 32.9 us on 108 of 64 x 128; 128
// rows: 34.7 us on 216 of 64 x 128, 43.7 us on 864 of 32 x 64).  Blocks of 64
// rows are not taken where 32-row blocks would leave out a twelfth of the rows
// (gated, 333 rows x 4096 -> 11008: 126 us against 140), nor with a scale per 32
// K, whose flushes then need more registers than there are (333 x 2048 -> 5632:
// 41.5 us against 71).
// A gated wave holds both matrices' n-tiles: half as many features each.
enum StripBlock { kStrip64xMost, kStrip64xHalf, kStrip64x64, kStrip32xHalf, kStrip32x64, kStrip32x32,
                  kStrip16x64, kStrip16x32, kStrip16x16 };

inline StripBlock q4_strip_block(long long R, long long N, int flushes, bool gated) {
    const int T = gated ? 1 : 2;
    auto fills = [&](int rows, int features) {
        return ceil_div(R, rows) * ceil_div(N, features) >= 170;
    };
    if (flushes < 4) {
        const long long by64 = ceil_div(R, 64) * 64, by32 = ceil_div(R, 32) * 32;
        if (R > 32 && by64 * 11 <= by32 * 12) {
            if (fills(64, 128 * T)) return kStrip64xMost;
            if (fills(64, 64 * T)) return kStrip64xHalf;
            if (!gated && fills(64, 64)) return kStrip64x64;
        }
    }
    if (R > 16) {
        if (fills(32, 64 * T)) return kStrip32xHalf;
        if (!gated && fills(32, 64)) return kStrip32x64;
        if (fills(32, 32)) return kStrip32x32;
    }
    if (fills(16, 64)) return kStrip16x64;
    return fills(16, 32) ? kStrip16x32 : kStrip16x16;
}

// Whether a 16-bit call takes tiles instead of strips: by the times they take per 4096 of
// K, with 1, 2 or 4 scales per 128 K.  Both run in rounds of the 256 CUs: strips' blocks
// one to a CU, 53, 58 or 76 us for 64 rows x 256 features and less in proportion; tiles
// see above.  4096 features of 4096, bf16, by strips and 128 x 128 tiles: 1024 rows 52 and
// 65 us, 1531 rows 89 and 83, 2048 rows 98 and 90; 5120 -> 13824: 256 rows 67 and 79, 300
// rows 110 and 101, 512 rows 130 and 113; gated 333 x 2048 -> 5632: 54 and 48, with 32
// K per scale 41 and 61.
inline bool q4_takes_tiles(long long R, long long N, int flushes, bool gated) {
    const long long per = gated ? 2 : 1;  // matrices
    static const struct { int rows, features; } kBlocks[] = {
        {64, 256}, {64, 128}, {64, 64}, {32, 128}, {32, 64}, {32, 32}, {16, 64}, {16, 32}, {16, 16}};
    const StripBlock block = q4_strip_block(R, N, flushes, gated);
    const bool by_pairs = block == kStrip64xMost || block == kStrip64xHalf || block == kStrip32xHalf;
    const long long rows = kBlocks[block].rows;
    const long long features = kBlocks[block].features / (by_pairs ? per : 1);
    const double strip = (flushes == 4 ? 76. : flushes == 2 ? 58. : 53.) * (rows * features * per) / (64 * 256);
    return plan_tiles(R, N, 1, gated, flushes).us < strip * ceil_div(ceil_div(R, rows) * ceil_div(N, features), 256);
}

// Whether a 16-bit call of at most four rows takes the rows kernel instead of strips:
// its x loads suit so few rows, but it has a workgroup per 16 features and matrix, so
// for one matrix only while these do not fill the chip several times over.  bf16, rows
// kernel and strips: one row of 4096, 688 workgroups 6.8 and 8.0 us, 768 6.9 and 8.5,
// 864 8.4 and 8.3, 1024 8.9 and 8.5; four rows 768 7.6 and 8.4, 864 9.3 and 8.5; one row
// of 8192, 768 12.4 and 14.4, 864 15.8 and 14.9; of 1024 within 0.3 of each other up to
// 768.  Gated, one row of 4096, 688: 12.8 and 13.6.
inline bool q4_takes_rows(long long R, long long N, bool gated) {
    return R <= 4 && (gated || ceil_div(N, 16) <= 768);
}

// Whether a 16-bit call of x that no 16-byte load fits takes the tiles' register path
// instead of the rows kernel's workgroups of 32 rows x 16 features.  fp16, rows and
// tiles: 504 workgroups of 1001 K 23 and 54 us, 1008 42 and 54, 2048 of 4097 K 251 and
// 217.
inline bool q4_slow_takes_tiles(long long R, long long N) {
    return R > 16 && ceil_div(R, 32) * ceil_div(N, 16) > 1500;
}

// The kernel of a 4-bit call (bytes: of an element; vec: x takes 16-byte loads).
enum Q4Path { kQ4Rows4, kQ4Rows16, kQ4Rows32, kQ4Strips, kQ4Tiles };

inline Q4Path q4_path(long long R, long long N, int flushes, bool gated, int bytes, bool vec) {
    if (bytes == 4 || (!vec && !q4_slow_takes_tiles(R, N))) return R <= 16 ? kQ4Rows16 : kQ4Rows32;
    if (!vec) return kQ4Tiles;
    if (q4_takes_rows(R, N, gated)) return kQ4Rows4;
    return q4_takes_tiles(R, N, flushes, gated) ? kQ4Tiles : kQ4Strips;
}

// ---- gated block of plain weights --------------------------------------------
// Rows up to which a 16-bit forward streams the weights, by rows or strips.
constexpr int kFfnRowsMax = 64;

// float32: up to 32 rows, and more while the workgroups of 32 rows x 16 features are
// about one round; tiles then leave more CUs without work (64 rows x 3968 -> 2 x 1504:
// 40 us by rows, 77 by tiles; 64 x 1000 -> 2400: 22 and 25; beyond, 64 x 2048 ->
// 2 x 5504: 64 and 44).
inline bool ffn_f32_takes_rows(long long R, long long N) {
    return R <= 32 || ceil_div(R, 32) * ceil_div(N, 16) <= 320;
}

// More rows still take strips where their blocks of 64 rows x 32 features are at
// most one round: a tile's workgroup is then alone with the whole of K (bf16, 256
// rows x 4096 -> 2 x 1504: 30 us by strips, 45 by tiles; 192 x 1000 -> 2400: 12
// and 18; 512 x 1000 -> 800: 12 and 18).  Beyond a round tiles win (256 x 1000 ->
// 2400: 21 and 19; 128 x 4096 -> 11008: 96 and 66).
// Only operands that 16-byte loads fit.
inline bool ffn_takes_strips(long long R, long long N) {
    return ceil_div(R, 64) * ceil_div(N, 32) <= 256;
}

// Strips of 64 features while these give half of the CUs a workgroup, else of 32.
inline bool ffn_wide_strips(long long N) { return ceil_div(N, 64) >= 128; }

// The kernel of a forward call (vec: x and the weights take 16-byte loads).
enum FfnPath { kFfnRows4, kFfnRows16, kFfnRows32, kFfnStrips32, kFfnStrips64, kFfnTiles };

inline FfnPath ffn_path(long long R, long long N, int bytes, bool vec) {
    if (bytes == 4 ? !ffn_f32_takes_rows(R, N) : R > kFfnRowsMax && !(vec && ffn_takes_strips(R, N)))
        return kFfnTiles;
    if (R <= 4) return kFfnRows4;
    if (R <= 16) return kFfnRows16;
    // From 17 rows on x goes through LDS.
    if (bytes == 4 || !vec) return kFfnRows32;
    return R <= 32 ? kFfnStrips32 : kFfnStrips64;
}

// ---- rotary positions --------------------------------------------------------
constexpr int kRopeThreads = 256;
constexpr int kRopeMaxDim = 1024;   // of a head
constexpr int kRopeUnitsMost = 4;   // units per thread

// Units per head, heads per workgroup and workgroups per row; v elements a unit (16
// bytes, or one element where those do not fit).
struct RopeGrid {
    int units, heads_per_group, groups;
};

// One workgroup per row once the rows fill the chip (4 per CU); with fewer rows, and
// where a thread would hold more than kRopeUnitsMost units, the heads are split too,
// down to one pass of the workgroup.
inline RopeGrid rope_grid(long long rows, long long heads, int head_dim, int rotary_dim,
                          bool interleaved, int v) {
    RopeGrid g;
    g.units = (interleaved ? (v > 1 ? rotary_dim / v : rotary_dim / 2) : rotary_dim / 2 / v) +
              (head_dim - rotary_dim) / v;
    static_assert(kRopeMaxDim <= kRopeThreads * kRopeUnitsMost, "a head fits a workgroup");
    const long long per_pass = std::max(1, kRopeThreads / g.units);
    const long long want = (1024ll + rows - 1) / rows;
    long long hpg = std::max(per_pass, (heads + want - 1) / want);
    hpg = std::min({hpg, heads, (long long)(kRopeThreads * kRopeUnitsMost / g.units)});
    g.heads_per_group = (int)hpg;
    g.groups = (int)((heads + hpg - 1) / hpg);
    return g;
}

// Units a thread takes: 1, 2 or kRopeUnitsMost, what the kernel is built for.
inline int rope_units_per_thread(int heads_per_group, int units) {
    const long long each = ceil_div((long long)heads_per_group * units, kRopeThreads);
    return each <= 1 ? 1 : each <= 2 ? 2 : kRopeUnitsMost;
}

}  // namespace sgmv
