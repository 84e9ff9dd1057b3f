// proj_launch.hpp -- host-side choice of tile shape and launch of the tile
// kernels, shared by the 4-bit and the gated entry points.
#pragma once

#include "proj_strip.hpp"
#include "proj_tile.hpp"
#include "sgmv_host.hpp"

#include <algorithm>

namespace sgmv {

using BigTile = TileShape<256, 256, 2, 4>;
using WideTile = TileShape<128, 256, 2, 4>;
using MidTile = TileShape<128, 128, 2, 2>;
// float32, whose products take eight times as long per byte: small tiles cost no
// more loads than there is time for, and leave fewer CUs without work.
using SmallTile = TileShape<64, 64, 2, 2>;
using TallTile = TileShape<128, 64, 2, 2>;

inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Rows and columns (of each matrix) of the output, in elements.
struct TileRange {
    long long m_first, m_end, n_first, n_end;
};

template <typename DT, typename SH, int AL, int BL, int kSegs, bool kGated, bool kDma, int kFlushes>
int launch_tiles(TileArgs a, TileRange r, hipStream_t st) {
    const long long tm = ceil_div(r.m_end - r.m_first, SH::BM);
    const long long tn = ceil_div(r.n_end - r.n_first, kGated ? SH::BN / 2 : SH::BN);
    const long long tiles = tm * tn * a.batches;
    if (tiles > 0x7FFFFFFFll) return SGMV_ERR_UNSUPPORTED;
    if (tiles == 0) return SGMV_OK;
    a.m_first = (int)r.m_first;
    a.n_first = (int)r.n_first;
    a.tiles_m = (int)tm;
    a.tiles_n = (int)tn;
    a.tiles = (int)tiles;
    launch(&tile_kernel<DT, SH, AL, BL, kSegs, kGated, kDma, kFlushes>, dim3((unsigned)tiles),
           dim3(SH::NT), st, a);
    return launch_status();
}

// Time of `tiles` tiles per 4096 of K, in microseconds, as rounds over the 256
// CUs (bf16, measured on whole rounds of products along K and across K): a round
// of 256 x 256 tiles takes 109 to 122, one of 128 x 256 tiles 62 to 79, two
// 128 x 128 tiles on each CU 67 to 83 and one on each 42 to 52.
enum TileKind { kBigTiles, kWideTiles, kMidTiles, kSmallTiles, kTallTiles };
constexpr double kBigTileUs = 118.;
constexpr double kBigGatedCodesUs = 150.;  // gated 4-bit tiles: their registers spill

inline double tiles_us(TileKind kind, long long tiles, double big_us = kBigTileUs) {
    if (kind == kBigTiles) return big_us * ceil_div(tiles, 256);
    if (kind == kWideTiles) return 64. * ceil_div(tiles, 256);
    const long long rest = tiles % 512;
    return 78. * (tiles / 512) + (rest == 0 ? 0. : rest <= 256 ? 45. : 78.);
}

// A plan: the kind of tile for the whole output, or 256 x 256 tiles for the first
// rows or columns, as many as fill whole rounds, and `kind` for the rest.
struct TilePlan {
    TileKind kind;
    TileRange big, rest;  // big: empty unless split
    double us;
};

// 128 x 256 tiles: 2048 rows x 4096 from 2 x 11008, f16, 365 us, without them 470.
// 4-bit weights have none: unpacking them for 128 rows costs what
// the larger tile saves (512 x 5120 -> 13824: 104 us against 99 by 128 x 128 tiles).
inline TilePlan plan_tiles(long long M, long long N, int batches, bool gated, bool codes) {
    const double big_us = gated && codes ? kBigGatedCodesUs : kBigTileUs;
    const long long bn = gated ? 128 : 256;  // columns per 256 of a tile
    auto count = [&](TileKind kind, const TileRange& r) {
        return ceil_div(r.m_end - r.m_first, kind == kBigTiles ? 256 : 128) *
               ceil_div(r.n_end - r.n_first, kind == kMidTiles ? bn / 2 : bn) * batches;
    };
    const TileRange all{0, M, 0, N}, none{0, 0, 0, 0};
    TilePlan best{kBigTiles, none, all, tiles_us(kBigTiles, count(kBigTiles, all), big_us)};
    auto offer = [&](TileKind kind, const TileRange& big, const TileRange& rest, double us) {
        if (codes && kind == kWideTiles) return;
        us += tiles_us(kind, count(kind, rest));
        if (us < best.us) best = TilePlan{kind, big, rest, us};
    };
    offer(kWideTiles, none, all, 0.);
    offer(kMidTiles, none, all, 0.);
    // 4096 x 4096 -> 2 x 11008 is 1376 tiles, 5.4 rounds: 690 us as six rounds,
    // 676 as five and one of 128 x 256 tiles; its weights' gradients 625 and 606.
    // The second launch is priced at 4 us.
    const long long tm = ceil_div(M, 256), tn = ceil_div(N, bn);
    const long long rounds = tm * tn * batches / 256;
    if (rounds > 0) {
        const long long rows = 256 * rounds / (tn * batches), cols = 256 * rounds / (tm * batches);
        for (int by_rows = 0; by_rows < 2; ++by_rows) {
            TileRange big = all, rest = all;
            if (by_rows) big.m_end = rest.m_first = std::min(rows * 256, M);
            else big.n_end = rest.n_first = std::min(cols * bn, N);
            if (big.m_end == 0 || big.n_end == 0 || rest.m_first == M || rest.n_first == N) continue;
            const double us = 4. + tiles_us(kBigTiles, count(kBigTiles, big), big_us);
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

// The register path (operands no 16-byte load fits) always takes the small tiles.
template <typename DT, int AL, int BL, int kSegs, bool kGated, int kFlushes = 1>
int launch_kind(TileKind kind, const TileArgs& a, const TileRange& r, bool direct, hipStream_t st) {
    if constexpr (DT::kBytes == 4) {
        if (!direct) return launch_tiles<DT, SmallTile, AL, BL, kSegs, kGated, false, kFlushes>(a, r, st);
        if (kind == kTallTiles)
            return launch_tiles<DT, TallTile, AL, BL, kSegs, kGated, true, kFlushes>(a, r, st);
        return launch_tiles<DT, SmallTile, AL, BL, kSegs, kGated, true, kFlushes>(a, r, st);
    } else {
        if (!direct) return launch_tiles<DT, MidTile, AL, BL, kSegs, kGated, false, kFlushes>(a, r, st);
        if (kind == kBigTiles)
            return launch_tiles<DT, BigTile, AL, BL, kSegs, kGated, true, kFlushes>(a, r, st);
        if constexpr (BL != kCodes) {
            if (kind == kWideTiles)
                return launch_tiles<DT, WideTile, AL, BL, kSegs, kGated, true, kFlushes>(a, r, st);
        }
        return launch_tiles<DT, MidTile, AL, BL, kSegs, kGated, true, kFlushes>(a, r, st);
    }
}

// Plans and launches a whole product.
template <typename DT, int AL, int BL, int kSegs, bool kGated, int kFlushes = 1>
int launch_tiles_any(const TileArgs& a, bool direct, hipStream_t st) {
    const TileRange all{0, a.M, 0, a.N};
    if (!direct) return launch_kind<DT, AL, BL, kSegs, kGated, kFlushes>(kMidTiles, a, all, false, st);
    if constexpr (DT::kBytes == 4) {
        return launch_kind<DT, AL, BL, kSegs, kGated>(f32_kind(a.M, a.N, a.batches, kGated), a, all,
                                                      true, st);
    } else {
        const TilePlan p = plan_tiles(a.M, a.N, a.batches, kGated, BL == kCodes);
        if (p.big.m_end > 0) {
            const int rc = launch_kind<DT, AL, BL, kSegs, kGated, kFlushes>(kBigTiles, a, p.big, true, st);
            if (rc != SGMV_OK) return rc;
        }
        return launch_kind<DT, AL, BL, kSegs, kGated, kFlushes>(p.kind, a, p.rest, true, st);
    }
}

// How the sum of two products over K is taken: by one workgroup per tile, or
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

inline SumPlan plan_sum(long long M, long long N, long long K, int dtype) {
    const bool f32 = dtype == SGMV_F32;
    const long long steps = ceil_div(2 * ceil_div(K, f32 ? 16 : 32), 4) * 4;
    // Microseconds per step of 32 (float32: 16) K; 128 of 32 are 4096.
    auto step_us = [&](TileKind kind, int ranges) {
        if (f32) return f32_step_us(kind, f32_tiles(kind, M, N, false) * ranges);
        return tiles_us(kind, ceil_div(M, 128) * ceil_div(N, kind == kMidTiles ? 128 : 256) * ranges) / 128.;
    };
    const long long stride = ceil_div(M * N, 64) * 64;
    SumPlan best{f32 ? f32_kind(M, N, 1, false) : kBigTiles, 1, (int)steps, stride};
    double best_us = steps * (f32 ? step_us(best.kind, 1) : plan_tiles(M, N, 1, false, false).us / 128.);
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

template <typename DT, typename Src, int MT, int NTW, int KG, int NG, int S, int FL, bool kGated>
int launch_strip(const RowsArgs& a, hipStream_t st) {
    const long long gx = ceil_div(a.N, 16 * NTW * NG), gy = ceil_div(a.R, 16 * MT);
    if (gy > 65535) return SGMV_ERR_UNSUPPORTED;
    launch(&strip_kernel<DT, Src, MT, NTW, KG, NG, S, FL, kGated>, dim3((unsigned)gx, (unsigned)gy),
           dim3(kRowsThreads), st, a);
    return launch_status();
}

// The largest block of rows and features that still gives about two of three
// CUs a workgroup.  Larger blocks read x and unpack weights less often; below
// that many workgroups the idle CUs cost more (5120 -> 13824, 4-bit, bf16, 64
// rows: 24.5 us on 216 workgroups of 64 x 64, 32.9 us on 108 of 64 x 128; 128
// rows: 34.7 us on 216 of 64 x 128, 43.7 us on 864 of 32 x 64).  Blocks of 64
// rows are not taken where 32-row blocks would leave out a twelfth of the rows
// (gated, 333 rows x 4096 -> 11008: 126 us against 140), nor with a scale per 32
// K, whose flushes then need more registers than there are (333 x 2048 -> 5632:
// 41.5 us against 71).
template <typename DT, typename Src, int FL, bool kGated>
int run_strip(const RowsArgs& a, hipStream_t st) {
    // A gated wave holds both matrices' n-tiles: half as many features each.
    constexpr int T = kGated ? 1 : 2;
    auto fills = [&](int rows, int features) {
        return ceil_div(a.R, rows) * ceil_div(a.N, features) >= 170;
    };
    if constexpr (FL > 1) {
        const long long by64 = ceil_div(a.R, 64) * 64, by32 = ceil_div(a.R, 32) * 32;
        if (a.R > 32 && by64 * 11 <= by32 * 12) {
            if (fills(64, 128 * T)) return launch_strip<DT, Src, 4, T, 1, 8, 2, FL, kGated>(a, st);
            if (fills(64, 64 * T)) return launch_strip<DT, Src, 4, T, 2, 4, 2, FL, kGated>(a, st);
            if (!kGated && fills(64, 64)) return launch_strip<DT, Src, 4, T, 4, 2, 2, FL, kGated>(a, st);
        }
    }
    if (a.R > 16) {
        if (fills(32, 64 * T)) return launch_strip<DT, Src, 2, T, 2, 4, 2, FL, kGated>(a, st);
        if (!kGated && fills(32, 64)) return launch_strip<DT, Src, 2, T, 4, 2, 2, FL, kGated>(a, st);
        if (fills(32, 32)) return launch_strip<DT, Src, 2, 1, 4, 2, 2, FL, kGated>(a, st);
    }
    if (fills(16, 64))
        return kGated ? launch_strip<DT, Src, 1, 1, 2, 4, 2, FL, kGated>(a, st)
                      : launch_strip<DT, Src, 1, 2, 4, 2, 2, FL, kGated>(a, st);
    if (fills(16, 32)) return launch_strip<DT, Src, 1, 1, 4, 2, 2, FL, kGated>(a, st);
    return launch_strip<DT, Src, 1, 1, 8, 1, 3, FL, kGated>(a, st);
}

inline int elem_size(int dtype) { return dtype == SGMV_F32 ? 4 : 2; }
inline int piece_elems(int dtype) { return dtype == SGMV_F32 ? 4 : 8; }
inline bool known_dtype(int dtype) {
    return dtype == SGMV_F32 || dtype == SGMV_F16 || dtype == SGMV_BF16;
}
inline bool known_act(int act) { return act >= SGMV_ACT_SILU && act <= SGMV_ACT_SIGMOID; }

}  // namespace sgmv
