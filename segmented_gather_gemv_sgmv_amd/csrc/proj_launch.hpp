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
enum TileKind { kBigTiles, kWideTiles, kMidTiles };
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

// 4-bit weights have no 128 x 256 tiles: unpacking them for 128 rows costs what
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
    // 4096 x 4096 -> 2 x 11008 is 1376 tiles, 5.4 rounds: 728 us as six rounds,
    // 717 as five and one of 128 x 256 tiles; its weights' gradients 650 and 631.
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

// The register path (operands no 16-byte load fits) always takes the small tiles.
template <typename DT, int AL, int BL, int kSegs, bool kGated, int kFlushes = 1>
int launch_kind(TileKind kind, const TileArgs& a, const TileRange& r, bool direct, hipStream_t st) {
    if (!direct) return launch_tiles<DT, MidTile, AL, BL, kSegs, kGated, false, kFlushes>(a, r, st);
    if (kind == kBigTiles)
        return launch_tiles<DT, BigTile, AL, BL, kSegs, kGated, true, kFlushes>(a, r, st);
    if constexpr (BL != kCodes) {
        if (kind == kWideTiles)
            return launch_tiles<DT, WideTile, AL, BL, kSegs, kGated, true, kFlushes>(a, r, st);
    }
    return launch_tiles<DT, MidTile, AL, BL, kSegs, kGated, true, kFlushes>(a, r, st);
}

// Plans and launches a whole product.
template <typename DT, int AL, int BL, int kSegs, bool kGated, int kFlushes = 1>
int launch_tiles_any(const TileArgs& a, bool direct, hipStream_t st) {
    const TileRange all{0, a.M, 0, a.N};
    if (!direct) return launch_kind<DT, AL, BL, kSegs, kGated, kFlushes>(kMidTiles, a, all, false, st);
    const TilePlan p = plan_tiles(a.M, a.N, a.batches, kGated, BL == kCodes);
    if (p.big.m_end > 0) {
        const int rc = launch_kind<DT, AL, BL, kSegs, kGated, kFlushes>(kBigTiles, a, p.big, true, st);
        if (rc != SGMV_OK) return rc;
    }
    return launch_kind<DT, AL, BL, kSegs, kGated, kFlushes>(p.kind, a, p.rest, true, st);
}

// How the sum of two products over K is taken: by one workgroup per tile, or
// (ranges > 1) in ranges of K, each by a workgroup of its own that leaves its
// float32 sums, joined by a second kernel.  Outputs of a few tiles are worth it:
// their long K would run on a few CUs (1237 rows x 1000 from 2 x 2744, f16:
// 64 us in one range, 32 in three; 512 x 2048 from 2 x 5504: bf16 105 and 38 in
// eight, f32 723 and 198 in eight).
struct SumPlan {
    TileKind kind;
    int ranges, range_steps;
    long long stride;  // floats per range's sums
};

constexpr long long kMaxSumBytes = 64ll << 20;

inline SumPlan plan_sum(long long M, long long N, long long K, int dtype) {
    const bool f32 = dtype == SGMV_F32;
    const long long steps = ceil_div(2 * ceil_div(K, f32 ? 16 : 32), 4) * 4;
    // Microseconds per step: 128 steps of 32 K are 4096; float32 steps (of 16 K)
    // multiply three terms on each side.
    const double per = (f32 ? 4. : 1.) / 128.;
    const long long stride = ceil_div(M * N, 64) * 64;
    SumPlan best{kBigTiles, 1, (int)steps, stride};
    double best_us = plan_tiles(M, N, 1, false, false).us * steps * per;
    if (stride > kMaxSumBytes / 8) return best;
    const long long wide = ceil_div(M, 128) * ceil_div(N, 256);
    const long long mid = ceil_div(M, 128) * ceil_div(N, 128);
    for (int ranges = 2; ranges <= 64; ++ranges) {
        const long long each = ceil_div(steps, 4ll * ranges) * 4;
        if (each < 16 || ranges * stride * 4 > kMaxSumBytes) break;
        if (ceil_div(steps, each) != ranges) continue;
        const double join = 5. + ranges * stride * 8 / 4e6;  // written and read at 4 TB/s
        for (const TileKind kind : {kWideTiles, kMidTiles}) {
            const double us = join + each * per * tiles_us(kind, ranges * (kind == kWideTiles ? wide : mid));
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
