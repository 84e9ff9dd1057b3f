// proj_launch.hpp -- host-side choice of tile shape and launch of the tile
// kernels, shared by the 4-bit and the gated entry points.
#pragma once

#include "proj_strip.hpp"
#include "proj_tile.hpp"
#include "sgmv_host.hpp"

#include <algorithm>

namespace sgmv {

using BigTile = TileShape<256, 256, 2, 4>;
using MidTile = TileShape<128, 128, 2, 2>;

inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Sets the tile grid of `a` for output width `width` (both matrices' columns
// for a gated call) and launches.
template <typename DT, typename SH, int AL, int BL, int kSegs, bool kGated, bool kDma, int kFlushes>
int launch_tiles(TileArgs a, hipStream_t st) {
    const long long tm = ceil_div(a.M, SH::BM);
    const long long tn = ceil_div(a.N, kGated ? SH::BN / 2 : SH::BN);
    const long long tiles = tm * tn * a.batches;
    if (tiles > 0x7FFFFFFFll) return SGMV_ERR_UNSUPPORTED;
    if (tiles == 0) return SGMV_OK;
    a.tiles_m = (int)tm;
    a.tiles_n = (int)tn;
    a.tiles = (int)tiles;
    launch(&tile_kernel<DT, SH, AL, BL, kSegs, kGated, kDma, kFlushes>, dim3((unsigned)tiles),
           dim3(SH::NT), st, a);
    return launch_status();
}

// Time of a tiled product per 4096 of K, in microseconds, as rounds of tiles over
// the 256 CUs: 106 us for one 256 x 256 tile per CU; 80 us for two 128 x 128
// tiles per CU (two workgroups share one), 52 us for one.  `big`, `mid`: tiles.
inline double big_tiles_us(long long big) { return 106. * ceil_div(big, 256); }
inline double mid_tiles_us(long long mid) { return mid <= 256 ? 52. : 80. * ceil_div(mid, 512); }

// The tile shape whose rounds take less time; the register path (operands no
// 16-byte load fits) always takes the small tiles.
template <typename DT, int AL, int BL, int kSegs, bool kGated, int kFlushes = 1>
int launch_tiles_any(const TileArgs& a, bool direct, hipStream_t st) {
    if (!direct) return launch_tiles<DT, MidTile, AL, BL, kSegs, kGated, false, kFlushes>(a, st);
    constexpr int per = kGated ? 2 : 1;
    const long long big = ceil_div(a.M, 256) * ceil_div((long long)a.N * per, 256) * a.batches;
    const long long mid = ceil_div(a.M, 128) * ceil_div((long long)a.N * per, 128) * a.batches;
    if (big_tiles_us(big) <= mid_tiles_us(mid))
        return launch_tiles<DT, BigTile, AL, BL, kSegs, kGated, true, kFlushes>(a, st);
    return launch_tiles<DT, MidTile, AL, BL, kSegs, kGated, true, kFlushes>(a, st);
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
