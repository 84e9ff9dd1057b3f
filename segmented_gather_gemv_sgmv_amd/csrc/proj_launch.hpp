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

// 256 x 256 tiles once they make a tile per CU, 128 x 128 below that; the
// register path (operands no 16-byte load fits) always takes the small ones.
template <typename DT, int AL, int BL, int kSegs, bool kGated, int kFlushes = 1>
int launch_tiles_any(const TileArgs& a, bool direct, hipStream_t st) {
    if (!direct) return launch_tiles<DT, MidTile, AL, BL, kSegs, kGated, false, kFlushes>(a, st);
    const long long big = ceil_div(a.M, 256) * ceil_div(a.N, kGated ? 128 : 256) * a.batches;
    if (big >= 192) return launch_tiles<DT, BigTile, AL, BL, kSegs, kGated, true, kFlushes>(a, st);
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

// The largest block of rows and features that still gives about three of four
// CUs a workgroup.  Larger blocks read x and unpack weights less often; below
// that many workgroups the idle CUs cost more (5120 -> 13824, 4-bit, bf16, 64
// rows: 24.5 us on 432 workgroups of 32 x 64, 32.9 us on 108 of 64 x 128; 128
// rows: 43.7 and 34.7 us).  S = 3 stages where a block's products are too few
// to cover one x load (16 rows: 13.2 -> 12.2 us), two otherwise.
template <typename DT, typename Src, int FL, bool kGated>
int run_strip(const RowsArgs& a, hipStream_t st) {
    // A gated wave holds both matrices' n-tiles: half as many features each.
    constexpr int T = kGated ? 1 : 2;
    auto fills = [&](int rows, int features) {
        return ceil_div(a.R, rows) * ceil_div(a.N, features) >= 190;
    };
    if (a.R > 32) {
        if (fills(64, 128 * T)) return launch_strip<DT, Src, 4, T, 1, 8, 2, FL, kGated>(a, st);
        if (fills(64, 64 * T)) return launch_strip<DT, Src, 4, T, 2, 4, 2, FL, kGated>(a, st);
    }
    if (a.R > 16) {
        if (!kGated && fills(32, 64)) return launch_strip<DT, Src, 2, T, 4, 2, 2, FL, kGated>(a, st);
        if (fills(32, 32)) return launch_strip<DT, Src, 2, 1, 4, 2, 2, FL, kGated>(a, st);
    }
    if (!kGated && fills(16, 64)) return launch_strip<DT, Src, 1, T, 4, 2, 3, FL, kGated>(a, st);
    if (fills(16, 32)) return launch_strip<DT, Src, 1, 1, 4, 2, 3, FL, kGated>(a, st);
    return launch_strip<DT, Src, 1, 1, 8, 1, 3, FL, kGated>(a, st);
}

inline int elem_size(int dtype) { return dtype == SGMV_F32 ? 4 : 2; }
inline int piece_elems(int dtype) { return dtype == SGMV_F32 ? 4 : 8; }
inline bool known_dtype(int dtype) {
    return dtype == SGMV_F32 || dtype == SGMV_F16 || dtype == SGMV_BF16;
}
inline bool known_act(int act) { return act >= SGMV_ACT_SILU && act <= SGMV_ACT_SIGMOID; }

}  // namespace sgmv
