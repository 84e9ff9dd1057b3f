// proj_launch.hpp -- launches of the tile and strip kernels, by the choices of
// proj_plan.hpp, shared by the 4-bit and the gated entry points.
#pragma once

#include "proj_plan.hpp"
#include "proj_strip.hpp"
#include "proj_tile.hpp"
#include "sgmv_host.hpp"

namespace sgmv {

using BigTile = TileShape<256, 256, 2, 4>;
using WideTile = TileShape<128, 256, 2, 4>;
using MidTile = TileShape<128, 128, 2, 2>;
using DeepTile = TileShape<256, 128, 4, 2>;
// float32, whose products take eight times as long per byte: small tiles cost no
// more loads than there is time for, and leave fewer CUs without work.
using SmallTile = TileShape<64, 64, 2, 2>;
using TallTile = TileShape<128, 64, 2, 2>;

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
        if constexpr (BL == kCodes) {
            if (kind == kDeepTiles)
                return launch_tiles<DT, DeepTile, AL, BL, kSegs, kGated, true, kFlushes>(a, r, st);
        } else {
            if (kind == kBigTiles)
                return launch_tiles<DT, BigTile, AL, BL, kSegs, kGated, true, kFlushes>(a, r, st);
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
        const TilePlan p = plan_tiles(a.M, a.N, a.batches, kGated, BL == kCodes ? kFlushes : 0);
        if (p.big.m_end > 0) {
            const int rc = launch_kind<DT, AL, BL, kSegs, kGated, kFlushes>(p.big_kind, a, p.big, true, st);
            if (rc != SGMV_OK) return rc;
        }
        return launch_kind<DT, AL, BL, kSegs, kGated, kFlushes>(p.kind, a, p.rest, true, st);
    }
}

template <typename DT, typename Src, int MT, int NTW, int KG, int NG, int S, int FL, bool kGated>
int launch_strip(const RowsArgs& a, hipStream_t st) {
    const long long gx = ceil_div(a.N, 16 * NTW * NG), gy = ceil_div(a.R, 16 * MT);
    if (gy > 65535) return SGMV_ERR_UNSUPPORTED;
    launch(&strip_kernel<DT, Src, MT, NTW, KG, NG, S, FL, kGated>, dim3((unsigned)gx, (unsigned)gy),
           dim3(kRowsThreads), st, a);
    return launch_status();
}

template <typename DT, typename Src, int FL, bool kGated>
int run_strip(const RowsArgs& a, hipStream_t st) {
    constexpr int T = kGated ? 1 : 2;
    switch (q4_strip_block(a.R, a.N, 4 / FL, kGated)) {
        case kStrip64xMost:
            if constexpr (FL > 1) return launch_strip<DT, Src, 4, T, 1, 8, 2, FL, kGated>(a, st);
            break;
        case kStrip64xHalf:
            if constexpr (FL > 1) return launch_strip<DT, Src, 4, T, 2, 4, 2, FL, kGated>(a, st);
            break;
        case kStrip64x64:
            if constexpr (FL > 1 && !kGated)
                return launch_strip<DT, Src, 4, T, 4, 2, 2, FL, kGated>(a, st);
            break;
        case kStrip32xHalf: return launch_strip<DT, Src, 2, T, 2, 4, 2, FL, kGated>(a, st);
        case kStrip32x64:
            if constexpr (!kGated) return launch_strip<DT, Src, 2, T, 4, 2, 2, FL, kGated>(a, st);
            break;
        case kStrip32x32: return launch_strip<DT, Src, 2, 1, 4, 2, 2, FL, kGated>(a, st);
        case kStrip16x64:
            return kGated ? launch_strip<DT, Src, 1, 1, 2, 4, 2, FL, kGated>(a, st)
                          : launch_strip<DT, Src, 1, 2, 4, 2, 2, FL, kGated>(a, st);
        case kStrip16x32: return launch_strip<DT, Src, 1, 1, 4, 2, 2, FL, kGated>(a, st);
        case kStrip16x16: return launch_strip<DT, Src, 1, 1, 8, 1, 3, FL, kGated>(a, st);
    }
    return SGMV_ERR_UNSUPPORTED;  // the choice above names no block that is not here
}

inline bool known_act(int act) { return act >= SGMV_ACT_SILU && act <= SGMV_ACT_SIGMOID; }

}  // namespace sgmv
