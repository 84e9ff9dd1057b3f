// q4_run.hpp -- kernel choice of the 4-bit projections.  run_q4 is instantiated
// for each element type in a source file of its own (q4_f32.hip, q4_f16.hip,
// q4_bf16.hip), which compile side by side.
#pragma once

#include "proj_launch.hpp"
#include "proj_strip.hpp"

namespace sgmv {

// Whether a 16-bit call of R rows takes tiles (scaled weights, each rounded
// once) instead of strips (exact codes, scales on float32 sums): by the times
// they take per 4096 of K.  Strips run at a steady rate, 240 us for 4096 x 4096
// outputs (350 with a scale per 32 K); for tiles see above, gated 256 x 256 tiles
// taking 150 us a round.  Measured, 4096 x 4096 weights, bf16: 1024 rows 48 us by
// strips, 52 by tiles; 1531 rows 78 and 72; 5120 -> 13824: 512 rows 134 and 96,
// 2048 rows 506 and 288.  Calls of up to kQ4ExactRows rows never round.
constexpr int kQ4ExactRows = 256;

inline bool q4_takes_tiles(int R, int N, int flushes, bool gated) {
    const int per = gated ? 2 : 1;  // matrices
    const double outputs = (double)ceil_div(R, 32) * 32 * N * per / (4096. * 4096.);
    const double us = plan_tiles(R, N, 1, gated, true).us;
    return us < outputs * (flushes == 4 ? 350. : 240.);
}

// FL: 4, 2 or 1 steps of 32 K per scale (1, 2 or 4 flushes per tile of 128 K).
template <typename DT, int XR, int MT, int PD, int FL, bool kGated>
int launch_q4_rows(const RowsArgs& a, hipStream_t st) {
    const long long gx = ceil_div(a.N, 16), gy = ceil_div(a.R, 16 * MT);
    if (gy > 65535) return SGMV_ERR_UNSUPPORTED;
    launch(&rows_kernel<DT, Q4Src<DT>, XR, MT, 1, PD, FL, kGated>, dim3((unsigned)gx, (unsigned)gy),
           dim3(kRowsThreads), st, a);
    return launch_status();
}

template <typename DT, int FL, bool kGated>
int run_q4_rows(const RowsArgs& a, hipStream_t st) {
    if constexpr (DT::kBytes == 2) {
        if (a.xvec) {
            // x loads for at most four rows; as many workgroups as n-tiles, so a
            // single matrix takes it only while these do not fill the chip several
            // times over (one row, 5120 -> 13824: 12.6 us against 11.2 by strips;
            // 4096 -> 11008: 7.8 against 8.5; gated 12.8 against 13.6).
            if (a.R <= 4 && (kGated || ceil_div(a.N, 16) < 768))
                return launch_q4_rows<DT, 4, 1, kGated ? 1 : FL == 1 ? 3 : 4, FL, kGated>(a, st);
            return run_strip<DT, Q4Src<DT>, FL, kGated>(a, st);
        }
        return a.R <= 16 ? launch_q4_rows<DT, 16, 1, 2, FL, kGated>(a, st)
                         : launch_q4_rows<DT, 16, 2, 1, FL, kGated>(a, st);
    } else {
        return a.R <= 16 ? launch_q4_rows<DT, 16, 1, 1, FL, kGated>(a, st)
                         : launch_q4_rows<DT, 16, 2, 1, FL, kGated>(a, st);
    }
}

template <typename DT, bool kGated>
int run_q4(const RowsArgs& a, int flushes, hipStream_t st) {
    if constexpr (DT::kBytes == 2) {
        if (a.R > kQ4ExactRows && (!a.xvec || q4_takes_tiles(a.R, a.N, flushes, kGated))) {
            TileArgs t{};
            t.a[0] = a.x;
            t.lda = a.K;
            t.out[0] = a.y;
            bool yvec = a.N % 4 == 0 && aligned16(a.y);
            for (int q = 0; q < 2; ++q) {
                t.q[q] = a.m[q];
                t.add[q] = a.add[q];
                yvec = yvec && aligned16(a.add[q]);
            }
            t.M = a.R;
            t.N = a.N;
            t.K = a.K;
            t.batches = 1;
            t.avec = a.xvec;
            t.yvec = yvec;
            t.kblocks = a.kblocks;
            t.act = a.act;
            const bool direct = a.xvec != 0;
            if (flushes == 1) return launch_tiles_any<DT, kAlongK, kCodes, 1, kGated, 1>(t, direct, st);
            if (flushes == 2) return launch_tiles_any<DT, kAlongK, kCodes, 1, kGated, 2>(t, direct, st);
            return launch_tiles_any<DT, kAlongK, kCodes, 1, kGated, 4>(t, direct, st);
        }
    }
    if (flushes == 1) return run_q4_rows<DT, 4, kGated>(a, st);
    if (flushes == 2) return run_q4_rows<DT, 2, kGated>(a, st);
    return run_q4_rows<DT, 1, kGated>(a, st);
}


extern template int run_q4<F32, false>(const RowsArgs&, int, hipStream_t);
extern template int run_q4<F32, true>(const RowsArgs&, int, hipStream_t);
extern template int run_q4<F16, false>(const RowsArgs&, int, hipStream_t);
extern template int run_q4<F16, true>(const RowsArgs&, int, hipStream_t);
extern template int run_q4<BF16, false>(const RowsArgs&, int, hipStream_t);
extern template int run_q4<BF16, true>(const RowsArgs&, int, hipStream_t);

}  // namespace sgmv
