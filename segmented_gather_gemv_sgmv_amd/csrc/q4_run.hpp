// q4_run.hpp -- kernel choice of the 4-bit projections.  run_q4 is instantiated
// for each element type in a source file of its own (q4_f32.hip, q4_f16.hip,
// q4_bf16.hip), which compile side by side.
#pragma once

#include "proj_launch.hpp"
#include "proj_strip.hpp"

namespace sgmv {

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
int run_q4_few(const RowsArgs& a, Q4Path path, hipStream_t st) {
    constexpr bool k16 = DT::kBytes == 2;
    if constexpr (k16) {
        if (path == kQ4Rows4)
            return launch_q4_rows<DT, 4, 1, kGated ? 1 : FL == 1 ? 3 : 4, FL, kGated>(a, st);
        if (path == kQ4Strips) return run_strip<DT, Q4Src<DT>, FL, kGated>(a, st);
    }
    return path == kQ4Rows16 ? launch_q4_rows<DT, 16, 1, k16 ? 2 : 1, FL, kGated>(a, st)
                             : launch_q4_rows<DT, 16, 2, 1, FL, kGated>(a, st);
}

template <typename DT, bool kGated>
int run_q4(const RowsArgs& a, int flushes, hipStream_t st) {
    const Q4Path path = q4_path(a.R, a.N, flushes, kGated, DT::kBytes, a.xvec != 0);
    if constexpr (DT::kBytes == 2) {
        if (path == kQ4Tiles) {
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
    if (flushes == 1) return run_q4_few<DT, 4, kGated>(a, path, st);
    if (flushes == 2) return run_q4_few<DT, 2, kGated>(a, path, st);
    return run_q4_few<DT, 1, kGated>(a, path, st);
}

extern template int run_q4<F32, false>(const RowsArgs&, int, hipStream_t);
extern template int run_q4<F32, true>(const RowsArgs&, int, hipStream_t);
extern template int run_q4<F16, false>(const RowsArgs&, int, hipStream_t);
extern template int run_q4<F16, true>(const RowsArgs&, int, hipStream_t);
extern template int run_q4<BF16, false>(const RowsArgs&, int, hipStream_t);
extern template int run_q4<BF16, true>(const RowsArgs&, int, hipStream_t);

}  // namespace sgmv
