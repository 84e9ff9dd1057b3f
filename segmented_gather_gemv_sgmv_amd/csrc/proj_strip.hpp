// proj_strip.hpp -- base projections of a few dozen rows, x through LDS.
//
// The rows kernel reads x straight into operand registers: 64-byte pieces of
// 16 rows per load, by every wave.  From about eight rows on those reads, not
// the weights, are what it waits for.  Here a workgroup's eight waves are KG
// groups along K times NG along the output features; a group's x block (16 MT
// rows by 128 K, 256 bytes of a row at a time) is brought by direct
// global-to-LDS loads, S - 1 blocks ahead, and shared by the group's NG waves,
// each with NTW n-tiles (of both matrices in the gated block).  Weights still
// go from memory to operand registers, two blocks ahead.  16-bit types.
//
// Bound: up to about 16 rows the weights' bytes with the start and end of a
// launch (5120 -> 13824 in 4 bits, 40 MB, bf16: 12.2 us for 16 rows, 15.9 for 32;
// a plain stream of those bytes takes 7.1); beyond, the unpacking and MFMAs of
// each block of rows (64 rows 22.9 us, 256 rows 72).
#pragma once

#include <type_traits>

#include "proj_rows.hpp"

namespace sgmv {

template <typename DT, typename Src, int MT, int NTW, int KG, int NG, int S, int FL, bool kGated>
__global__ __launch_bounds__(kRowsThreads) void strip_kernel(RowsArgs a) {
    static_assert(DT::kBytes == 2 && KG * NG == kRowsWaves, "eight waves, 16-bit types");
    constexpr int NM = kGated ? 2 : 1;
    constexpr int kFlushes = 4 / FL;
    constexpr int kWL = Src::kQ4 ? 1 : 4;
    constexpr int kWLoads = NM * NTW * (Src::kQ4 ? 2 : 4);  // loads of a weight block
    constexpr int kStage = MT * 4096;                       // bytes of a group's x block
    constexpr int kXLoads = MT * 4 / NG;                    // of a wave
    static_assert(kXLoads * NG == MT * 4, "whole loads per wave");
    constexpr int kTiles = NG * NM * MT * NTW;              // of a group
    constexpr int kPart = KG * kTiles * 1024;               // bytes of the partial sums
    constexpr int kBytes = KG * kStage > kPart ? KG * kStage : kPart;
    __shared__ __attribute__((aligned(16))) uint8_t s_x0[kBytes];
    __shared__ __attribute__((aligned(16))) uint8_t s_x1[KG * kStage];
    __shared__ __attribute__((aligned(16))) uint8_t s_x2[S > 2 ? KG * kStage : 16];
    __shared__ __attribute__((aligned(16))) uint8_t s_x3[S > 3 ? KG * kStage : 16];
    static_assert(S >= 2 && S <= 4, "two to four stages");

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int kg = wid / NG, ng = wid % NG;
    const int lr = lane & 15, lg = lane >> 4;
    const int nt0 = ((int)blockIdx.x * NG + ng) * NTW;
    const int m0 = (int)blockIdx.y * (16 * MT);
    const int ntiles = (a.N + 15) / 16;
    const int nit = (a.kblocks + KG - 1) / KG;  // blocks per group; past K x is zeros

    acc4_t acc[NM][MT][NTW];
#pragma unroll
    for (int q = 0; q < NM; ++q)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NTW; ++j) acc[q][i][j] = acc4_t{0.f, 0.f, 0.f, 0.f};

    // x: load u of the wave fills rows 4 (ng kXLoads + u) .. + 3 of the group's
    // block; 16-byte piece p of row r lies in slot p ^ (r % 16), which spreads the
    // 16 rows of an operand read over the banks.  Rows past R read the last row.
    const char* xsrc[kXLoads];
    int xpiece[kXLoads];
#pragma unroll
    for (int u = 0; u < kXLoads; ++u) {
        const int r = (ng * kXLoads + u) * 4 + lg;
        xpiece[u] = lr ^ (r & 15);
        xsrc[u] = (const char*)a.x + ((long long)min(m0 + r, a.R - 1) * a.K + xpiece[u] * 8) * 2;
    }
    using lds_t = __attribute__((address_space(3))) void;
    auto issue_x = [&](uint8_t* st, int it) {
        const int kb = kg + it * KG;
#pragma unroll
        for (int u = 0; u < kXLoads; ++u) {
            const char* p = kb * 128 + xpiece[u] * 8 < a.K ? xsrc[u] + (long long)kb * 256
                                                           : (const char*)&g_zero_piece;
            __builtin_amdgcn_global_load_lds(
                (const void*)p, (lds_t*)(st + kg * kStage + (ng * kXLoads + u) * 1024), 16, 0, 0);
        }
    };

    const char* wbase[NM][NTW];
    const char* mbase[NM][NTW];
#pragma unroll
    for (int q = 0; q < NM; ++q)
#pragma unroll
        for (int j = 0; j < NTW; ++j) {
            if constexpr (Src::kQ4) {
                const long long nt = min(nt0 + j, ntiles - 1);
                wbase[q][j] = (const char*)a.m[q].w + nt * a.kblocks * 1024 + lane * 16;
                mbase[q][j] = (const char*)a.m[q].meta + (nt * a.kblocks * 16 + lr) * (4 * kFlushes);
            } else {
                wbase[q][j] = (const char*)a.m[q].w +
                              (long long)min((nt0 + j) * 16 + lr, a.N - 1) * a.K * 2;
                mbase[q][j] = nullptr;
            }
        }
    struct Block {
        uint4 w[NM][NTW][kWL];
        uint32_t meta[NM][NTW][kFlushes];
    };
    // Blocks past the last re-read it; they are not used.
    auto load_w = [&](Block& b, int it) {
        const int kb = min(kg + it * KG, a.kblocks - 1);
#pragma unroll
        for (int q = 0; q < NM; ++q)
#pragma unroll
            for (int j = 0; j < NTW; ++j) {
                if constexpr (Src::kQ4) {
                    b.w[q][j][0] = load16_stream(wbase[q][j] + (long long)kb * 1024);
                    load_dwords<kFlushes>(mbase[q][j] + (long long)kb * (64 * kFlushes), b.meta[q][j]);
                } else {
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        // K is a multiple of 8: a piece past it is x's zeros
                        // against the row's last piece.
                        const int k = min(kb * 128 + s * 32 + 8 * lg, a.K - 8);
                        b.w[q][j][s] = load16(wbase[q][j] + (long long)k * 2);
                    }
                }
            }
    };
    // Operand of step s: row tile i at xoff[s] + 4096 i of the group's block.
    int xoff[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) xoff[s] = kg * kStage + lr * 256 + (((4 * s + lg) ^ lr) << 4);

    auto compute = [&](const uint8_t* st, const Block& b) {
        if constexpr (Src::kQ4) {
#pragma unroll
            for (int f = 0; f < kFlushes; ++f) {
                uint4 xv[FL][MT];
                acc4_t sx[MT];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    sx[i] = acc4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = 0; s < FL; ++s) {
                        xv[s][i] = load16(st + xoff[f * FL + s] + 4096 * i);
                        sx[i] = PieceOps<DT>::mma(xv[s][i], ones_piece<DT>(), sx[i]);
                    }
                }
#pragma unroll
                for (int q = 0; q < NM; ++q)
#pragma unroll
                    for (int j = 0; j < NTW; ++j) {
                        const uint4 wv = b.w[q][j][0];
                        const uint32_t wd[4] = {wv.x, wv.y, wv.z, wv.w};
                        float sc, zb;
                        meta_values<DT>(b.meta[q][j][f], sc, zb);
                        uint4 wp[FL];
#pragma unroll
                        for (int s = 0; s < FL; ++s) wp[s] = codes_biased<DT>(wd[f * FL + s]);
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            acc4_t t = acc4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int s = 0; s < FL; ++s) t = PieceOps<DT>::mma(xv[s][i], wp[s], t);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                acc[q][i][j][e] += sc * (t[e] - zb * sx[i][e]);
                        }
                    }
            }
        } else {
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const uint4 xv = load16(st + xoff[s] + 4096 * i);
#pragma unroll
                    for (int q = 0; q < NM; ++q)
#pragma unroll
                        for (int j = 0; j < NTW; ++j)
                            acc[q][i][j] = PieceOps<DT>::mma(xv, b.w[q][j][s], acc[q][i][j]);
                }
        }
    };

    // Loads are issued in the one order W(0); x(0), W(1); x(1), W(2); ..., before
    // the loop as in it, with nothing moved across the fences: the waits count
    // on it, and the compiler's own waits for the weight registers stay exact
    // only if every way into the loop has the same loads in flight, and nothing in
    // it branches: where two ways meet, it waits for every load.
    auto fence = [] {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // Block `it`: x has landed for this wave (only what was issued after it may be
    // outstanding: S - 1 weight blocks and S - 2 x blocks) and, after the barrier,
    // for every wave, each past block it - 1; then the stage that held that block
    // takes block it + S - 1.  That count is of the loop's loads: the steps after the
    // loop load weights that nobody uses, which the compiler drops, so they wait for
    // every load instead (the second of three would else read a block in flight).
    constexpr int kAfter = (S - 1) * kWLoads + (S - 2) * kXLoads;
    static_assert(kAfter < 64, "the wait count fits vmcnt");
    using InLoop = std::integral_constant<int, (kAfter & 15) | ((kAfter >> 4) << 14) | 0x0070>;
    using AllLoads = std::integral_constant<int, 0x0070>;
    auto step = [&](auto wait, uint8_t* st, uint8_t* ahead, Block& b, int it) {
        fence();
        __builtin_amdgcn_s_waitcnt(decltype(wait)::value);
        __builtin_amdgcn_s_barrier();
        fence();
        issue_x(ahead, it + S - 1);
        fence();
        compute(st, b);
        load_w(b, it + S);
        fence();
    };
    Block blk[S];
    load_w(blk[0], 0);
    fence();
    issue_x(s_x0, 0);
    fence();
    load_w(blk[1], 1);
    fence();
    if constexpr (S > 2) {
        issue_x(s_x1, 1);
        fence();
        load_w(blk[2], 2);
        fence();
    }
    if constexpr (S > 3) {
        issue_x(s_x2, 2);
        fence();
        load_w(blk[S - 1], 3);
        fence();
    }
    int it = 0;
    for (; it + S <= nit; it += S) {
        step(InLoop{}, s_x0, S == 2 ? s_x1 : S == 3 ? s_x2 : s_x3, blk[0], it);
        step(InLoop{}, s_x1, s_x0, blk[1], it + 1);
        if constexpr (S > 2) step(InLoop{}, s_x2, s_x1, blk[2], it + 2);
        if constexpr (S > 3) step(InLoop{}, s_x3, s_x2, blk[S - 1], it + 3);
    }
    if (it < nit) step(AllLoads{}, s_x0, S == 2 ? s_x1 : S == 3 ? s_x2 : s_x3, blk[0], it);
    if (S > 2 && it + 1 < nit) step(AllLoads{}, s_x1, s_x0, blk[1], it + 1);
    if constexpr (S > 3) {
        if (it + 2 < nit) step(AllLoads{}, s_x2, s_x1, blk[2], it + 2);
    }
    // Every wave's last reads are done, and no load past the last block is left in
    // flight to the stage that the partial sums take.
    fence();
    __builtin_amdgcn_s_waitcnt(AllLoads::value);
    __syncthreads();

    // ---- add the groups' partial tiles, finish, store -------------------------
    float* part = reinterpret_cast<float*>(s_x0);
#pragma unroll
    for (int q = 0; q < NM; ++q)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NTW; ++j) {
                const int tile = ((ng * NTW + j) * MT + i) * NM + q;
                *reinterpret_cast<acc4_t*>(part + (kg * kTiles + tile) * 256 + 4 * lane) = acc[q][i][j];
            }
    __syncthreads();
    for (int e = tid; e < kTiles / NM * 64; e += kRowsThreads) {
        const int tile = e >> 6, l = e & 63;
        const int mq = m0 + 16 * (tile % MT) + 4 * (l >> 4);
        const int n = ((int)blockIdx.x * NG * NTW + tile / MT) * 16 + (l & 15);
        if (mq >= a.R || n >= a.N) continue;
        acc4_t v[NM];
#pragma unroll
        for (int q = 0; q < NM; ++q) {
            v[q] = acc4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < KG; ++w)
                v[q] += *reinterpret_cast<const acc4_t*>(part + (w * kTiles + tile * NM + q) * 256 + 4 * l);
        }
        finish_rows<DT, kGated>(a, v, mq, n);
    }
}

}  // namespace sgmv
