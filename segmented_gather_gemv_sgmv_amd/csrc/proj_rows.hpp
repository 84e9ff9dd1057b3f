// proj_rows.hpp -- base projections of few rows (decode batches): x W^T with
// 4-bit or plain weights, and the gated block act(x Wg^T + a_g) (x Wu^T + a_u).
//
// Bound: the weights' bytes.  Each workgroup owns 16 * NTW output features
// (of one matrix, or of both of the gated block) and 16 * MT rows, and its
// eight waves split K in blocks of four operand pieces, so every weight is
// read once per 16 * MT rows, straight from memory into the MFMA operand
// registers; the eight float32 partial tiles are added in a fixed order
// through LDS.  Rows ride in the MFMA's 16 columns: a single row costs the
// same matrix-core time as 16, which is far below the weights' stream time.
//
// Weights are the first MFMA operand, so a lane ends with four consecutive
// features of one row.
#pragma once

#include "proj_device.hpp"

namespace sgmv {

constexpr int kRowsWaves = 8;
constexpr int kRowsThreads = kRowsWaves * kWave;

// One weight matrix: plain [N, K] (w), or 4-bit: packed tiles (w) with
// scales [N / 16][groups][16] and zero points likewise (NULL: 8).
struct ProjWeight {
    const void* w;
    const void* scales;
    const uint8_t* zeros;
};

struct RowsArgs {
    void* y;
    const void* x;
    ProjWeight m[2];      // m[1]: the up projection of the gated block
    const void* add[2];   // gated: addends before the activation [R, N] or NULL;
                          // else add[0] = bias [N] or NULL
    void* save[2];        // gated: where g and u are kept [R, N], or NULL
    int R, N, K;
    int kblocks;          // ceil(K / (16 kPK))
    int group_steps;      // 4-bit: steps of 32 K per group
    uint32_t group_magic; // ceil(2^32 / group_steps)
    int groups;           // 4-bit: groups per row
    int act;
    int xvec, wvec, yvec; // 16-byte pieces of x / of W; 4-element pieces of y and the addends
};

// Plain weights: one K block is four 16-byte pieces of a row.
template <typename DT>
struct PlainSrc {
    static constexpr bool kQ4 = false;
    static constexpr int kStepK = 4 * PieceOps<DT>::kPK;
    static constexpr int kXP = 1;  // x pieces per step
};
// 4-bit weights: one K block is four steps of 32 codes; float32 rows enter
// as three bf16 terms (their 24 bits exactly), so kXP = 3.
template <typename DT>
struct Q4Src {
    static constexpr bool kQ4 = true;
    static constexpr int kStepK = 32;
    static constexpr int kXP = 1;
};
template <>
struct Q4Src<F32> {
    static constexpr bool kQ4 = true;
    static constexpr int kStepK = 32;
    static constexpr int kXP = 3;
};

// The 16-bit type whose MFMA takes the codes.
template <typename DT>
struct CodeType {
    using type = DT;
};
template <>
struct CodeType<F32> {
    using type = BF16;
};

// Eight floats as three bf16 pieces whose sum is exact: each term is the
// truncation of what is left, 8 significant bits at a time.
__device__ __forceinline__ void split3(const float* f, uint4* out) {
    uint32_t t[3][4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        float a = f[2 * p], b = f[2 * p + 1];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const uint32_t ha = __float_as_uint(a) & 0xFFFF0000u;
            const uint32_t hb = __float_as_uint(b) & 0xFFFF0000u;
            t[i][p] = (ha >> 16) | hb;
            a -= __uint_as_float(ha);
            b -= __uint_as_float(hb);
        }
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) out[i] = make_uint4(t[i][0], t[i][1], t[i][2], t[i][3]);
}

// x for one step of 32 K (or one piece, plain weights).
template <typename DT, typename Src>
__device__ __forceinline__ void load_x_step(const typename DT::storage* row, int k0, int lg, int K,
                                            bool vec, uint4* out) {
    if constexpr (Src::kXP == 3) {
        float f[8];
        F32::unpack(load_piece<F32>(row, k0 + 8 * lg, K, vec), f);
        F32::unpack(load_piece<F32>(row, k0 + 8 * lg + 4, K, vec), f + 4);
        split3(f, out);
    } else {
        out[0] = load_piece<DT>(row, k0 + PieceOps<DT>::kPK * lg, K, vec);
    }
}

// Four consecutive scales (features 4 lg .. 4 lg + 3 of an n-tile) as floats.
template <typename DT>
__device__ __forceinline__ void load_scales4(const void* scales, long long index, float* s) {
    load4f<DT>((const typename DT::storage*)scales + index, 4, true, s);
}

// FL: steps per scale flush (4-bit): the group is a multiple of 32 FL.
template <typename DT, typename Src, int MT, int NTW, int FL, bool kGated>
__global__ __launch_bounds__(kRowsThreads) void rows_kernel(RowsArgs a) {
    using T = typename DT::storage;
    using CT = typename CodeType<DT>::type;
    constexpr int NM = kGated ? 2 : 1;
    constexpr int XP = Src::kXP;
    __shared__ __attribute__((aligned(16))) float s_part[kRowsWaves][NM * MT * NTW * 256];

    const int tid = threadIdx.x, lane = tid & (kWave - 1), wid = tid / kWave;
    const int lr = lane & 15, lg = lane >> 4;
    const int nt0 = (int)blockIdx.x * NTW;
    const int m0 = (int)blockIdx.y * (16 * MT);
    const int ntiles = (a.N + 15) / 16;
    const T* x = (const T*)a.x;

    acc4_t acc[NM][MT][NTW];
#pragma unroll
    for (int q = 0; q < NM; ++q)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NTW; ++j) acc[q][i][j] = acc4_t{0.f, 0.f, 0.f, 0.f};

    // Rows past R read the last row: their columns of the MFMA are not stored.
    const T* xrow[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
        xrow[i] = x + (long long)min(m0 + 16 * i + lr, a.R - 1) * a.K;

    for (int kb = wid; kb < a.kblocks; kb += kRowsWaves) {
        const int k0 = kb * 4 * Src::kStepK;
        uint4 xv[4][MT][XP];
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < MT; ++i)
                load_x_step<DT, Src>(xrow[i], k0 + s * Src::kStepK, lg, a.K, a.xvec, xv[s][i]);
        if constexpr (Src::kQ4) {
            // Sum of x over each flush, in every lane of the row's column: the
            // codes enter biased by 16, which is taken out with the zero point.
            acc4_t sx[4 / FL][MT];
#pragma unroll
            for (int f = 0; f < 4 / FL; ++f)
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    sx[f][i] = acc4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = 0; s < FL; ++s)
#pragma unroll
                        for (int p = 0; p < XP; ++p)
                            sx[f][i] = PieceOps<CT>::mma(ones_piece<CT>(), xv[f * FL + s][i][p], sx[f][i]);
                }
#pragma unroll
            for (int q = 0; q < NM; ++q)
#pragma unroll
                for (int j = 0; j < NTW; ++j) {
                    const int nt = min(nt0 + j, ntiles - 1);
                    const uint4 wv =
                        load16((const uint4*)a.m[q].w + ((long long)nt * a.kblocks + kb) * 64 + lane);
                    const uint32_t wd[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
                    for (int f = 0; f < 4 / FL; ++f) {
                        const int step = kb * 4 + f * FL;
                        int g = a.group_steps == 1 ? step : (int)__umulhi((uint32_t)step, a.group_magic);
                        g = min(g, a.groups - 1);  // the last block may run past K
                        const long long gi = ((long long)nt * a.groups + g) * 16 + 4 * lg;
                        float sc[4], zp[4];
                        load_scales4<DT>(a.m[q].scales, gi, sc);
                        uint32_t zw = 0x08080808u;
                        if (a.m[q].zeros) zw = *reinterpret_cast<const uint32_t*>(a.m[q].zeros + gi);
#pragma unroll
                        for (int e = 0; e < 4; ++e) zp[e] = kCodeBias + (float)((zw >> (8 * e)) & 255u);
                        uint4 wp[FL];
#pragma unroll
                        for (int s = 0; s < FL; ++s) wp[s] = codes_biased<CT>(wd[f * FL + s]);
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            acc4_t t = acc4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int s = 0; s < FL; ++s)
#pragma unroll
                                for (int p = 0; p < XP; ++p)
                                    t = PieceOps<CT>::mma(wp[s], xv[f * FL + s][i][p], t);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                acc[q][i][j][e] += sc[e] * (t[e] - zp[e] * sx[f][i][e]);
                        }
                    }
                }
        } else {
#pragma unroll
            for (int q = 0; q < NM; ++q)
#pragma unroll
                for (int j = 0; j < NTW; ++j) {
                    const T* wrow = (const T*)a.m[q].w +
                                    (long long)min((nt0 + j) * 16 + lr, a.N - 1) * a.K;
                    uint4 wp[4];
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        wp[s] = load_piece<DT>(wrow, k0 + s * Src::kStepK + PieceOps<DT>::kPK * lg,
                                               a.K, a.wvec);
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            acc[q][i][j] = PieceOps<DT>::mma(wp[s], xv[s][i][0], acc[q][i][j]);
                }
        }
    }

    // ---- add the waves' partial tiles, finish, store -------------------------
#pragma unroll
    for (int q = 0; q < NM; ++q)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NTW; ++j)
                *reinterpret_cast<acc4_t*>(&s_part[wid][((q * MT + i) * NTW + j) * 256 + 4 * lane]) =
                    acc[q][i][j];
    __syncthreads();
    for (int e = tid; e < MT * NTW * 64; e += kRowsThreads) {
        const int tile = e >> 6, l = e & 63;  // tile = i * NTW + j
        const int m = m0 + 16 * (tile / NTW) + (l & 15);
        const int n = (nt0 + tile % NTW) * 16 + 4 * (l >> 4);
        if (m >= a.R || n >= a.N) continue;
        float v[NM][4];
#pragma unroll
        for (int q = 0; q < NM; ++q) {
            acc4_t s = acc4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kRowsWaves; ++w)
                s += *reinterpret_cast<const acc4_t*>(&s_part[w][(q * MT * NTW + tile) * 256 + 4 * l]);
#pragma unroll
            for (int c = 0; c < 4; ++c) v[q][c] = s[c];
        }
        const long long at = (long long)m * a.N + n;
        const int left = a.N - n;
        float o[4];
        if constexpr (kGated) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (a.add[q]) {
                    float b[4];
                    load4f<DT>((const T*)a.add[q] + at, left, a.yvec, b);
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[q][c] += b[c];
                }
                if (a.save[q]) store4f<DT>((T*)a.save[q] + at, left, a.yvec, v[q]);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) o[c] = act_value(a.act, v[0][c]) * v[1][c];
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) o[c] = v[0][c];
            if (a.add[0]) {
                float b[4];
                load4f<DT>((const T*)a.add[0] + n, left, a.yvec, b);
#pragma unroll
                for (int c = 0; c < 4; ++c) o[c] += b[c];
            }
        }
        store4f<DT>((T*)a.y + at, left, a.yvec, o);
    }
}

}  // namespace sgmv
