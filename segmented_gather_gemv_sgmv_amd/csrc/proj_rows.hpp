// proj_rows.hpp -- base projections of few rows (decode batches): x W^T with
// 4-bit or plain weights, and the gated block act(x Wg^T + a_g) (x Wu^T + a_u).
//
// Bound: the weights' bytes.  Each workgroup owns 16 * NTW output features
// (of one matrix, or of both of the gated block) and 16 * MT rows, and its
// eight waves split K in blocks of four operand pieces, so every weight is
// read once per 16 * MT rows, straight from memory into the MFMA operand
// registers, PD blocks ahead of its use (one fp16 row, 4096 -> 4096 in 4 bits,
// 8.7 MB: 4.7 us, against 3.1 for a plain stream of those bytes; one bf16 row
// through the gated block of 4096 -> 11008, 180 MB: 33 us against 28); the eight
// float32 partial tiles are added in a fixed order through LDS.  Rows ride in
// the MFMA's 16 columns: a single row costs the same matrix-core time as 16,
// which is far below the weights' stream time.
//
// x is the first MFMA operand, so a lane's sums all belong to one output
// feature, lane % 16, and a 4-bit weight's scale is one value per lane.
#pragma once

#include "proj_device.hpp"

namespace sgmv {

constexpr int kRowsWaves = 8;
constexpr int kRowsThreads = kRowsWaves * kWave;

// One weight matrix: plain [N, K] (w), or 4-bit: packed tiles (w) and their
// scales (meta): per tile of 16 features by 128 K and feature, kFlushes = 1, 2
// or 4 pairs of scale and biased zero point 16 + z, one for each 128, 64 or 32
// of the tile's K (a longer group is repeated), so that a lane reads what it
// needs for a tile beside it in one load.  A pair is two 16-bit values of the
// activations' type in a dword, or two floats.
struct ProjWeight {
    const void* w;
    const void* meta;
};

struct RowsArgs {
    void* y;
    const void* x;
    ProjWeight m[2];      // m[1]: the up projection of the gated block
    const void* add[2];   // gated: addends before the activation [R, N] or NULL;
                          // else add[0] = bias [N] or NULL
    void* save[2];        // gated: where g and u are kept [R, N], or NULL
    int save_f32;         // they are kept in float32
    int R, N, K;
    int kblocks;          // blocks of four pieces of K
    int act;
    int xvec, wvec;       // 16-byte pieces of x / of W
};

// Plain weights: one K block is four 16-byte pieces of a row.  4-bit weights:
// four steps of 32 codes; float32 rows enter as three bf16 terms (their 24
// bits exactly).
template <typename DT>
struct PlainSrc {
    static constexpr bool kQ4 = false;
    static constexpr int kStepK = 4 * PieceOps<DT>::kPK;
    static constexpr int kXL = 1;  // 16-byte loads of x per step
    static constexpr int kXP = 1;  // MFMA operands of x per step
};
template <typename DT>
struct Q4Src {
    static constexpr bool kQ4 = true;
    static constexpr int kStepK = 32;
    static constexpr int kXL = DT::kBytes / 2;
    static constexpr int kXP = DT::kBytes == 4 ? 3 : 1;
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

// The scale and biased zero point of a 16-bit meta dword.
template <typename DT>
__device__ __forceinline__ void meta_values(uint32_t m, float& s, float& zb) {
    float f[2];
    DT::unpack2(m, f);
    s = f[0];
    zb = f[1];
}

// A piece of codes less their zero point, from the piece of codes biased by 16
// and zb = 16 + z: whole numbers of up to 8 bits, exact in bf16.  float32 results
// take them so; biased codes with 16 + z taken out of the sum are fewer
// instructions, but their sums are several times the result's size, and its
// rounding with them (5 rows x 1000: error 5e-7 that way, 1e-7 this way).
__device__ __forceinline__ uint4 codes_less_zero(const uint4& biased, float zb) {
    auto one = [zb](uint32_t d) {
        const uint32_t lo = __float_as_uint(__uint_as_float(d << 16) - zb);
        const uint32_t hi = __float_as_uint(__uint_as_float(d & 0xFFFF0000u) - zb);
        return (lo >> 16) | (hi & 0xFFFF0000u);
    };
    return make_uint4(one(biased.x), one(biased.y), one(biased.z), one(biased.w));
}

// n dwords at p in one load (p aligned to 4 n bytes).
template <int N>
__device__ __forceinline__ void load_dwords(const void* p, uint32_t* out) {
    if constexpr (N == 1) {
        out[0] = *(const uint32_t*)p;
    } else if constexpr (N == 2) {
        const uint2 v = load_pair(p);
        out[0] = v.x, out[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 v = load16((const uint4*)p + i);
            out[4 * i] = v.x, out[4 * i + 1] = v.y, out[4 * i + 2] = v.z, out[4 * i + 3] = v.w;
        }
    }
}

// Rotates each row of 16 lanes so that lanes 0..3 receive what lanes
// N .. N + 3 hold: DPP row_ror by 16 - N.
template <int N>
__device__ __forceinline__ uint4 row_down(const uint4& v) {
    if constexpr (N == 0) {
        return v;
    } else {
        auto one = [](uint32_t d) {
            return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)d, 0x120 + 16 - N, 0xf, 0xf, false);
        };
        return make_uint4(one(v.x), one(v.y), one(v.z), one(v.w));
    }
}

// Four rows' sums of feature n: addends, activation and product (gated) or
// bias, one rounding, store.
template <typename DT, bool kGated>
__device__ __forceinline__ void finish_rows(const RowsArgs& a, const acc4_t (&v)[kGated ? 2 : 1],
                                            int mq, int n) {
    using T = typename DT::storage;
    float bias = 0.f;
    if constexpr (!kGated) {
        if (a.add[0]) bias = DT::load1((const T*)a.add[0] + n);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (mq + c >= a.R) break;
        const long long at = (long long)(mq + c) * a.N + n;
        float o;
        if constexpr (kGated) {
            float p[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                p[q] = v[q][c];
                if (a.add[q]) p[q] += DT::load1((const T*)a.add[q] + at);
                if (a.save[q]) {
                    if (a.save_f32) ((float*)a.save[q])[at] = p[q];
                    else ((T*)a.save[q])[at] = DT::from_float(kept<DT>(p[q]));
                }
            }
            o = act_value(a.act, p[0]) * p[1];
        } else {
            o = v[0][c] + bias;
        }
        ((T*)a.y)[at] = DT::from_float(o);
    }
}

// XR: rows an x load brings.  16: lane lr loads row lr, one step per load.
// 4 (calls of at most four rows): one load brings the four steps of a block,
// lane lr taking row lr % 4 of step lr / 4, and a rotation moves a step's rows
// to the front (the MFMA's other columns then hold other steps' rows, and are
// not stored): x costs a quarter of the loads.  4096 -> 4096, one fp16 row:
// 4.6 us, against 5.6 us for the strip kernel's best shape.
// FL: steps per scale flush (4-bit): the group is a multiple of 32 FL.
template <typename DT, typename Src, int XR, int MT, int NTW, int PD, int FL, bool kGated>
__global__ __launch_bounds__(kRowsThreads) void rows_kernel(RowsArgs a) {
    using T = typename DT::storage;
    using CT = typename CodeType<DT>::type;
    constexpr int NM = kGated ? 2 : 1;
    constexpr int PK = PieceOps<DT>::kPK;
    constexpr int XL = Src::kXL, XP = Src::kXP;
    constexpr int kXLoads = XR == 16 ? 4 * XL : 1;  // x loads per block and row tile
    static_assert(XR == 16 || (XR == 4 && MT == 1 && XL == 1), "packed x loads are for one row tile");
    constexpr int kFlushes = 4 / FL;
    constexpr int kMeta = kFlushes * DT::kBytes / 2;  // dwords of a lane's pairs per tile
    constexpr int kWL = Src::kQ4 ? 1 : 4;      // weight loads per block and n-tile
    __shared__ __attribute__((aligned(16))) float s_part[kRowsWaves][NM * MT * NTW * 256];

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int lr = lane & 15, lg = lane >> 4;
    const int nt0 = (int)blockIdx.x * NTW;
    const int m0 = (int)blockIdx.y * (16 * MT);
    const int ntiles = (a.N + 15) / 16;

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
        xrow[i] = (const T*)a.x + (long long)min(m0 + 16 * i + lr % XR, a.R - 1) * a.K;
    const char* wbase[NM][NTW];
    const char* mbase[NM][NTW];
#pragma unroll
    for (int q = 0; q < NM; ++q)
#pragma unroll
        for (int j = 0; j < NTW; ++j) {
            if constexpr (Src::kQ4) {
                const long long nt = min(nt0 + j, ntiles - 1);
                wbase[q][j] = (const char*)a.m[q].w + nt * a.kblocks * 1024 + lane * 16;
                mbase[q][j] = (const char*)a.m[q].meta + (nt * a.kblocks * 16 + lr) * (4 * kMeta);
            } else {
                wbase[q][j] = (const char*)a.m[q].w +
                              (long long)min((nt0 + j) * 16 + lr, a.N - 1) * a.K * DT::kBytes;
                mbase[q][j] = nullptr;
            }
        }

    struct Block {
        uint4 x[MT][kXLoads];
        uint4 w[NM][NTW][kWL];
        uint32_t meta[Src::kQ4 ? NM : 1][NTW][kMeta];
    };
    Block blk[PD];
    // Blocks past the last re-read it (an L2 hit); they are not used.
    auto load = [&](Block& b, int kb) {
        kb = min(kb, a.kblocks - 1);
        const int k0 = kb * 4 * Src::kStepK;
#pragma unroll
        for (int q = 0; q < NM; ++q)
#pragma unroll
            for (int j = 0; j < NTW; ++j) {
                if constexpr (Src::kQ4) {
                    b.w[q][j][0] = load16_stream(wbase[q][j] + (long long)kb * 1024);
                    load_dwords<kMeta>(mbase[q][j] + (long long)kb * (64 * kMeta), b.meta[q][j]);
                } else {
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        b.w[q][j][s] = load_piece<DT>((const T*)wbase[q][j],
                                                      k0 + s * Src::kStepK + PK * lg, a.K, a.wvec);
                }
            }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int s = 0; s < kXLoads; ++s) {
                if constexpr (XR == 16) {
                    b.x[i][s] = load_piece<DT>(
                        xrow[i], k0 + (s / XL) * Src::kStepK + XL * PK * lg + PK * (s % XL), a.K, a.xvec);
                } else {
                    b.x[i][s] = load_piece<DT>(xrow[i], k0 + lr / 4 * Src::kStepK + PK * lg, a.K, a.xvec);
                }
            }
    };
    auto compute = [&](const Block& b) {
        uint4 xv[4][MT][XP];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            if constexpr (XR == 4) {
                xv[0][i][0] = b.x[i][0];
                xv[1][i][0] = row_down<4>(b.x[i][0]);
                xv[2][i][0] = row_down<8>(b.x[i][0]);
                xv[3][i][0] = row_down<12>(b.x[i][0]);
            } else {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    if constexpr (XP == 3) {
                        float f[8];
                        F32::unpack(b.x[i][2 * s], f);
                        F32::unpack(b.x[i][2 * s + 1], f + 4);
                        split3(f, xv[s][i]);
                    } else {
                        xv[s][i][0] = b.x[i][s];
                    }
                }
            }
        }
        if constexpr (Src::kQ4) {
            // 16-bit types: the codes enter biased by 16, which is taken out with
            // the zero point by the sum of x over each flush, in every column.
            constexpr bool kBiased = DT::kBytes == 2;
#pragma unroll
            for (int f = 0; f < kFlushes; ++f) {
                acc4_t sx[MT];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    sx[i] = acc4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = 0; s < (kBiased ? FL : 0); ++s)
                        sx[i] = PieceOps<CT>::mma(xv[f * FL + s][i][0], ones_piece<CT>(), sx[i]);
                }
#pragma unroll
                for (int q = 0; q < NM; ++q)
#pragma unroll
                    for (int j = 0; j < NTW; ++j) {
                        const uint4 wv = b.w[q][j][0];
                        const uint32_t wd[4] = {wv.x, wv.y, wv.z, wv.w};
                        float sc, zb;
                        if constexpr (DT::kBytes == 2) {
                            meta_values<DT>(b.meta[q][j][f], sc, zb);
                        } else {
                            sc = __uint_as_float(b.meta[q][j][2 * f]);
                            zb = __uint_as_float(b.meta[q][j][2 * f + 1]);
                        }
                        uint4 wp[FL];
#pragma unroll
                        for (int s = 0; s < FL; ++s) {
                            wp[s] = codes_biased<CT>(wd[f * FL + s]);
                            if constexpr (!kBiased) wp[s] = codes_less_zero(wp[s], zb);
                        }
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            acc4_t t = acc4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int s = 0; s < FL; ++s)
#pragma unroll
                                for (int p = 0; p < XP; ++p)
                                    t = PieceOps<CT>::mma(xv[f * FL + s][i][p], wp[s], t);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                acc[q][i][j][e] += sc * (kBiased ? t[e] - zb * sx[i][e] : t[e]);
                        }
                        // One n-tile's products at a time: interleaved freely, their
                        // partial sums spill.
                        if constexpr (MT * NTW >= 4) __builtin_amdgcn_sched_barrier(0);
                    }
            }
        } else {
#pragma unroll
            for (int q = 0; q < NM; ++q)
#pragma unroll
                for (int j = 0; j < NTW; ++j)
#pragma unroll
                    for (int s = 0; s < 4; ++s)
#pragma unroll
                        for (int i = 0; i < MT; ++i)
                            acc[q][i][j] = PieceOps<DT>::mma(xv[s][i][0], b.w[q][j][s], acc[q][i][j]);
        }
    };
#pragma unroll
    for (int d = 0; d < PD; ++d) load(blk[d], wid + d * kRowsWaves);
    int kb = wid;
    for (; kb + PD * kRowsWaves < a.kblocks; kb += PD * kRowsWaves) {
#pragma unroll
        for (int d = 0; d < PD; ++d) {
            compute(blk[d]);
            load(blk[d], kb + (d + PD) * kRowsWaves);
        }
    }
#pragma unroll
    for (int d = 0; d < PD; ++d)
        if (kb + d * kRowsWaves < a.kblocks) compute(blk[d]);

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
        const int mq = m0 + 16 * (tile / NTW) + 4 * (l >> 4);
        const int n = (nt0 + tile % NTW) * 16 + (l & 15);
        if (mq >= a.R || n >= a.N) continue;
        acc4_t v[NM];
#pragma unroll
        for (int q = 0; q < NM; ++q) {
            v[q] = acc4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kRowsWaves; ++w)
                v[q] += *reinterpret_cast<const acc4_t*>(&s_part[w][(q * MT * NTW + tile) * 256 + 4 * l]);
        }
        finish_rows<DT, kGated>(a, v, mq, n);
    }
}

}  // namespace sgmv
