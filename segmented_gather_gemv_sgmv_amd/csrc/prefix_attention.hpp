// prefix_attention.hpp -- attention of a batch over the quantized cache, where runs of
// sequences share a prefix that is read once for all of them.
//
// Row (i, h) of sequence s sees its run's prefix (all of it) and its own tokens up to
// its place (n rows are the last n of its tokens):
//     o = sum_k p_k v_k / sum_k p_k,  p_k = exp(scale q k_k - m),  lse = m + log sum_k p_k.
// The work is cut into stacks, tiles and chunks (prefix_plan.hpp); every item keeps running
// maxima and sums, and attn_join_kernel joins a row's items.
//
// Bound: HBM for decode batches (every code is read once per tile of rows), exponentials
// and conversions of codes beside the matrix cores for prompts and wide prefixes.
//
// A wave takes 64 keys a step and R tiles of 16 rows.  Both products run on
// v_mfma_f32_16x16x32 with the rows as columns: S^T = K Q^T and O^T = V^T P^T, so a row
// stays in one lane column (lane % 16) from its scores to its output and running maxima need
// no exchange but two lane swaps.  Which 16 keys form a tile of S is free, and so is
// the order of K within a product: S tile t, row m is key 16 (m / 4) + 4 t + m % 4,
// so that lane group g = lane / 16 holds scores of keys 16 g .. 16 g + 15, exactly the
// tokens of V that it reads as one 16-byte line.  No score passes through LDS, no code
// is transposed, every load is 16 bytes (K: pieces of a token's row).
//
// Types: codes of K become operands of q's type, scaled, in one conversion (exact; float32
// q goes through in three bfloat16 terms, which hold its 24 bits).  V's scale differs by
// key, so it multiplies p; p 2^e goes into float16 operands (11 bits; two terms, 22 bits, for
// float16 and float32 outputs), relative to the largest exponent seen, with 2^11 of
// headroom: what underflows is below 2^-35 of the largest value.  Sums, maxima and outputs
// are float32.
#pragma once

#include <type_traits>

#include "prefix_plan.hpp"
#include "proj_device.hpp"

namespace sgmv {

struct AttnArgs {
    const void* q;
    void* o;
    float* lse;                       // [rows, q_heads], or NULL
    long long q_row, q_head, o_row, o_head;  // strides in elements
    const uint8_t *k, *v, *k_scales, *v_scales;
    int num_pages, blocks_per_page;   // of 16 tokens
    uint32_t page_magic;              // ceil(2^32 / blocks_per_page)
    const int *own_pages, *prefix_pages;
    int own_width, prefix_width;
    const int* plan;
    PlanLayout at;
    float* part_o;                    // [slot][P]
    float2* part_ml;                  // [slot]: maximum (of base 2), sum
    int rows, seqs, prefixes, q_heads, kv_heads, rep, D;
    float c;                          // scale * log2(e)
    int vec;                          // q takes 16-byte loads
};

// ---------------------------------------------------------------------------
// Operands.
// ---------------------------------------------------------------------------
template <int BYTES>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
    if constexpr (BYTES % 16 == 0) {
#pragma unroll
        for (int i = 0; i < BYTES / 16; ++i) {
            const uint4 v = load16(p + 16 * i);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    } else if constexpr (BYTES % 8 == 0) {
#pragma unroll
        for (int i = 0; i < BYTES / 8; ++i) {
            const uint2 v = *reinterpret_cast<const uint2*>(p + 8 * i);
            w[2 * i] = v.x;
            w[2 * i + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < BYTES / 4; ++i) w[i] = *reinterpret_cast<const uint32_t*>(p + 4 * i);
    }
}

template <typename V>
__device__ __forceinline__ uint32_t bits2(V v) {
    return __builtin_bit_cast(uint32_t, v);
}

// Two codes of a word (its half or byte `sel`) as two operands of K, scaled.
template <typename QT, int BITS, int SEL>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, float scale) {
    if constexpr (std::is_same<QT, F16>::value) {
        if constexpr (BITS == 8) return bits2(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, SEL != 0));
        else return bits2(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, SEL));
    } else {
        if constexpr (BITS == 8) return bits2(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, SEL != 0));
        else return bits2(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL));
    }
}

// 8 consecutive codes (two words, or one of 4-bit codes) as an operand piece.
template <typename QT, int BITS>
__device__ __forceinline__ uint4 code_piece(const uint32_t* w, float scale) {
    if constexpr (BITS == 8)
        return make_uint4(code_pair<QT, 8, 0>(w[0], scale), code_pair<QT, 8, 1>(w[0], scale),
                          code_pair<QT, 8, 0>(w[1], scale), code_pair<QT, 8, 1>(w[1], scale));
    else
        return make_uint4(code_pair<QT, 4, 0>(w[0], scale), code_pair<QT, 4, 1>(w[0], scale),
                          code_pair<QT, 4, 2>(w[0], scale), code_pair<QT, 4, 3>(w[0], scale));
}

// Largest over the lanes of a column (lane % 16) and their sum.
__device__ __forceinline__ float column_max(float v) {
    auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
    s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float column_sum(float v) {
    auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) { return F16::pack2(a, b); }

// ---------------------------------------------------------------------------
// An item.
// ---------------------------------------------------------------------------
constexpr float kAttnSlack = 4.f;   // p may reach 2^4 before the maximum is moved
constexpr int kAttnHeadroom = 11;   // 2^(4 + 11) stays below float16's largest value

template <typename QT, int BITS, int P, int RMAX>
struct Attn {
    static constexpr int kSteps = P / 32;                 // products over d of S
    static constexpr int kDTiles = P / 16;                // tiles of O over d
    static constexpr int kRow = P * BITS / 8;             // bytes of a token's codes
    static constexpr int kPiece = kRow / 4;               // of a lane's
    static constexpr int kLines = BITS == 8 ? P / 16 : P / 32;  // 16-byte lines of V a lane reads
    static constexpr int kGroups = BITS == 8 ? 1 : P / 32;
    static constexpr int kKGroups = BITS == 8 || P == 64 || P == 128 ? 1 : 2;  // that a lane's piece of K meets
    static constexpr int kQTerms = QT::kBytes == 4 ? 3 : 1;
    static constexpr int kPTerms = std::is_same<QT, BF16>::value ? 1 : 2;
    using KT = std::conditional_t<std::is_same<QT, F16>::value, F16, BF16>;  // operands of S

    // Waves of one group over rows hold their sums here, one after the other.
    static constexpr int kLdsFloats = kAttnWaves / 2 * kDTiles * RMAX * 256;

    template <int R>
    static __device__ __forceinline__ void run(const AttnArgs& a, const int* e, float* s_o, float2* s_ml) {
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
        const int lr = lane & 15, lg = lane >> 4;
        const int stack = e[0], head = e[1], m0 = e[2], blk0 = e[3], tile = e[6];
        const int* rec = a.plan + a.at.stacks + (long long)stack * kStackInts;
        const int row0 = rec[0], M = rec[1] * a.rep, len = rec[2];
        const bool own = stack >= a.prefixes;
        const int* table = own ? a.own_pages + (long long)(stack - a.prefixes) * a.own_width
                               : a.prefix_pages + (long long)stack * a.prefix_width;
        const int waves_m = tile / (16 * R);
        const int waves_k = kAttnWaves / waves_m;
        const int wm = wave % waves_m, wk = wave / waves_m;
        const int mw = m0 + wm * 16 * R;  // first row of the wave
        // Keys that a row sees; rows of an own stack are the last of its tokens.
        const int hidden = own ? len - rec[1] : len;
        int lim[R];
        int most = 0;  // of the wave's rows
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int m = mw + 16 * r + lr;
            lim[r] = m >= M ? len : own ? hidden + m / a.rep + 1 : len;
        }
        {
            const int last = min(mw + 16 * R, M) - 1;
            most = last < mw ? 0 : own ? hidden + last / a.rep + 1 : len;
        }
        const int blk1 = min(e[4], (most + kAttnKeys - 1) / kAttnKeys);

        // q: lane (lr, lg) holds d = lg P / 4 + 8 s + 0..7 of row lr of each tile.
        uint4 qf[R][kQTerms][kSteps];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int m = mw + 16 * r + lr;
            const bool ok = m < M;
            const int i = ok ? m / a.rep : 0;
            const int h = head * a.rep + (ok ? m - i * a.rep : 0);
            const typename QT::storage* p =
                (const typename QT::storage*)a.q + (long long)(row0 + i) * a.q_row + (long long)h * a.q_head;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int d = lg * (P / 4) + 8 * s;
                float f[8];
                if (ok && a.vec && d + 8 <= a.D) {
                    if constexpr (QT::kBytes == 2) {
                        qf[r][0][s] = load16(p + d);
                        continue;
                    } else {
                        QT::unpack(load16(p + d), f);
                        QT::unpack(load16(p + d + 4), f + 4);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < 8; ++x) f[x] = ok && d + x < a.D ? QT::load1(p + d + x) : 0.f;
                }
#pragma unroll
                for (int t = 0; t < kQTerms; ++t) {
                    qf[r][t][s] = make_uint4(pack2_rne<KT>(f[0], f[1]), pack2_rne<KT>(f[2], f[3]),
                                             pack2_rne<KT>(f[4], f[5]), pack2_rne<KT>(f[6], f[7]));
                    if (t + 1 < kQTerms) {
                        float g[8];
                        KT::unpack(qf[r][t][s], g);
#pragma unroll
                        for (int x = 0; x < 8; ++x) f[x] -= g[x];
                    }
                }
            }
        }

        acc4_t o[R][kDTiles];
        float mref[R], l[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mref[r] = -__builtin_inff();
            l[r] = 0.f;
#pragma unroll
            for (int t = 0; t < kDTiles; ++t) o[r][t] = acc4_t{0.f, 0.f, 0.f, 0.f};
        }
        int eref = 20;  // biased exponent that p 2^e is relative to

        // Where 16-token block `b` of the stack lies (page 0 where there is none), if it is there.
        auto place = [&](int b, bool& ok) {
            const int pi = (int)__umulhi((uint32_t)b, a.page_magic);
            const int page_index = a.blocks_per_page == 1 ? b : pi;
            ok = b * kKvBlock < len;
            const int page = ok ? table[page_index] : 0;
            ok = ok && (unsigned)page < (unsigned)a.num_pages;
            const int in = ok ? b - page_index * a.blocks_per_page : 0;
            return ((long long)(ok ? page : 0) * a.kv_heads + head) * a.blocks_per_page + in;
        };
        uint32_t kw[4][kPiece / 4], ks[kKGroups][4];
        uint32_t vw[kLines][4], vs[kGroups][4];
        bool v_ok = false;
        const int g0 = BITS == 8 ? 0 : (lg * (P / 4)) >> 5;
        auto load_k = [&](int blk) {
            bool ok;
            const long long b = place(blk * 4 + (lr >> 2), ok);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                load_words<kPiece>(a.k + (b * 16 + t * 4 + (lr & 3)) * kRow + lg * kPiece, kw[t]);
#pragma unroll
            for (int g = 0; g < kKGroups; ++g)
                load_words<16>(a.k_scales + (b * kGroups + min(g0 + g, kGroups - 1)) * 16, ks[g]);
        };
        auto load_v = [&](int blk) {
            const long long b = place(blk * 4 + lg, v_ok);
#pragma unroll
            for (int i = 0; i < kLines; ++i) load_words<16>(a.v + (b * kRow + i * 16 + lr) * 16, vw[i]);
#pragma unroll
            for (int g = 0; g < kGroups; ++g) load_words<16>(a.v_scales + (b * kGroups + g) * 16, vs[g]);
        };

        int blk = blk0 + wk;
        if (blk < blk1) {
            load_k(blk);
            load_v(blk);
        }
        for (; blk < blk1; blk += waves_k) {
            // Scores.
            acc4_t s[R][4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                float sc[kKGroups];
#pragma unroll
                for (int g = 0; g < kKGroups; ++g) sc[g] = __uint_as_float(((ks[g][t] >> (8 * (lr & 3))) & 255u) << 23);
#pragma unroll
                for (int r = 0; r < R; ++r) s[r][t] = acc4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int d = 0; d < kSteps; ++d) {
                    float scale = sc[0];
                    if constexpr (kKGroups == 2)
                        if (((lg * (P / 4) + 8 * d) >> 5) != g0) scale = sc[1];
                    const uint4 kf = code_piece<KT, BITS>(kw[t] + d * (BITS / 4), scale);
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int x = 0; x < kQTerms; ++x) s[r][t] = PieceOps<KT>::mma(kf, qf[r][x][d], s[r][t]);
                }
            }
            const bool more = blk + waves_k < blk1;
            if (more) load_k(blk + waves_k);

            // Keys past a row's limit, or on a page that is not there.
            int rem[R];
            bool whole = true;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                rem[r] = v_ok ? lim[r] - (blk * kAttnKeys + lg * 16) : 0;
                whole = whole && rem[r] >= 16;
            }
            const bool all = __all(whole);
            const int there = v_ok ? len - (blk * kAttnKeys + lg * 16) : 0;  // tokens of the lane's block
            if (!all) {
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (t * 4 + i >= rem[r]) s[r][t][i] = -__builtin_inff();
            }
            // Running maxima, moved only where p would pass 2^4.
            float mx[R];
            bool move = false;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float v = -__builtin_inff();
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) v = fmaxf(v, s[r][t][i]);
                mx[r] = column_max(v) * a.c;
                move = move || mx[r] > mref[r] + kAttnSlack;
            }
            if (__any(move)) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float m = fmaxf(mref[r], mx[r]);
                    const float f = m == mref[r] ? 1.f : __builtin_amdgcn_exp2f(mref[r] - m);
                    mref[r] = m;
                    l[r] *= f;
#pragma unroll
                    for (int t = 0; t < kDTiles; ++t) o[r][t] *= f;
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float m = mref[r] == -__builtin_inff() ? 0.f : mref[r];
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][t][i], a.c, -m));
                        s[r][t][i] = p;
                        l[r] += p;
                    }
            }
            // V's scales; the largest exponent of tokens that are there (a NaN's is left out).
            auto factors = [&](int g, float* f) {
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    f[4 * t] = __uint_as_float((vs[g][t] << 23) & 0x7F800000u);
                    f[4 * t + 1] = __uint_as_float((vs[g][t] << 15) & 0x7F800000u);
                    f[4 * t + 2] = __uint_as_float((vs[g][t] << 7) & 0x7F800000u);
                    f[4 * t + 3] = __uint_as_float((vs[g][t] >> 1) & 0x7F800000u);
                }
                if (!all) {
#pragma unroll
                    for (int t = 0; t < 16; ++t) f[t] = t < there ? f[t] : 0.f;
                }
            };
            float top = 0.f;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                float f[16];
                factors(g, f);
#pragma unroll
                for (int t = 0; t < 16; ++t) top = fmaxf(top, f[t]);
            }
            top = column_max(top);
            if (__builtin_expect(__any(top == __builtin_inff()), 0)) {
                top = 0.f;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    float f[16];
                    factors(g, f);
#pragma unroll
                    for (int t = 0; t < 16; ++t) top = fmaxf(top, f[t] == __builtin_inff() ? 0.f : f[t]);
                }
                top = column_max(top);
            }
            const int etop = __builtin_amdgcn_readfirstlane((int)(__float_as_uint(top) >> 23));
            if (etop > eref) {
                const float f = __builtin_ldexpf(1.f, max(eref - etop, -126));
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int t = 0; t < kDTiles; ++t) o[r][t] *= f;
                eref = etop;
            }
            // 2^(headroom + 127 - eref): with a scale 2^(b - 127), p is multiplied by 2^(b - eref + headroom)
            const float unit = __builtin_ldexpf(1.f, kAttnHeadroom + 127 - eref);

            // O^T += V^T (p 2^e)^T: half u of a line's tokens at a time.
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                float f[16];
                factors(g, f);
#pragma unroll
                for (int t = 0; t < 16; ++t) f[t] *= unit;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint4 pf[R][kPTerms];
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        float w[8];
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            w[x] = s[r][2 * u + x / 4][x % 4] * f[8 * u + x];
                            if (!all && 8 * u + x >= rem[r]) w[x] = 0.f;  // what lies there may be NaN
                        }
#pragma unroll
                        for (int x = 0; x < kPTerms; ++x) {
                            pf[r][x] = make_uint4(pack_f16(w[0], w[1]), pack_f16(w[2], w[3]), pack_f16(w[4], w[5]),
                                                  pack_f16(w[6], w[7]));
                            if (x + 1 < kPTerms) {
                                float h[8];
                                F16::unpack(pf[r][x], h);
#pragma unroll
                                for (int y = 0; y < 8; ++y) w[y] -= h[y];
                            }
                        }
                    }
                    if constexpr (BITS == 8) {
#pragma unroll
                        for (int t = 0; t < kDTiles; ++t) {
                            const uint4 vf = code_piece<F16, 8>(vw[t] + 2 * u, 1.f);
#pragma unroll
                            for (int r = 0; r < R; ++r)
#pragma unroll
                                for (int x = 0; x < kPTerms; ++x) o[r][t] = PieceOps<F16>::mma(vf, pf[r][x], o[r][t]);
                        }
                    } else {
                        // A byte holds a token's codes of tiles 2 g (low) and 2 g + 1.
                        uint32_t c[8];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            c[4 * y] = code_pair<F16, 4, 0>(vw[g][2 * u + y], 1.f);
                            c[4 * y + 1] = code_pair<F16, 4, 1>(vw[g][2 * u + y], 1.f);
                            c[4 * y + 2] = code_pair<F16, 4, 2>(vw[g][2 * u + y], 1.f);
                            c[4 * y + 3] = code_pair<F16, 4, 3>(vw[g][2 * u + y], 1.f);
                        }
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint32_t sel = y ? 0x07060302u : 0x05040100u;
                            const uint4 vf = make_uint4(
                                __builtin_amdgcn_perm(c[1], c[0], sel), __builtin_amdgcn_perm(c[3], c[2], sel),
                                __builtin_amdgcn_perm(c[5], c[4], sel), __builtin_amdgcn_perm(c[7], c[6], sel));
#pragma unroll
                            for (int r = 0; r < R; ++r)
#pragma unroll
                                for (int x = 0; x < kPTerms; ++x)
                                    o[r][2 * g + y] = PieceOps<F16>::mma(vf, pf[r][x], o[r][2 * g + y]);
                        }
                    }
                }
            }
            if (more) load_v(blk + waves_k);
        }

        // The waves over the keys of the same rows: their maxima, then their sums pairwise.
#pragma unroll
        for (int r = 0; r < R; ++r) l[r] = column_sum(l[r]);
        const float back = __builtin_ldexpf(1.f, eref - 127 - kAttnHeadroom);
        if (lg == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) s_ml[(wave * R + r) * 16 + lr] = make_float2(mref[r], l[r]);
        __syncthreads();
        float m_all[R], l_all[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float m = -__builtin_inff();
            for (int k = 0; k < waves_k; ++k) m = fmaxf(m, s_ml[((k * waves_m + wm) * R + r) * 16 + lr].x);
            float t = 0.f;
            for (int k = 0; k < waves_k; ++k) {
                const float2 x = s_ml[((k * waves_m + wm) * R + r) * 16 + lr];
                t += x.x == m ? x.y : x.y * __builtin_amdgcn_exp2f(x.x - m);
            }
            m_all[r] = m;
            l_all[r] = t;
            const float f = (mref[r] == m ? 1.f : __builtin_amdgcn_exp2f(mref[r] - m)) * back;
#pragma unroll
            for (int d = 0; d < kDTiles; ++d) o[r][d] *= f;
        }
        for (int half = waves_k / 2; half > 0; half /= 2) {
            float* at = s_o + (size_t)(wm * (waves_k / 2) + (wk >= half ? wk - half : wk)) * (kDTiles * R * 256);
            if (wk >= half && wk < 2 * half) {
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int d = 0; d < kDTiles; ++d)
                        *reinterpret_cast<acc4_t*>(at + ((r * kDTiles + d) * 64 + lane) * 4) = o[r][d];
            }
            __syncthreads();
            if (wk < half) {
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int d = 0; d < kDTiles; ++d)
                        o[r][d] += *reinterpret_cast<const acc4_t*>(at + ((r * kDTiles + d) * 64 + lane) * 4);
            }
            __syncthreads();
        }
        if (wk == 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int m = mw + 16 * r + lr;
                if (m >= M) continue;
                const long long slot = (long long)e[5] + m - m0;
                float* out = a.part_o + slot * P + lg * 4;
#pragma unroll
                for (int d = 0; d < kDTiles; ++d) *reinterpret_cast<acc4_t*>(out + 16 * d) = o[r][d];
                if (lg == 0) a.part_ml[slot] = make_float2(m_all[r], l_all[r]);
            }
        }
    }
};

template <typename QT, int BITS, int P, int RMAX>
__global__ __launch_bounds__(kAttnThreads, 1) void attn_kernel(AttnArgs a) {
    using A = Attn<QT, BITS, P, RMAX>;
    __shared__ __align__(16) float s_o[A::kLdsFloats];
    __shared__ float2 s_ml[kAttnWaves * RMAX * 16];
    if ((int)blockIdx.x >= a.plan[0]) return;
    const int* e = a.plan + a.at.items + (long long)blockIdx.x * kItemInts;
    if constexpr (RMAX == 2) {
        if (e[6] == 16) {
            A::template run<1>(a, e, s_o, s_ml);
            return;
        }
    }
    A::template run<RMAX>(a, e, s_o, s_ml);
}

// A row's items into its output: LANES lanes, 4 elements each.
template <typename DT, int P>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
    using T = typename DT::storage;
    constexpr int kLanes = P <= 64 ? 16 : P <= 128 ? 32 : 64;
    const int lane = threadIdx.x & (kLanes - 1);
    const long long i = (long long)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
    if (i >= (long long)a.rows * a.q_heads) return;
    const int row = (int)(i / a.q_heads), h = (int)(i - (long long)row * a.q_heads);
    const int seq = a.plan[a.at.row_seq + row];
    if (seq < 0 || seq >= a.seqs) return;
    // The sequence's stack and its prefix's, looked over since a table may be malformed.
    int first[2], step[2], chunks[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        first[w] = step[w] = chunks[w] = 0;
        int stack = a.prefixes + seq;
        if (w == 1) {
            if (a.prefixes == 0) continue;
            stack = a.plan[a.at.seq_prefix + seq];
            if (stack < 0 || stack >= a.prefixes) continue;
        }
        const int* r = a.plan + a.at.stacks + (long long)stack * kStackInts;
        if (row < r[0] || row >= r[0] + r[1]) {
            if (w == 0) return;  // covered by no sequence after all
            continue;
        }
        const int m = (row - r[0]) * a.rep + h % a.rep, mt = m / r[6];
        chunks[w] = r[4];
        step[w] = r[6];
        first[w] = r[7] + ((h / a.rep) * r[5] + mt) * r[4] * r[6] + (m - mt * r[6]);
    }
    const int n = chunks[0] + chunks[1];
    auto slot = [&](int j) {
        return j < chunks[0] ? first[0] + j * step[0] : first[1] + (j - chunks[0]) * step[1];
    };
    float m = -__builtin_inff();
    for (int j = lane; j < n; j += kLanes) {
        const float2 x = a.part_ml[slot(j)];
        if (x.y != 0.f) m = fmaxf(m, x.x);
    }
#pragma unroll
    for (int k = 1; k < kLanes; k *= 2) m = fmaxf(m, __shfl_xor(m, k));
    float l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < n; ++j) {
        const float2 x = a.part_ml[slot(j)];
        if (x.y == 0.f) continue;  // no key was visible; a NaN goes on
        const float f = x.x == m ? 1.f : __builtin_amdgcn_exp2f(x.x - m);
        l += f * x.y;
        if (lane * 4 < P) {
            const float4 v = *reinterpret_cast<const float4*>(a.part_o + (long long)slot(j) * P + lane * 4);
            o[0] += f * v.x;
            o[1] += f * v.y;
            o[2] += f * v.z;
            o[3] += f * v.w;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T* out = (T*)a.o + (long long)row * a.o_row + (long long)h * a.o_head;
#pragma unroll
    for (int x = 0; x < 4; ++x)
        if (lane * 4 + x < a.D) out[lane * 4 + x] = DT::from_float(o[x] * inv);
    if (a.lse && lane == 0)
        a.lse[i] = l == 0.f ? -__builtin_inff() : (m + __builtin_log2f(l)) * 0.69314718055994531f;
}

}  // namespace sgmv
