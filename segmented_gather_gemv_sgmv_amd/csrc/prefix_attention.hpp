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
// and conversions of codes beside the matrix cores for prompts and wide prefixes.  Measured (kernel + join; heads
// of 128): 64 sequences of up to 1200 tokens behind 16384, 32 / 8 heads, 8 bits, bfloat16, 47 + 7 us (133 MB: 26
// at a copy's rate); 24 of up to 2000 behind 6000, 40 heads, 4 bits, float16, 49 + 5 (164 MB: 32); 5 prompts
// of 1556 rows behind 2048, 32 / 8 heads, 8 bits, bfloat16, 126 + 5 (70 GFLOP: 50 at a library product's rate).
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
// q goes through in three bfloat16 terms, which hold its 24 bits).  V's scale differs by key; how
// it and p enter the second product is told at the two kinds of items.  Sums, maxima and outputs are
// float32.
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
    uint32_t page_magic, page_one;    // ceil(2^32 / blocks_per_page) and 0; 0 and ~0 for one block a page
    const int *own_pages, *prefix_pages;
    int own_width, prefix_width;
    const int* plan;
    PlanLayout at;
    float* part_o;                    // [slot][P]
    float2* part_ml;                  // [slot]: maximum (of base 2), sum
    int rows, seqs, prefixes, q_heads, kv_heads, rep, D;
    float c;                          // scale * log2(e)
    int vec, o_vec;                   // q takes 16-byte loads, o stores of 4 elements
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
// Largest over a wave: quads swapped, halves of 8 and 16 mirrored, rows swapped.
__device__ __forceinline__ int wave_max(int v) {
    v = max(v, __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xf, 0xf, true));
    v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xf, 0xf, true));
    v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, true));
    v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x140, 0xf, 0xf, true));
    auto s = __builtin_amdgcn_permlane16_swap((unsigned)v, (unsigned)v, false, false);
    v = max((int)s[0], (int)s[1]);
    s = __builtin_amdgcn_permlane32_swap((unsigned)v, (unsigned)v, false, false);
    return __builtin_amdgcn_readfirstlane(max((int)s[0], (int)s[1]));
}

// Scale byte `i` of a word as the exponent of a float; sign and mantissa hold other bytes' bits,
// which the conversions of codes do not look at.
__device__ __forceinline__ float scale_operand(uint32_t w, int i) {
    return __uint_as_float(__builtin_amdgcn_alignbit(w, w, 9 + 8 * i));
}

// Two floats to two operands, nearest-even, in one instruction.
template <typename OT>
__device__ __forceinline__ uint32_t pack_operands(float a, float b) {
    typedef float f2_t __attribute__((ext_vector_type(2)));
    typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
    if constexpr (std::is_same<OT, F16>::value) return bits2(__builtin_convertvector((f2_t){a, b}, h2_t));
    else return pack2_rne<BF16>(a, b);
}

// ---------------------------------------------------------------------------
// The rows of a wave: R tiles of 16 rows, one row a lane column.  VT: the operands of the second product
// (see the two kinds of items below).
// ---------------------------------------------------------------------------
constexpr float kAttnSlack = 4.f;  // p may reach 2^4 before the maximum is moved

template <typename QT, int BITS, int P>
struct AttnTypes {
    static constexpr int kSteps = P / 32;                 // products over d of S
    static constexpr int kDTiles = P / 16;                // tiles of O over d
    static constexpr int kRow = P * BITS / 8;             // bytes of a token's codes; lines of V
    static constexpr int kPiece = kRow / 4;               // bytes of a token's codes that a lane takes
    static constexpr int kLines = kRow / 16;              // 16-byte lines of V a lane takes
    static constexpr int kLineTiles = 8 / BITS;           // tiles of O that a line feeds
    static constexpr int kGroups = BITS == 8 ? 1 : P / 32;
    static constexpr int kKGroups = BITS == 8 || P == 64 || P == 128 ? 1 : 2;  // that a lane's piece of K meets
    static constexpr int kQTerms = QT::kBytes == 4 ? 3 : 1;
    using KT = std::conditional_t<std::is_same<QT, F16>::value, F16, BF16>;  // operands of S
};

// An item as its workgroup sees it.  Its steps of 64 keys run over the prefix in front, if any, and then over the
// stack's keys.
struct Keys {
    int len;
    const int* table;   // pages
};
struct Item {
    int tile, head, m0, blk0, blk1, slot, row0, M;
    Keys keys, front;
    int front_blocks;
    bool own, final;    // own: the rows are the last of the keys' tokens; final: outputs come from here
    int hidden;         // own: tokens before the first row
    uint32_t stride, base;  // blocks of a page (of all heads), of the heads before this one
};

__device__ __forceinline__ Item attn_item(const AttnArgs& a, const int* e) {
    Item t;
    t.tile = e[kItemTile];
    t.head = e[kItemHead];
    t.m0 = e[kItemM0];
    t.blk0 = e[kItemBlk0];
    t.blk1 = e[kItemBlk1];
    t.slot = e[kItemSlot];
    t.row0 = e[kItemRow0];
    t.M = e[kItemM];
    t.own = e[kItemOwn] != 0;
    t.hidden = e[kItemHidden];
    t.final = e[kItemFinal] != 0;
    t.keys.len = e[kItemLen];
    t.keys.table = t.own ? a.own_pages + (long long)e[kItemTable] * a.own_width
                         : a.prefix_pages + (long long)e[kItemTable] * a.prefix_width;
    t.front.len = e[kItemFrontLen];
    t.front.table = a.prefix_pages + (long long)max(e[kItemFrontTable], 0) * a.prefix_width;
    t.front_blocks = e[kItemFrontBlocks];
    t.stride = (uint32_t)a.kv_heads * a.blocks_per_page;
    t.base = (uint32_t)t.head * a.blocks_per_page;
    return t;
}

// End of the steps that row `m` sees, and with it all rows before it.  A row whose place lies before the first own
// token (fewer tokens than rows) sees none of them, and all of a prefix in front.
__device__ __forceinline__ int steps_seen(const AttnArgs& a, const Item& it, int m) {
    const int keys = it.own ? max(it.hidden + m / a.rep + 1, 0) : it.keys.len;
    return min(it.blk1, it.front_blocks + (keys + kAttnKeys - 1) / kAttnKeys);
}

// Where a wave's next steps find their keys: steps `first`, first + stride, ... of the item, four 16-token blocks
// each.  A lane looks up one block, so the wave knows 16 steps at a time; a step gets its blocks from
// their lanes.  Page entries for the 16 steps after that are asked for by every step (from L1), so that
// the load stands in no branch and no step waits for the one it has just issued.
struct KeyWalk {
    static constexpr uint32_t kNone = ~0u;
    const AttnArgs& a;
    const Item& it;
    int lane, blk, stride;     // blk: of the group to come
    uint32_t cur;              // blocks of the group at hand, counted over pages and heads; kNone: not there
    int pos, page, in;
    bool there;
    const int* entry;          // of the group to come

    __device__ __forceinline__ KeyWalk(const AttnArgs& args, const Item& item, int l, int first, int step)
        : a(args), it(item), lane(l), blk(first), stride(step) {
        aim();
        page = *entry;
        turn();
        page = *entry;
    }
    // The lane's block of the group that begins at step blk.
    __device__ __forceinline__ void aim() {
        const int s = blk + (lane >> 2) * stride;
        const bool front = s < it.front_blocks;
        const Keys keys = front || it.keys.len == 0 ? it.front : it.keys;
        const int b = (front ? s : s - it.front_blocks) * 4 + (lane & 3);
        there = b * kKvBlock < keys.len && s < it.blk1;
        const uint32_t c = there ? (uint32_t)b : 0u;  // entry 0 where there is none: an item has a token
        const uint32_t index = __umulhi(c, a.page_magic) + (c & a.page_one);
        in = (int)(c - index * (uint32_t)a.blocks_per_page);
        entry = keys.table + index;
    }
    __device__ __forceinline__ void turn() {
        const bool ok = there && (unsigned)page < (unsigned)a.num_pages;
        cur = ok ? (uint32_t)page * it.stride + it.base + (uint32_t)in : kNone;
        pos = 0;
        blk += 16 * stride;
        aim();
    }
    // Of the next step, the block of K that the lane's token lies in and the lane's block of V.
    __device__ __forceinline__ void next(int sub_k, int sub_v, uint32_t& k, uint32_t& v) {
        if (pos == 16) turn();
        page = *entry;
        k = (uint32_t)__builtin_amdgcn_ds_bpermute((pos * 4 + sub_k) * 4, (int)cur);
        v = (uint32_t)__builtin_amdgcn_ds_bpermute((pos * 4 + sub_v) * 4, (int)cur);
        ++pos;
    }
};
constexpr int kWaitLoads = 0x0F70;  // s_waitcnt: no load outstanding, LDS and scalars as they are

// Keeps loads before it where they are written: without, a loop's loads for its next round are moved into that round.
__device__ __forceinline__ void loads_stay() { asm volatile("" ::: "memory"); }

// Natural logarithm of l 2^m, minus infinity for no key.
__device__ __forceinline__ float log_sum(float m, float l) {
    return l == 0.f ? -__builtin_inff() : (m + __builtin_log2f(l)) * 0.69314718055994531f;
}

// HEAD: p is held times 2^HEAD.  TERMS: operands that p is split into, one after the other.
template <typename QT, int BITS, int P, int R, typename VT, int TERMS, int HEAD>
struct AttnRows {
    using A = AttnTypes<QT, BITS, P>;
    using KT = typename A::KT;
    uint4 qf[R][A::kQTerms][A::kSteps];
    acc4_t o[R][A::kDTiles], s[R][4];
    float mref[R], l[R];
    int lim[R];   // keys that the lane's row sees (behind a prefix in front)
    int m_first;  // first row of the wave
    int blk_end;  // blocks that any of its rows sees

    // q: lane (lr, lg) holds d = lg P / 4 + 8 s + 0..7 of row lr of each tile.
    __device__ __forceinline__ void init(const AttnArgs& a, const Item& it, int first, int lr, int lg) {
        m_first = first;
        const int last = min(first + 16 * R, it.M) - 1;
        blk_end = last < first ? 0 : steps_seen(a, it, last);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int m = first + 16 * r + lr;
            const bool ok = m < it.M;
            const int i = ok ? m / a.rep : 0;
            const int h = it.head * a.rep + (ok ? m - i * a.rep : 0);
            lim[r] = ok && it.own ? it.hidden + i + 1 : it.keys.len;
            mref[r] = -__builtin_inff();
            l[r] = 0.f;
#pragma unroll
            for (int t = 0; t < A::kDTiles; ++t) o[r][t] = acc4_t{0.f, 0.f, 0.f, 0.f};
            const typename QT::storage* p =
                (const typename QT::storage*)a.q + (long long)(it.row0 + i) * a.q_row + (long long)h * a.q_head;
#pragma unroll
            for (int x = 0; x < A::kSteps; ++x) {
                const int d = lg * (P / 4) + 8 * x;
                float f[8];
                if (ok && a.vec && d + 8 <= a.D) {
                    if constexpr (QT::kBytes == 2) {
                        qf[r][0][x] = load16(p + d);
                        continue;
                    } else {
                        QT::unpack(load16(p + d), f);
                        QT::unpack(load16(p + d + 4), f + 4);
                    }
                } else {
#pragma unroll
                    for (int y = 0; y < 8; ++y) f[y] = ok && d + y < a.D ? QT::load1(p + d + y) : 0.f;
                }
#pragma unroll
                for (int t = 0; t < A::kQTerms; ++t) {
                    qf[r][t][x] = make_uint4(pack2_rne<KT>(f[0], f[1]), pack2_rne<KT>(f[2], f[3]),
                                             pack2_rne<KT>(f[4], f[5]), pack2_rne<KT>(f[6], f[7]));
                    if (t + 1 < A::kQTerms) {
                        float g[8];
                        KT::unpack(qf[r][t][x], g);
#pragma unroll
                        for (int y = 0; y < 8; ++y) f[y] -= g[y];
                    }
                }
            }
        }
    }

    // S tile t += K Q^T of the d of step x.
    __device__ __forceinline__ void score(int t, int x, const uint4& kf) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int y = 0; y < A::kQTerms; ++y)
                s[r][t] = PieceOps<KT>::mma(kf, qf[r][y][x], x == 0 && y == 0 ? acc4_t{0.f, 0.f, 0.f, 0.f} : s[r][t]);
    }

    // Of the lane's 16 keys from `first` on, `there` are in the cache; rows see all of a prefix in `front` of their own
    // keys.  How many a row sees, and whether every row of the wave sees all of its 16.
    __device__ __forceinline__ int seen(int r, int first, int there, bool front) const {
        return front ? there : min(lim[r] - first, there);
    }
    __device__ __forceinline__ bool all_seen(int first, int there, bool front) const {
        bool whole = true;
#pragma unroll
        for (int r = 0; r < R; ++r) whole = whole && seen(r, first, there, front) >= 16;
        return __all(whole);
    }

    // Keys that a row does not see: their scores.
    __device__ __forceinline__ void mask(int first, int there, bool front) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int rem = seen(r, first, there, front);
#pragma unroll
            for (int t = 0; t < 16; ++t)
                if (t >= rem) s[r][t / 4][t % 4] = -__builtin_inff();
        }
    }

    // Running maxima, moved only where p would pass 2^4.
    __device__ __forceinline__ void maxima(float c) {
        float mx[R];
        bool move = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float v = s[r][0][0];
#pragma unroll
            for (int t = 1; t < 16; ++t) v = fmaxf(v, s[r][t / 4][t % 4]);
            mx[r] = column_max(v) * c;
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
                for (int t = 0; t < A::kDTiles; ++t) o[r][t] *= f;
            }
        }
    }

    // Scores of half u of the lane's keys, tile r, to p; running sums.
    __device__ __forceinline__ void soften(float c, int r, int u) {
        const float m = (mref[r] == -__builtin_inff() ? 0.f : mref[r]) - HEAD;
#pragma unroll
        for (int t = 8 * u; t < 8 * u + 8; ++t) {
            const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][t / 4][t % 4], c, -m));
            s[r][t / 4][t % 4] = p;
            l[r] += p;
        }
    }

    // w [8] as operands, each part what the parts before left.
    static __device__ __forceinline__ void split(float* w, uint4* pf) {
#pragma unroll
        for (int x = 0; x < TERMS; ++x) {
            pf[x] = make_uint4(pack_operands<VT>(w[0], w[1]), pack_operands<VT>(w[2], w[3]),
                               pack_operands<VT>(w[4], w[5]), pack_operands<VT>(w[6], w[7]));
            if (x + 1 < TERMS) {
                float h[8];
                VT::unpack(pf[x], h);
#pragma unroll
                for (int y = 0; y < 8; ++y) w[y] -= h[y];
            }
        }
    }

    __device__ __forceinline__ void product(int tile, int r, const uint4& vf, const uint4* pf) {
#pragma unroll
        for (int x = 0; x < TERMS; ++x) o[r][tile] = PieceOps<VT>::mma(vf, pf[x], o[r][tile]);
    }

    // The wave's rows to their slots, or to the outputs.
    __device__ __forceinline__ void write(const AttnArgs& a, const Item& it, int lr, int lg) const {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int m = m_first + 16 * r + lr;
            if (m >= it.M) continue;
            if (it.final) {
                const int i = m / a.rep, h = it.head * a.rep + m - i * a.rep;
                const long long row = it.row0 + i;
                const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
                typename QT::storage* out = (typename QT::storage*)a.o + row * a.o_row + (long long)h * a.o_head + lg * 4;
#pragma unroll
                for (int d = 0; d < A::kDTiles; ++d) {
                    float f[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) f[x] = o[r][d][x] * inv;
                    store4f<QT>(out + 16 * d, a.D - 16 * d - lg * 4, a.o_vec, f);
                }
                if (a.lse && lg == 0) a.lse[row * a.q_heads + h] = log_sum(mref[r], l[r]);
                continue;
            }
            const long long slot = (long long)it.slot + m - it.m0;
            float* out = a.part_o + slot * P + lg * 4;
#pragma unroll
            for (int d = 0; d < A::kDTiles; ++d) *reinterpret_cast<acc4_t*>(out + 16 * d) = o[r][d];
            if (lg == 0) a.part_ml[slot] = make_float2(mref[r], l[r]);
        }
    }
};

// 4-bit codes of a line, two words (8 tokens): a byte holds a token's codes of two tiles.  Converted with the
// tokens' scales, then sorted by tile.
template <typename VT>
__device__ __forceinline__ void line_operands4(const uint32_t* w, const float* scale, uint4* vf) {
    uint32_t c[8];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        c[4 * y] = code_pair<VT, 4, 0>(w[y], scale[4 * y]);
        c[4 * y + 1] = code_pair<VT, 4, 1>(w[y], scale[4 * y + 1]);
        c[4 * y + 2] = code_pair<VT, 4, 2>(w[y], scale[4 * y + 2]);
        c[4 * y + 3] = code_pair<VT, 4, 3>(w[y], scale[4 * y + 3]);
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const uint32_t sel = y ? 0x07060302u : 0x05040100u;
        vf[y] = make_uint4(__builtin_amdgcn_perm(c[1], c[0], sel), __builtin_amdgcn_perm(c[3], c[2], sel),
                           __builtin_amdgcn_perm(c[5], c[4], sel), __builtin_amdgcn_perm(c[7], c[6], sel));
    }
}

// ---------------------------------------------------------------------------
// Items of up to 32 rows: codes go from memory to operand registers, every wave has keys of its own
// (of 32 rows two waves share them), and the waves' results are joined through LDS.
//
// Operands of the second product are bfloat16, whose range takes every scale as it is: 8-bit codes enter
// as they are and p times the key's scale, in two terms (16 bits; float32 outputs: three); 4-bit
// codes enter with their scale, p alone.
// ---------------------------------------------------------------------------
template <typename QT, int BITS, int P>
__device__ __forceinline__ void attn_direct(const AttnArgs& a, const Item& it, unsigned char* lds) {
    using A = AttnTypes<QT, BITS, P>;
    constexpr int kTerms = QT::kBytes == 4 ? 3 : 2;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int lr = lane & 15, lg = lane >> 4;
    const int waves_m = it.tile / 16, waves_k = kAttnWaves / waves_m;
    const int wm = wave % waves_m, wk = wave / waves_m;
    AttnRows<QT, BITS, P, 1, BF16, kTerms, 0> rows;
    rows.init(a, it, it.m0 + wm * 16, lr, lg);

    int blk = it.blk0 + wk;
    const int end = rows.blk_end;
    uint32_t kw[4][A::kPiece / 4], ks[A::kKGroups][4], vw[A::kLines][4], vs[A::kGroups][4];
    bool v_ok = false;
    const int g0 = BITS == 8 ? 0 : (lg * (P / 4)) >> 5;
    // Behind the last step loads go on, to block 0 of the cache: in a branch they would have every step wait for all.
    KeyWalk walk(a, it, lane, blk, waves_k);
    uint32_t block_v;
    auto load_k = [&] {
        uint32_t b;
        walk.next(lr >> 2, lg, b, block_v);
        b = b == KeyWalk::kNone ? 0u : b;
        const uint8_t* p = a.k + ((lr & 3) * A::kRow + lg * A::kPiece) + (uint64_t)b * (16 * A::kRow);
#pragma unroll
        for (int t = 0; t < 4; ++t) load_words<A::kPiece>(p + t * 4 * A::kRow, kw[t]);
        const uint8_t* scales = a.k_scales + (uint64_t)b * (16 * A::kGroups);
#pragma unroll
        for (int g = 0; g < A::kKGroups; ++g) load_words<16>(scales + min(g0 + g, A::kGroups - 1) * 16, ks[g]);
    };
    auto load_v = [&] {
        v_ok = block_v != KeyWalk::kNone;
        const uint32_t b = v_ok ? block_v : 0u;
        const uint8_t* p = a.v + lr * 16 + (uint64_t)b * (16 * A::kRow);
#pragma unroll
        for (int i = 0; i < A::kLines; ++i) load_words<16>(p + i * 256, vw[i]);
        const uint8_t* scales = a.v_scales + (uint64_t)b * (16 * A::kGroups);
#pragma unroll
        for (int g = 0; g < A::kGroups; ++g) load_words<16>(scales + g * 16, vs[g]);
    };
    // A step whose keys are not all seen by all rows.  V's scales of tokens that are not there may be
    // anything, and a NaN's must not meet rows that do not see it: both become 0, and the rows
    // that do see it (returned) are to be made NaN.
    auto partial = [&](int first, int there) {
        rows.mask(first, there, false);
        const int rem = rows.seen(0, first, there, false);
        bool poison = false;
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            const uint32_t bits = 255u << (8 * (t % 4));
            const bool nan = (vs[0][t / 4] & bits) == bits && t < there;
            poison = poison || (nan && t < rem);
#pragma unroll
            for (int g = 0; g < A::kGroups; ++g)
                if (nan || t >= there) vs[g][t / 4] &= ~bits;
        }
        return poison;
    };

    if (blk < end) {
        load_k();
        load_v();
        // q is there with them: else the loop's first step, and with it every one, would wait for it anew.
        __builtin_amdgcn_s_waitcnt(kWaitLoads);
    }
    while (blk < end) {
        // The step after this one is asked for behind its scores and behind its products.
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            float sc[A::kKGroups];
#pragma unroll
            for (int g = 0; g < A::kKGroups; ++g) sc[g] = scale_operand(ks[g][t], lr & 3);
#pragma unroll
            for (int x = 0; x < A::kSteps; ++x) {
                float scale = sc[0];
                if constexpr (A::kKGroups == 2)
                    if (((lg * (P / 4) + 8 * x) >> 5) != g0) scale = sc[1];
                rows.score(t, x, code_piece<typename A::KT, BITS>(kw[t] + x * (BITS / 4), scale));
            }
        }
        load_k();
        const int first = blk * kAttnKeys + lg * 16;
        const int there = v_ok ? it.keys.len - first : 0;
        bool poison = false;
        if (!rows.all_seen(first, there, false)) poison = partial(first, there);
        rows.maxima(a.c);
        rows.soften(a.c, 0, 0);
        rows.soften(a.c, 0, 1);
        uint4 pf[2][kTerms];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float w[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int t = 8 * u + x;
                w[x] = rows.s[0][t / 4][t % 4];
                if constexpr (BITS == 8) w[x] *= __uint_as_float(((vs[0][t / 4] >> (8 * (t % 4))) & 255u) << 23);
            }
            rows.split(w, pf[u]);
        }
#pragma unroll
        for (int i = 0; i < A::kLines; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if constexpr (BITS == 8) {
                    rows.product(i, 0, code_piece<BF16, 8>(vw[i] + 2 * u, 1.f), pf[u]);
                } else {
                    float scale[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) scale[x] = scale_operand(vs[i][2 * u + x / 4], x % 4);
                    uint4 vf[2];
                    line_operands4<BF16>(vw[i] + 2 * u, scale, vf);
                    rows.product(2 * i, 0, vf[0], pf[u]);
                    rows.product(2 * i + 1, 0, vf[1], pf[u]);
                }
            }
        if (__any(poison)) {
            const float nan = column_max(poison ? 1.f : 0.f) > 0.f ? __builtin_nanf("") : 0.f;
#pragma unroll
            for (int d = 0; d < A::kDTiles; ++d) rows.o[0][d] += nan;
        }
        load_v();
        loads_stay();
        blk += waves_k;
    }

    // The waves over the keys of the same rows: their maxima, then their sums pairwise.
    float* s_o = (float*)lds;
    float2* s_ml = (float2*)(lds + kAttnWaves / 2 * A::kDTiles * 1024);
    rows.l[0] = column_sum(rows.l[0]);
    if (lg == 0) s_ml[wave * 16 + lr] = make_float2(rows.mref[0], rows.l[0]);
    __syncthreads();
    float m = -__builtin_inff();
    for (int k = 0; k < waves_k; ++k) m = fmaxf(m, s_ml[(k * waves_m + wm) * 16 + lr].x);
    float l = 0.f;
    for (int k = 0; k < waves_k; ++k) {
        const float2 x = s_ml[(k * waves_m + wm) * 16 + lr];
        l += x.x == m ? x.y : x.y * __builtin_amdgcn_exp2f(x.x - m);
    }
    const float f = rows.mref[0] == m ? 1.f : __builtin_amdgcn_exp2f(rows.mref[0] - m);
#pragma unroll
    for (int d = 0; d < A::kDTiles; ++d) rows.o[0][d] *= f;
    rows.mref[0] = m;
    rows.l[0] = l;
    for (int half = waves_k / 2; half > 0; half /= 2) {
        float* at = s_o + (wm * (waves_k / 2) + (wk >= half ? wk - half : wk)) * (A::kDTiles * 256);
        if (wk >= half && wk < 2 * half) {
#pragma unroll
            for (int d = 0; d < A::kDTiles; ++d) *reinterpret_cast<acc4_t*>(at + (d * 64 + lane) * 4) = rows.o[0][d];
        }
        __syncthreads();
        if (wk < half) {
#pragma unroll
            for (int d = 0; d < A::kDTiles; ++d)
                rows.o[0][d] += *reinterpret_cast<const acc4_t*>(at + (d * 64 + lane) * 4);
        }
        __syncthreads();
    }
    if (wk == 0) rows.write(a, it, lr, lg);
}

// ---------------------------------------------------------------------------
// Items of 64 or 128 rows: the four waves share the keys.  Each converts a quarter of a step's codes
// into LDS, in the order in which lanes read them as operands (piece after piece of 16
// bytes a lane: no bank is met twice), one step ahead of the products.
//
// Operands of the second product are float16: p in one term (11 bits) for bfloat16 outputs, an eighth of what their
// own rounding loses (a second term: prompts 124 -> 157 us, 64 sequences behind 16384 tokens 47 -> 54), in two (22)
// for the others, and V scaled relative to the largest exponent that the item has met, which all waves follow alike;
// a value below 2^-32 of the largest is lost.  When a larger exponent comes, O is scaled down.
// ---------------------------------------------------------------------------
// Asks for MFMAS matrix instructions with VALU others, WRITES LDS writes and TRANS exponentials behind each.
template <int MFMAS, int VALU, int WRITES, int TRANS>
__device__ __forceinline__ void interleave() {
#pragma unroll
    for (int i = 0; i < MFMAS; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x2, VALU, 0);
        if constexpr (TRANS > 0) __builtin_amdgcn_sched_group_barrier(0x400, TRANS, 0);
        if constexpr (WRITES > 0) __builtin_amdgcn_sched_group_barrier(0x200, WRITES, 0);
    }
}

constexpr int kAttnHead = 11;  // p 2^11 reaches 2^15 at most

template <typename QT, int BITS, int P, int R>
__device__ __forceinline__ void attn_shared(const AttnArgs& a, const Item& it, unsigned char* lds) {
    using A = AttnTypes<QT, BITS, P>;
    constexpr int kTerms = std::is_same<QT, BF16>::value ? 1 : 2;
    constexpr int kMine = (A::kLines + kAttnWaves - 1) / kAttnWaves;  // lines of V that a wave converts
    constexpr int kKPieces = 4 * A::kSteps, kVPieces = A::kDTiles * 2, kStage = (kKPieces + kVPieces) * 64;
    constexpr int kUp = BITS == 8 ? 7 : 13;  // largest code 2^kUp stays below 65504
    static_assert(kAttnWaves == 4, "a wave converts one tile of K");
    uint4* stage = (uint4*)lds;  // two of kStage pieces
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    uint32_t* factors = (uint32_t*)(stage + 2 * kStage) + wave * 64 * kMine;  // the wave's own
    const int lr = lane & 15, lg = lane >> 4;
    AttnRows<QT, BITS, P, R, F16, kTerms, kAttnHead> rows;
    rows.init(a, it, it.m0 + wave * 16 * R, lr, lg);
    const int end = steps_seen(a, it, min(it.m0 + it.tile, it.M) - 1);  // of the workgroup's rows

    // Codes of the next step; vb: its scale bytes of V, one token a lane.
    uint32_t kw[A::kPiece / 4], vw[kMine][4], ks[A::kKGroups], vb[A::kGroups];
    const uint8_t *v_bytes = nullptr, *v_bytes_now = nullptr;  // of the lane's block
    bool ok = false;
    const int g0 = BITS == 8 ? 0 : (lg * (P / 4)) >> 5;
    KeyWalk walk(a, it, lane, it.blk0, 1);  // as in attn_direct loads go on behind the last step
    const int token = wave * 4 + (lr & 3);
    auto load = [&] {
        uint32_t bk, bv;
        walk.next(lr >> 2, lg, bk, bv);
        ok = bv != KeyWalk::kNone;
        bk = bk == KeyWalk::kNone ? 0u : bk;
        bv = ok ? bv : 0u;
        load_words<A::kPiece>(a.k + (token * A::kRow + lg * A::kPiece) + (uint64_t)bk * (16 * A::kRow), kw);
        const uint8_t* k_scales = a.k_scales + token + (uint64_t)bk * (16 * A::kGroups);
#pragma unroll
        for (int g = 0; g < A::kKGroups; ++g) ks[g] = k_scales[min(g0 + g, A::kGroups - 1) * 16];
        const uint8_t* p = a.v + (wave * 16 + lr) * 16 + (uint64_t)bv * (16 * A::kRow);
#pragma unroll
        for (int i = 0; i < kMine; ++i)
            if (A::kLines % kAttnWaves == 0 || i * kAttnWaves + wave < A::kLines)
                load_words<16>(p + i * kAttnWaves * 256, vw[i]);
        const uint8_t* v_scales = a.v_scales + lr + (uint64_t)bv * (16 * A::kGroups);
#pragma unroll
        for (int g = 0; g < A::kGroups; ++g) vb[g] = v_scales[g * 16];
        v_bytes = a.v_scales + (uint64_t)bv * (16 * A::kGroups);
    };
    // Exponents of the converted steps (biased), whether one of their tokens is a NaN, and whether the
    // lane's block of 16 tokens is there.
    int eref = 20, eref_next = 20;
    bool nan = false, nan_next = false, ok_now = false;
    // Step blk among its keys: the first of them, and how many there are.
    auto key_of = [&](int blk) { return (blk < it.front_blocks ? blk : blk - it.front_blocks) * kAttnKeys; };
    auto len_of = [&](int blk) { return blk < it.front_blocks ? it.front.len : it.keys.len; };
    auto convert = [&](int blk, uint4* to) {
        const bool there = ok && key_of(blk) + lane < len_of(blk);
        nan_next = __any(there && vb[0] == kKvNaN);
        int top = 0;
#pragma unroll
        for (int g = 0; g < A::kGroups; ++g) {
            if (!there || vb[g] == kKvNaN) vb[g] = 0;
            top = max(top, (int)vb[g]);
        }
        eref_next = max(eref_next, wave_max(top));
        // The tokens' factors 2^(b - eref + kUp), through the wave's own LDS from lane = token to all lanes of their
        // block: written here, read behind K's conversion.
#pragma unroll
        for (int i = 0; i < (BITS == 8 ? 1 : kMine); ++i) {
            uint32_t b = vb[0];
            if constexpr (BITS == 4) {
#pragma unroll
                for (int g = 1; g < A::kGroups; ++g) b = g == i * kAttnWaves + wave ? vb[g] : b;
            }
            const uint32_t bits = (uint32_t)max((int)b - eref_next + 127 + kUp, 0) << 23;
            if constexpr (BITS == 8) ((uint16_t*)factors)[lane] = F16::from_float(__uint_as_float(bits));
            else factors[i * 64 + lane] = bits;
        }
#pragma unroll
        for (int x = 0; x < A::kSteps; ++x) {
            uint32_t b = ks[0];
            if constexpr (A::kKGroups == 2)
                if (((lg * (P / 4) + 8 * x) >> 5) != g0) b = ks[1];
            to[(wave * A::kSteps + x) * 64 + lane] =
                code_piece<typename A::KT, BITS>(kw + x * (BITS / 4), __uint_as_float(b << 23));
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
        uint4 f[BITS == 8 ? 1 : kMine][BITS == 8 ? 2 : 4];
#pragma unroll
        for (int i = 0; i < (BITS == 8 ? 1 : kMine); ++i)
#pragma unroll
            for (int x = 0; x < (BITS == 8 ? 2 : 4); ++x)
                f[i][x] = ((const uint4*)factors)[BITS == 8 ? lg * 2 + x : i * 16 + lg * 4 + x];
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int line = i * kAttnWaves + wave;
            if (A::kLines % kAttnWaves != 0 && line >= A::kLines) continue;
            if constexpr (BITS == 8) {
                typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint4 c = code_piece<F16, 8>(vw[i] + 2 * u, 1.f);
                    auto times = [](uint32_t x, uint32_t y) {
                        return bits2(__builtin_bit_cast(h2_t, x) * __builtin_bit_cast(h2_t, y));
                    };
                    to[(kKPieces + line * 2 + u) * 64 + lane] =
                        make_uint4(times(c.x, f[0][u].x), times(c.y, f[0][u].y), times(c.z, f[0][u].z), times(c.w, f[0][u].w));
                }
            } else {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float scale[8];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint4 w = f[i][u * 2 + x];
                        scale[4 * x] = __uint_as_float(w.x);
                        scale[4 * x + 1] = __uint_as_float(w.y);
                        scale[4 * x + 2] = __uint_as_float(w.z);
                        scale[4 * x + 3] = __uint_as_float(w.w);
                    }
                    uint4 vf[2];
                    line_operands4<F16>(vw[i] + 2 * u, scale, vf);
#pragma unroll
                    for (int y = 0; y < 2; ++y) to[(kKPieces + (line * 2 + y) * 2 + u) * 64 + lane] = vf[y];
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    };
    // The loop is left out, not entered, where there is nothing: a path to it past the first conversion, which
    // waits for all loads, q's too, would have every step wait for the codes it has just asked for.  For the same
    // reason nothing is converted or asked for in a branch.
    int blk = it.blk0, n = 0;
    if (blk < end) {
        load();
        convert(blk, stage);
        ok_now = ok;
        v_bytes_now = v_bytes;
        nan = nan_next;
        load();
        do {
        // The stage of this step is written, and the other one read, by all waves.  Only LDS is waited for.
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
        const uint4* from = stage + n * kStage + lane;
        const bool mine = blk < rows.blk_end;
        if (eref_next > eref) {  // this step's values are relative to a larger exponent
            const float f = __builtin_ldexpf(1.f, max(eref - eref_next, -126));
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int t = 0; t < A::kDTiles; ++t) rows.o[r][t] *= f;
            eref = eref_next;
        }
        const bool ok_then = ok;
        const uint8_t* v_bytes_then = v_bytes;
        // Scores, K's operands a tile ahead of their products; behind the last operands the next step's codes are
        // converted, between the products: a wave issues one instruction in about five cycles, a product takes 16.
        uint4 kf[2][A::kSteps];
        auto fetch_k = [&](int t) {
#pragma unroll
            for (int x = 0; x < A::kSteps; ++x) kf[t & 1][x] = from[(t * A::kSteps + x) * 64];
        };
        auto score = [&](int t) {
#pragma unroll
            for (int x = 0; x < A::kSteps; ++x) rows.score(t, x, kf[t & 1][x]);
        };
        fetch_k(0);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            fetch_k(t + 1);
            __builtin_amdgcn_sched_barrier(0);
            score(t);
            __builtin_amdgcn_sched_barrier(0);
        }
        fetch_k(3);
        score(2);
        score(3);
        convert(blk + 1, stage + (n ^ 1) * kStage);
        interleave<2 * A::kSteps * R * A::kQTerms, 4, 1, 0>();
        load();
        if (mine) {
            const int first = key_of(blk) + lg * 16;
            const int there = ok_now ? len_of(blk) - first : 0;
            const bool front = blk < it.front_blocks;
            if (!rows.all_seen(first, there, front)) rows.mask(first, there, front);
            // V's operands four pieces ahead of their products, the first ones across the exponentials; p of the
            // second half of the keys between the products of the first.
            constexpr int kAhead = 4;
            uint4 vf[2][kAhead];
            auto fetch = [&](int i) {  // pieces [i, i + kAhead) in the order of their use: half u, tile
#pragma unroll
                for (int x = 0; x < kAhead; ++x)
                    vf[(i / kAhead) & 1][x] = from[(kKPieces + (i + x) % A::kDTiles * 2 + (i + x) / A::kDTiles) * 64];
            };
            static_assert(A::kDTiles % 2 == 0 && kVPieces % kAhead == 0, "whole groups of pieces");
            uint4 pf[2][R][kTerms];
            auto weigh = [&](int u) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    rows.soften(a.c, r, u);
                    float w[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) w[x] = rows.s[r][2 * u + x / 4][x % 4];
                    rows.split(w, pf[u][r]);
                }
            };
            auto products = [&](int i) {
#pragma unroll
                for (int x = 0; x < kAhead; ++x)
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        rows.product((i + x) % A::kDTiles, r, vf[(i / kAhead) & 1][x], pf[(i + x) / A::kDTiles][r]);
            };
            fetch(0);
            rows.maxima(a.c);
            weigh(0);
            __builtin_amdgcn_sched_barrier(0);
            weigh(1);
#pragma unroll
            for (int i = 0; i < A::kDTiles / kAhead * kAhead; i += kAhead) {
                fetch(i + kAhead);
                products(i);
            }
            interleave<A::kDTiles / kAhead * kAhead * R * kTerms, 4, 0, 1>();
#pragma unroll
            for (int i = A::kDTiles / kAhead * kAhead; i < kVPieces; i += kAhead) {
                if (i + kAhead < kVPieces) fetch(i + kAhead);
                __builtin_amdgcn_sched_barrier(0);
                products(i);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (__builtin_expect(nan, 0)) {
                // A NaN's values went in as zeros: rows that see it are made NaN.
                uint32_t w[4];
                load_words<16>(v_bytes_now, w);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int rem = rows.seen(r, first, there, front);
                    float bad = 0.f;
#pragma unroll
                    for (int t = 0; t < 16; ++t)
                        if (t < rem && ((w[t / 4] >> (8 * (t % 4))) & 255u) == kKvNaN) bad = 1.f;
                    const float v = column_max(bad) > 0.f ? __builtin_nanf("") : 0.f;
#pragma unroll
                    for (int t = 0; t < A::kDTiles; ++t) rows.o[r][t] += v;
                }
            }
        }
        ok_now = ok_then;
        v_bytes_now = v_bytes_then;
        nan = nan_next;
        n ^= 1;
        } while (++blk < end);
    }
    const float back = __builtin_ldexpf(1.f, eref - 127 - kUp - kAttnHead);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        rows.l[r] = column_sum(rows.l[r]) * (1.f / (1 << kAttnHead));
#pragma unroll
        for (int d = 0; d < A::kDTiles; ++d) rows.o[r][d] *= back;
    }
    rows.write(a, it, lr, lg);
}

template <typename QT, int BITS, int P, int RMAX>
__global__ __launch_bounds__(kAttnThreads, P <= 128 ? 2 : 1) void attn_kernel(AttnArgs a) {
    // attn_direct: sums of half the waves, maxima; attn_shared: two stages, factors.
    constexpr int kDirect = kAttnWaves / 2 * P / 16 * 1024 + kAttnWaves * 16 * 8;
    constexpr int kShared = 2 * P * 64 * 2 * 2 + (P * BITS / 128 + 3) / 4 * kAttnWaves * 64 * 4;
    __shared__ __align__(16) unsigned char lds[kDirect > kShared ? kDirect : kShared];
    if ((int)blockIdx.x >= a.plan[0]) return;
    const Item it = attn_item(a, a.plan + a.at.items + (long long)blockIdx.x * kItemInts);
    if (it.tile <= 32) attn_direct<QT, BITS, P>(a, it, lds);
    else if (RMAX == 1 || it.tile == 64) attn_shared<QT, BITS, P, 1>(a, it, lds);
    else attn_shared<QT, BITS, P, RMAX>(a, it, lds);
}

// A row's items into its output: LANES lanes, 4 elements each.
template <typename DT, int P>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
    using T = typename DT::storage;
    constexpr int kLanes = attn_join_lanes(P);
    const int lane = threadIdx.x & (kLanes - 1);
    const long long i = (long long)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
    if (i >= (long long)a.rows * a.q_heads) return;
    const int row = (int)(i / a.q_heads), h = (int)(i - (long long)row * a.q_heads);
    const int seq = a.plan[a.at.row_seq + row];
    if (seq < 0 || seq >= a.seqs) return;
    // The sequence's stack and its prefix's, looked over since a table may be malformed.
    int first[2], step[2], chunks[2];
    int prefix = -1;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        first[w] = step[w] = chunks[w] = 0;
        const int stack = w == 0 ? a.prefixes + seq : prefix;
        if (stack < 0 || (w == 1 && stack >= a.prefixes)) continue;
        const int* r = a.plan + a.at.stacks + (long long)stack * kStackInts;
        if (w == 0) {
            if (r[kStackDone]) return;
            prefix = r[kStackPrefix];
        }
        if (row < r[kStackRow0] || row >= r[kStackRow0] + r[kStackRows]) {
            if (w == 0) return;  // covered by no sequence after all
            continue;
        }
        const int tile = r[kStackTile], m = (row - r[kStackRow0]) * a.rep + h % a.rep, mt = m / tile;
        chunks[w] = r[kStackChunks];
        step[w] = tile;
        first[w] = r[kStackSlot0] + ((h / a.rep) * r[kStackTiles] + mt) * chunks[w] * tile + (m - mt * tile);
    }
    const int n = chunks[0] + chunks[1];
    auto slot = [&](int j) {
        return (long long)(j < chunks[0] ? first[0] + j * step[0] : first[1] + (j - chunks[0]) * step[1]);
    };
    // Factors of the items' results, one a lane; where there are more items than lanes, in turns, what was summed
    // before becoming one more result.
    float m = -__builtin_inff(), l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool mine = lane * 4 < P;
    for (int j0 = 0; j0 < n; j0 += kLanes) {
        const int count = min(n - j0, kLanes);
        float2 x = make_float2(-__builtin_inff(), 0.f);
        if (lane < count) x = a.part_ml[slot(j0 + lane)];
        float top = x.y != 0.f ? x.x : -__builtin_inff();  // no key was visible: nothing; a NaN goes on
#pragma unroll
        for (int k = 1; k < kLanes; k *= 2) top = fmaxf(top, __shfl_xor(top, k));
        top = fmaxf(top, m);
        const float keep = l == 0.f ? 0.f : m == top ? 1.f : __builtin_amdgcn_exp2f(m - top);
        const float f = x.y == 0.f ? 0.f : x.x == top ? 1.f : __builtin_amdgcn_exp2f(x.x - top);
        float sum = f * x.y;
#pragma unroll
        for (int k = 1; k < kLanes; k *= 2) sum += __shfl_xor(sum, k);
        l = l * keep + sum;
        o.x *= keep;
        o.y *= keep;
        o.z *= keep;
        o.w *= keep;
        m = top;
        // Results of no weight enter too: a visible NaN of V shows in them alone.
        for (int j = 0; j < count; j += 8) {
            float4 v[8];
            float g[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int at = min(j + k, count - 1);
                g[k] = __shfl(f, at, kLanes);
                v[k] = *reinterpret_cast<const float4*>(a.part_o + slot(j0 + at) * P + (mine ? lane * 4 : 0));
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (j + k >= count) continue;  // the last one again
                o.x += g[k] * v[k].x;
                o.y += g[k] * v[k].y;
                o.z += g[k] * v[k].z;
                o.w += g[k] * v[k].w;
            }
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T* out = (T*)a.o + (long long)row * a.o_row + (long long)h * a.o_head + lane * 4;
    const float f[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
    if (mine) store4f<DT>(out, a.D - lane * 4, a.o_vec, f);
    if (a.lse && lane == 0) a.lse[i] = log_sum(m, l);
}

}  // namespace sgmv
