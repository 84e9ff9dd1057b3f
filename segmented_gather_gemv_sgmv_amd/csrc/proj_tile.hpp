// proj_tile.hpp -- matrix products of many rows on the matrix cores: the
// gated block's forward, its gradients with respect to x and to the weights,
// and 4-bit projections of prompts.
//
// A workgroup computes a BM x BN tile of C[m][n] = sum_k A[m][k] B[n][k] in
// steps of 64 bytes of K (32 16-bit or 16 float32 values) through four LDS
// stages, filled by direct global-to-LDS loads three steps ahead, so no register
// holds a tile in flight.  A lane past the end of K loads zeros (an offset past
// its buffer's range).  Operands that no 16-byte load fits go through registers
// instead (kDma false), several times slower.
//
// Bound: the matrix cores at the clock the chip holds under them.  A step of a
// 256 x 256 tile is 64 MFMAs per SIMD, 0.57 us at the 1.8 GHz measured under this
// load (2.4 GHz without; products of random values alone, out of registers, reach
// 1.75 to 2.0 PFLOP/s).  Measured, bf16: 0.78 us a step where the tiles are one
// round (dx of 4096 x 4096 from 2 x 10240: 510 to 555 us by the card, 1.24 to 1.35
// PFLOP/s), 0.92 us over several rounds of the forward (4096 x 4096 -> 2 x 10240: 585
// us, 1.17 PFLOP/s), matrix cores busy 59 to 67 % of the cycles, LDS reads 22 %, no
// bank conflicts; loads
// that all hit L2 change nothing.  The same loop with the barrier at the end of a
// step is 14 % slower: the next step's operands then arrive with no products left
// to hide them.  Two waves per SIMD is what the sums (128
// registers a lane) leave room for; four waves of 128 x 128 spill.
//
// An operand lies in memory either along K (x, W as used by the forward) or
// across it (the gradients' transposed operands): the latter keep their
// layout in LDS and are transposed by the reads that feed the MFMAs
// (ds_read_b64_tr_b16), so no transposed copy of a weight or of an
// activation is ever written.
#pragma once

#include "proj_rows.hpp"

namespace sgmv {

enum { kAlongK = 0, kAcrossK = 1, kCodes = 2 };

template <int BM_, int BN_, int WM_, int WN_>
struct TileShape {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int NW = WM * WN;                 // waves
    static constexpr int NT = NW * kWave;              // threads
    static constexpr int TM = BM / (16 * WM), TN = BN / (16 * WN);  // MFMA tiles per wave
};

struct TileArgs {
    // One product C = A B^T over K, or the sum of kSegs of the same shapes; `batches`
    // == 2: two such, of a and b from [kSegs z] on -> out[z].
    const void* a[4];
    const void* b[4];
    long long lda, ldb;   // elements between rows (kAlongK) or K (kAcrossK)
    ProjWeight q[2];      // kCodes
    void* out[2];         // [M, N]
    const void* add[2];   // gated: addends [M, N]; else add[0] = bias [N]; or NULL
    void* save[2];        // gated: g and u [M, N], or NULL
    int save_f32;         // these in float32
    int M, N, K;          // gated: N columns of each matrix
    int batches;
    int in_ranges;        // kSegs > 1: the batches are ranges of K of one product
    int range_steps;      // in_ranges, direct loads: steps per range, a multiple of 4
    float* partial;       // in_ranges: their sums, [batches][partial_stride]; or NULL
    long long partial_stride;
    int m_first, n_first;            // row and column (of each matrix) of the first tile
    int tiles_m, tiles_n, tiles;     // of this launch
    int avec, bvec, yvec; // 16-byte pieces of A / B; 4-element pieces of [M, N] arrays
    int kblocks;          // 4-bit: tiles of 128 K
    int act;
};

// Where 16-byte piece p of K row k of an operand kept across K lies in its
// LDS row.  A transposing read takes, per group of 16 lanes, 32 bytes of each
// of four K rows; the 32-byte units of a row are permuted by its K so that the
// 16 rows one read touches fall on different banks.
template <typename DT, int COLS>
struct AcrossLayout {
    static constexpr int kRow = COLS * DT::kBytes;  // bytes of a K row
    static constexpr int kUnits = kRow / 32;
    static constexpr int kRowsPerLoad = 1024 / kRow;
    static constexpr bool kPermute = DT::kBytes == 2;
    __device__ static __forceinline__ int permute(int k) {
        return kPermute ? ((k & 3) | (((k >> 3) & 3) << 2)) & (kUnits - 1) : 0;
    }
};

// Byte offset of 16-byte slot s of stage row r of an operand kept along K:
// slot s holds piece s ^ ((r >> 1) & 3), which spreads the 16 rows an MFMA
// operand read touches over the banks.
__device__ __forceinline__ int along_piece(int r, int s) { return s ^ ((r >> 1) & 3); }

// MFMA operand (16 rows or columns from c0 on) out of a stage.
template <typename DT, int LAYOUT, int COLS>
struct StageReader {
    int off;       // lane's byte offset
    int f;         // AcrossLayout permutation of this lane's rows
    __device__ __forceinline__ StageReader(int c0, int lr, int lg) {
        if constexpr (LAYOUT != kAcrossK) {
            off = (c0 + lr) * 64 + (along_piece(lr, lg) << 4);
            f = 0;
        } else if constexpr (DT::kBytes == 2) {
            using L = AcrossLayout<DT, COLS>;
            off = (lg * 8 + (lr >> 2)) * L::kRow + (lr & 3) * 8;
            f = L::permute(lg * 8 + (lr >> 2)) ^ (c0 >> 4);
        } else {
            off = lg * 4 * (COLS * 4) + (c0 + lr) * 4;
            f = 0;
        }
    }
    __device__ __forceinline__ uint4 operator()(const uint8_t* st, int i) const {
        if constexpr (LAYOUT != kAcrossK) {
            return load16(st + off + i * 1024);
        } else if constexpr (DT::kBytes == 2) {
#if __HIP_DEVICE_COMPILE__
            using L = AcrossLayout<DT, COLS>;
            typedef short v4s __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) v4s lds_v4s;
            typedef __attribute__((address_space(3))) uint8_t lds_u8;
            int u = f;
            asm("" : "+v"(u));  // recomputed per read: kept, the offsets would take a register each
            const uint8_t* p = st + off + ((u ^ i) << 5);
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(lds_u8*)p);
            const v4s hi =
                __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(lds_u8*)(p + 4 * L::kRow));
            const uint2 l = __builtin_bit_cast(uint2, lo), h = __builtin_bit_cast(uint2, hi);
            return make_uint4(l.x, l.y, h.x, h.y);
#else
            return make_uint4(0, 0, 0, 0);
#endif
        } else {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(st + off + i * 64);
            constexpr int r = COLS;  // dwords of a K row
            return make_uint4(p[0], p[r], p[2 * r], p[3 * r]);
        }
    }
};

// A lane's eight codes less their zero point, whole numbers of five bits: exact.
template <typename DT>
__device__ __forceinline__ uint4 plain_codes(uint32_t w, float zb) {
    const uint4 b = codes_biased<DT>(w);
    if constexpr (std::is_same<DT, F16>::value) {
        typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
        const h2_t zz = {(_Float16)zb, (_Float16)zb};
        auto one = [&](uint32_t v) {
            return __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2_t, v) - zz);
        };
        return make_uint4(one(b.x), one(b.y), one(b.z), one(b.w));
    } else {
        return codes_less_zero(b, zb);
    }
}

// kFlushes: scale pairs per feature and tile of 128 K (kCodes), else 1.
//
// 4-bit B: threads unpack a block's codes into the stages, exactly (less their zero
// points), and the products of the steps that share a scale are summed apart; the
// first products of the next such group find that sum done, and scale it into the
// result's.  So nothing is rounded but float32 sums, as in the calls of few rows.  Two
// sums per output leave a wave 64 x 64 outputs, whose operands' LDS reads take as long
// as its products; a scale costs a multiply-add per output (5120 -> 13824, bf16, a
// scale per 128 K: 512 rows 85 us, 2048 rows 333 us, 870 TFLOP/s; per 32 K 125 and 462).
// Scaled weights rounded to the type before the products would fit 256 x 256 tiles, 269
// us for the 2048 rows, and put results off by 2.1e-3 of their size (root mean square,
// bf16) where their own rounding is 1.65e-3.
template <typename DT, typename SH, int AL, int BL, int kSegs, bool kGated, bool kDma, int kFlushes>
__global__ __launch_bounds__(SH::NT, BL == kCodes ? 2 : 1) void tile_kernel(TileArgs g) {
    using T = typename DT::storage;
    using Ops = PieceOps<DT>;
    constexpr int BM = SH::BM, BN = SH::BN, TM = SH::TM, TN = SH::TN, NT = SH::NT, NW = SH::NW;
    constexpr int B = DT::kBytes, PK = Ops::kPK;
    constexpr int KE = 4 * PK;                 // K per step
    static_assert(BL != kCodes || (B == 2 && AL == kAlongK), "codes feed 16-bit tiles along K");
    static_assert(!kGated || TN % 2 == 0, "a gated wave holds both matrices' columns");
    // Four stages of 64 bytes of K for each operand.  They are arrays of their own,
    // and every load names its array: the compiler, which orders LDS accesses
    // after the direct loads into the same array, then needs no wait but ours.
    __shared__ __attribute__((aligned(16))) uint8_t s_a0[BM * 64], s_b0[BN * 64];
    __shared__ __attribute__((aligned(16))) uint8_t s_a1[BM * 64], s_b1[BN * 64];
    __shared__ __attribute__((aligned(16))) uint8_t s_a2[BM * 64], s_b2[BN * 64];
    __shared__ __attribute__((aligned(16))) uint8_t s_a3[BM * 64], s_b3[BN * 64];

    // 4-bit: scales of the stage rows of B, by the first step of their group in a turn
    // of the loop (groups of steps that share a scale: kGroup steps).
    constexpr int kGroup = 4 / kFlushes;
    __shared__ __attribute__((aligned(16))) float s_scale[BL == kCodes ? 8 : 1][BL == kCodes ? BN : 4];
    __shared__ uint8_t s_unread[NW == 8 && kDma ? 256 * NW : 1];  // where prefetches land

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int lr = lane & 15, lg = lane >> 4;

    // Tile of this workgroup.  Workgroup b runs on XCD b % 8: each XCD takes a
    // contiguous range of the tile order, which walks groups of eight tile
    // rows column by column, so that the tiles an XCD holds at one time share
    // their operands in its L2.
    int t = (int)blockIdx.x;
    {
        const int x = t & 7, per = g.tiles >> 3, rest = g.tiles & 7;
        t = x * per + min(x, rest) + (t >> 3);
    }
    const int per_batch = g.tiles_m * g.tiles_n;
    const int z = t / per_batch;
    t -= z * per_batch;
    const int group = t / (8 * g.tiles_n);
    const int in_group = t - group * 8 * g.tiles_n;
    const int rows_here = min(8, g.tiles_m - 8 * group);
    const int row8 = in_group % rows_here;  // tile row within the group
    const int m0 = g.m_first + (8 * group + row8) * BM;
    const int tn = in_group / rows_here;
    // Columns per tile: a gated tile holds BN / 2 of each matrix.
    const int n0 = g.n_first + tn * (kGated ? BN / 2 : BN);
    const int wr0 = (wid / SH::WN) * (16 * TM), wc = wid % SH::WN, wc0 = wc * (16 * TN);
    const int M = g.M, N = g.N, K = g.K;

    // Stage row r of B, gated: waves' column blocks of 16 TN rows, the first
    // half of each from the gate's matrix and the second from the up matrix.
    auto gated_row = [&](int r, int& which) {
        const int blk = r / (16 * TN), in = r % (16 * TN);
        which = in >= 8 * TN;
        return n0 + blk * (8 * TN) + (which ? in - 8 * TN : in);
    };

    // 4-bit weights: unit u of a wave is n-tile wid + u NW of the stage's, a lane holding
    // one packed dword per step.
    constexpr int kUnits = BL == kCodes ? BN / 16 / NW : 1;
    static_assert(BL != kCodes || kUnits * NW * 16 == BN, "whole units per wave");
    struct Codes {
        uint4 w;
        uint32_t meta[kFlushes];
    };
    auto load_codes = [&](int kb, Codes(&c)[kUnits]) {
        if constexpr (BL == kCodes) {
            kb = min(kb, g.kblocks - 1);
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                int which = 0;
                const int first = (wid + u * NW) * 16;
                const int row = kGated ? gated_row(first, which) : n0 + first;
                const long long tile = (long long)min(row >> 4, ((N + 15) >> 4) - 1) * g.kblocks + kb;
                const ProjWeight& q = g.q[which];
                c[u].w = load16((const uint4*)q.w + tile * 64 + lane);
                load_dwords<kFlushes>((const uint32_t*)q.meta + tile * 16 * kFlushes + lr * kFlushes,
                                      c[u].meta);
            }
        }
    };
    auto store_codes = [&](uint8_t* sb, const Codes(&c)[kUnits], int s, int slot) {
        if constexpr (BL == kCodes) {
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                const int first = (wid + u * NW) * 16;
                const uint32_t w = s == 0 ? c[u].w.x : s == 1 ? c[u].w.y : s == 2 ? c[u].w.z : c[u].w.w;
                float sc, zb;
                meta_values<DT>(c[u].meta[s * kFlushes / 4], sc, zb);
                const int unit = tid + u * NT, l = unit & 63, row = (unit >> 6) * 16 + (l & 15);
                store16(sb + row * 64 + (along_piece(row, l >> 4) << 4), plain_codes<DT>(w, zb));
                // By all four lanes that hold it: a branch here would make the compiler wait
                // for every load.
                if (s % kGroup == 0) s_scale[slot][first + lr] = sc;
            }
        }
    };

    acc4_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = acc4_t{0.f, 0.f, 0.f, 0.f};

    const StageReader<DT, AL, BM> rd_a(wr0, lr, lg);
    const StageReader<DT, BL, BN> rd_b(wc0, lr, lg);
    auto fence = [] {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // 4-bit: sums of the group in hand, and the scales of this lane's features (those of
    // its sums' four elements) for the group whose sums are done.
    constexpr int TMC = BL == kCodes ? TM : 1, TNC = BL == kCodes ? TN : 1;
    acc4_t part[TMC][TNC];
    auto scales = [&](int slot, int j) {
        return *reinterpret_cast<const acc4_t*>(&s_scale[slot][wc0 + 16 * j + 4 * lg]);
    };
    auto add_part = [&](int i, int j, const acc4_t& scale) {
        if constexpr (BL == kCodes) {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] += scale[e] * part[i][j][e];
            // Here and not later: left until the result is used, a turn's sums spill.
            asm volatile("" : "+v"(acc[i][j]));
        }
    };
    // 4-bit: products of rows [i0, i1) of a step.  The first step of a group scales the
    // sums of the group before it, whose scales are in slot `done`, into the result's.
    auto code_products = [&](auto i0, auto i1, const uint4(&a)[TM], const uint4(&b)[TN], auto done) {
        constexpr int I0 = decltype(i0)::value, I1 = decltype(i1)::value, D = decltype(done)::value;
        if constexpr (BL == kCodes && D >= 0) {
            constexpr int kHeld = kFlushes == 4 || (kFlushes == 2 && NW == 8) ? 1 : TN;  // as registers allow
            acc4_t sc[TN];
#pragma unroll
            for (int j = 0; j < kHeld; ++j) sc[j] = scales(D, j);
#pragma unroll
            for (int j = 0; j < TN; ++j) {
#pragma unroll
                for (int i = I0; i < I1; ++i) {
                    add_part(i, j, sc[j]);
                    part[i][j] = Ops::mma(b[j], a[i], acc4_t{0.f, 0.f, 0.f, 0.f});
                }
                if (j + kHeld < TN) {
                    fence();
                    sc[j + kHeld] = scales(D, j + kHeld);
                }
            }
        } else if constexpr (BL == kCodes) {
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = I0; i < I1; ++i) part[i][j] = Ops::mma(b[j], a[i], part[i][j]);
        }
    };
    using Row0 = std::integral_constant<int, 0>;
    using RowMid = std::integral_constant<int, TM / 2>;
    using RowEnd = std::integral_constant<int, TM>;
    using NoneDone = std::integral_constant<int, -1>;
    auto finish_parts = [&](int slot) {
        if constexpr (BL == kCodes) {
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const acc4_t sc = scales(slot, j);
#pragma unroll
                for (int i = 0; i < TM; ++i) add_part(i, j, sc);
            }
        }
    };
    if constexpr (BL == kCodes) {
        // The first group finds zeros: sums, and the scales of the slot before it.
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) part[i][j] = acc4_t{0.f, 0.f, 0.f, 0.f};
        for (int r = tid; r < BN; r += NT) s_scale[8 - kGroup][r] = 0.f;
    }
    auto compute = [&](const uint8_t* sa, const uint8_t* sb) {
        uint4 b[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j) b[j] = rd_b(sb, j);
        if constexpr (BL == kCodes) {
            uint4 a[TM];
#pragma unroll
            for (int i = 0; i < TM; ++i) a[i] = rd_a(sa, i);
            code_products(Row0{}, RowEnd{}, a, b, NoneDone{});
        } else {
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const uint4 a = rd_a(sa, i);
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = Ops::mma(b[j], a, acc[i][j]);
            }
        }
    };

    // ---- K through registers, zero filled: four steps from kc on ------------
    // What 16-byte slot e of an operand's stage holds.
    auto guarded = [&](auto layout, auto cols_c, const void* base, long long ld, int r0, int rows,
                       int e, int kc, bool vec) -> uint4 {
        constexpr int L = decltype(layout)::value, COLS = decltype(cols_c)::value;
        const T* p = (const T*)base;
        if constexpr (L == kAlongK) {
            const int row = e >> 2, k = kc + along_piece(row, e & 3) * PK;
            if (r0 + row >= rows) return make_uint4(0, 0, 0, 0);
            return load_piece<DT>(p + (long long)(r0 + row) * ld, k, K, vec);
        } else {
            using LY = AcrossLayout<DT, COLS>;
            const int kr = e * 16 / LY::kRow, slot = (e * 16 % LY::kRow) / 16;
            const int piece = (((slot >> 1) ^ LY::permute(kr)) << 1) | (slot & 1);
            if (kc + kr >= K) return make_uint4(0, 0, 0, 0);
            return load_piece<DT>(p + (long long)(kc + kr) * ld, r0 + piece * PK, rows, vec);
        }
    };
    const int pair0 = kSegs > 1 && g.in_ranges ? 0 : kSegs * z;  // this product's first a and b
    auto slow_steps = [&](int seg, int kc) {
        const int which = pair0 + seg;
        constexpr int kA = BM * 4 / NT, kB = BL == kCodes ? 0 : BN * 4 / NT;
        static_assert(kA * NT == BM * 4 && (BL == kCodes || kB * NT == BN * 4), "whole slots per thread");
        constexpr int kBn = kB > 0 ? kB : 1;
        uint4 ra[4][kA], rb[4][kBn];
        Codes cc[kUnits];
        if constexpr (BL == kCodes) load_codes(kc / 128, cc);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
            for (int u = 0; u < kA; ++u)
                ra[s][u] = guarded(std::integral_constant<int, AL>{}, std::integral_constant<int, BM>{},
                                   g.a[which], g.lda, m0, M, tid + u * NT, kc + s * KE, g.avec);
#pragma unroll
            for (int u = 0; u < kB; ++u) {
                const int e = tid + u * NT;
                if constexpr (kGated) {
                    int w2;
                    const int row = gated_row(e >> 2, w2);
                    const int k = kc + s * KE + along_piece(e >> 2, e & 3) * PK;
                    rb[s][u] = row < N ? load_piece<DT>((const T*)g.b[w2] + (long long)row * g.ldb, k,
                                                        K, g.bvec)
                                       : make_uint4(0, 0, 0, 0);
                } else {
                    rb[s][u] = guarded(std::integral_constant<int, BL>{},
                                       std::integral_constant<int, BN>{}, g.b[which], g.ldb, n0, N,
                                       e, kc + s * KE, g.bvec);
                }
            }
        }
        __syncthreads();  // the stages' last reads are done
        auto put = [&](uint8_t* sa, uint8_t* sb, int s) {
#pragma unroll
            for (int u = 0; u < kA; ++u) store16(sa + (tid + u * NT) * 16, ra[s][u]);
#pragma unroll
            for (int u = 0; u < kB; ++u) store16(sb + (tid + u * NT) * 16, rb[s][u]);
            if constexpr (BL == kCodes) store_codes(sb, cc, s, s);
        };
        put(s_a0, s_b0, 0);
        put(s_a1, s_b1, 1);
        put(s_a2, s_b2, 2);
        put(s_a3, s_b3, 3);
        __syncthreads();
        // A group's sums are done, and scaled, with its last step; steps past K add zeros.
        auto one = [&](const uint8_t* sa, const uint8_t* sb, auto index) {
            constexpr int s = decltype(index)::value;
            if constexpr (BL == kCodes) {
                if constexpr (s % kGroup == 0) {
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int j = 0; j < TN; ++j) part[i][j] = acc4_t{0.f, 0.f, 0.f, 0.f};
                }
            }
            if (kc + s * KE < K) compute(sa, sb);
            if constexpr ((s + 1) % kGroup == 0) finish_parts(s + 1 - kGroup);
        };
        one(s_a0, s_b0, std::integral_constant<int, 0>{});
        one(s_a1, s_b1, std::integral_constant<int, 1>{});
        one(s_a2, s_b2, std::integral_constant<int, 2>{});
        one(s_a3, s_b3, std::integral_constant<int, 3>{});
    };
    if constexpr (!kDma) {
        const int seg_turns = (K + 4 * KE - 1) / (4 * KE);
        int turn = 0, end = kSegs * seg_turns;
        if (kSegs > 1 && g.in_ranges) {
            const int each = (end + g.batches - 1) / g.batches;  // turns per range
            turn = z * each;
            end = min(end, turn + each);
        }
        for (; turn < end; ++turn) {
            const int seg = kSegs > 1 ? turn / seg_turns : 0;
            slow_steps(seg, (turn - seg * seg_turns) * 4 * KE);
        }
    }

    // ---- K by direct loads ----------------------------------------------------
    if constexpr (kDma) {
        // Steps per segment, and in all: whole turns of the loops below.
        constexpr int kTurn = BL == kCodes ? 8 : 4;
        const int seg_steps = (K + KE - 1) / KE;
        int nsteps = (kSegs * seg_steps + kTurn - 1) / kTurn * kTurn;
        int step0 = 0;  // first step of this workgroup's range
        if (kSegs > 1 && g.in_ranges) {
            step0 = z * g.range_steps;
            nsteps = min(nsteps - step0, g.range_steps);
        }
        {
            // A load brings 1 KB: 16 stage rows of an operand along K, or the K rows
            // that fit.  Wave w takes loads w, w + NW, ... of A and of B.
            constexpr int kLA = BM / 16 / NW, kLB = BL == kCodes ? 0 : BN / 16 / NW;
            constexpr int kLoads = kLA + kLB, kLBn = kLB > 0 ? kLB : 1;
            static_assert(kLA * NW * 16 == BM && (BL == kCodes || kLB * NW * 16 == BN), "whole loads per wave");
            static_assert(2 * kLoads < 64, "the wait count fits vmcnt");
            constexpr int kWaitSteps = (2 * kLoads & 15) | ((2 * kLoads >> 4) << 14) | 0x0070;
            using lds_t = __attribute__((address_space(3))) void;
            const int which = pair0;
            // Lane's byte offset in load `load` of an operand from its tile's first row
            // (along K) or first column (across K), and its first K within a step; past
            // the end of the rows (columns) it reads the last.
            auto source = [&](auto layout, auto cols_c, long long ld, int r0, int rows, int load,
                              int& k) {
                if constexpr (decltype(layout)::value == kAlongK) {
                    const int row = load * 16 + (lane >> 2);
                    k = along_piece(row, lane & 3) * PK;
                    return (uint32_t)(min(row, rows - 1 - r0) * ld + k) * B;
                } else {
                    using LY = AcrossLayout<DT, decltype(cols_c)::value>;
                    const int byte = lane * 16;
                    k = load * LY::kRowsPerLoad + byte / LY::kRow;
                    const int slot = (byte % LY::kRow) / 16;
                    const int piece = (((slot >> 1) ^ LY::permute(k)) << 1) | (slot & 1);
                    return (uint32_t)(k * ld + min(piece * PK, rows - PK - r0)) * B;
                }
            };
            auto corner = [&](auto layout, const void* base, long long ld, int r0) {
                return (const char*)base + (decltype(layout)::value == kAlongK ? r0 * ld : r0) * B;
            };
            using AL_t = std::integral_constant<int, AL>;
            using BL_t = std::integral_constant<int, BL>;
            uint32_t off_a[kLA], off_b[kLBn];
            int ka[kLA], kb[kLBn];
            const char *base_a, *base_b[kLBn];  // uniform over the wave
            base_a = corner(AL_t{}, g.a[which], g.lda, m0);
#pragma unroll
            for (int u = 0; u < kLA; ++u)
                off_a[u] = source(AL_t{}, std::integral_constant<int, BM>{}, g.lda, m0, M, wid + u * NW, ka[u]);
#pragma unroll
            for (int u = 0; u < kLB; ++u) {
                const int load = wid + u * NW;
                if constexpr (kGated) {
                    // A load's 16 stage rows lie in one matrix.  Its rows may lie past
                    // N altogether, so the corner is the first row that does not.
                    int w2;
                    const int row = gated_row(load * 16, w2), at = min(row, N - 1);
                    base_b[u] = corner(BL_t{}, g.b[w2], g.ldb, at);
                    const int r = load * 16 + (lane >> 2);
                    kb[u] = along_piece(r, lane & 3) * PK;
                    off_b[u] = (uint32_t)(min(lane >> 2, N - 1 - at) * g.ldb + kb[u]) * B;
                } else {
                    base_b[u] = corner(BL_t{}, g.b[which], g.ldb, n0);
                    off_b[u] = source(BL_t{}, std::integral_constant<int, BN>{}, g.ldb, n0, N, load, kb[u]);
                }
            }
            const long long stride_a = AL == kAlongK ? 64 : KE * g.lda * B;  // bytes per step
            const long long stride_b = BL == kAcrossK ? KE * g.ldb * B : 64;
            // From the first segment's operands to the others'.
            struct Jumps {
                long long to[kSegs];
            };
            Jumps jump_a, jump_b;
#pragma unroll
            for (int s = 0; s < kSegs; ++s) {
                jump_a.to[s] = (const char*)g.a[which + s] - (const char*)g.a[which];
                jump_b.to[s] = (const char*)g.b[which + s] - (const char*)g.b[which];
            }
            // A step within its segment, and that segment (past the last step, the last).
            auto segment = [&](int& step) {
                int seg = 0;
#pragma unroll
                for (int s = 1; s < kSegs; ++s) seg += step >= s * seg_steps;
                step -= seg * seg_steps;
                return seg;
            };
            auto jump = [](const Jumps& j, int seg) {
                long long at = 0;
#pragma unroll
                for (int s = 1; s < kSegs; ++s)
                    if (seg >= s) at = j.to[s];
                return at;
            };
            // Buffer loads: the step's address is the (scalar) base, a lane adds its
            // 32-bit offset, and a lane past the end of K takes an offset past the
            // buffer's range, for which the load returns zeros.
            auto load_lds = [](const char* base, int offset, uint8_t* to) {
#if __HIP_DEVICE_COMPILE__  // the host pass does not know buffer resources
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, 0x7FFFFFFF, 0x00020000),
                    (lds_t*)to, 16, offset, 0, 0, 0);
#endif
            };
            auto load_lds4 = [](const char* base, int offset, uint8_t* to) {
#if __HIP_DEVICE_COMPILE__
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, 0x7FFFFFFF, 0x00020000),
                    (lds_t*)to, 4, offset, 0, 0, 0);
#endif
            };
            // Load u of a step (A's, then B's).
            auto issue1 = [&](uint8_t* sa, uint8_t* sb, int step, int u) {
                step += step0;
                const int seg = segment(step);
                const int k_left = K - step * KE;  // not positive past the last step
                if (u < kLA) {
                    const int o = ka[u < kLA ? u : 0] < k_left ? (int)off_a[u < kLA ? u : 0] : -16;
                    load_lds(base_a + (jump(jump_a, seg) + step * stride_a), o, sa + (wid + u * NW) * 1024);
                } else {
                    const int v = u >= kLA ? u - kLA : 0;
                    const int o = kb[v] < k_left ? (int)off_b[v] : -16;
                    load_lds(base_b[v] + (jump(jump_b, seg) + step * stride_b), o, sb + (wid + v * NW) * 1024);
                }
            };
            // L2 prefetch, kAhead steps before a step is loaded, of 128-byte lines that
            // hold two steps: one 4-byte load per line, into LDS that nobody reads.
            // The tiles that an XCD holds at one time are eight tile rows by four tile
            // columns (see the tile order above), so each workgroup fetches a quarter
            // of its A lines and an eighth of its B lines, and the direct loads find
            // all of them in L2.  Waves 0-3 fetch A's share, waves 4-7 B's.
            constexpr int kAhead = 6;
            constexpr bool kPrefetch = NW == 8;
            const char* pf_base = base_a;
            long long pf_stride = stride_a;
            Jumps pf_jump = jump_a;
            int pf_off = -16, pf_k = 0;
            if constexpr (kPrefetch) {
                // Line `id` of an operand's tile of COLS rows (columns), two steps being
                // COLS lines: row id along K; across K, line id % (COLS / 64) of K row
                // id / (COLS / 64) (float32: its first half; a line holds one step then).
                auto line = [&](auto layout, auto cols_c, long long ld, int id, int rows_left) {
                    if constexpr (decltype(layout)::value == kAlongK) {
                        return (int)(min(id, rows_left - 1) * ld) * B;
                    } else {
                        constexpr int kLines = decltype(cols_c)::value / 64;
                        pf_k = id / kLines;
                        return (int)(pf_k * ld + min(id % kLines * (128 / B), rows_left - PK)) * B;
                    }
                };
                if (wid < 4) {
                    if (lane < BM / 16)
                        pf_off = line(AL_t{}, std::integral_constant<int, BM>{}, g.lda,
                                      (tn & 3) * (BM / 4) + wid * (BM / 16) + lane, M - m0);
                } else if constexpr (BL != kCodes) {
                    const int first = row8 * (BN / 8) + (wid - 4) * (BN / 32);
                    pf_base = base_b[0];
                    pf_stride = stride_b;
                    pf_jump = jump_b;
                    if constexpr (kGated) {  // 8 stage rows lie in one matrix
                        int w2;
                        const int row = gated_row(first, w2), at = min(row, N - 1);
                        pf_base = corner(BL_t{}, g.b[w2], g.ldb, at);
                        if (lane < BN / 32) pf_off = (int)(min(lane, N - 1 - at) * g.ldb) * B;
                    } else if (lane < BN / 32) {
                        pf_off = line(BL_t{}, std::integral_constant<int, BN>{}, g.ldb, first + lane, N - n0);
                    }
                }
            }
            auto prefetch = [&](int step) {
                step += step0;
                const long long at = jump(pf_jump, segment(step));
                const int o = pf_k < K - step * KE ? pf_off : -16;
                load_lds4(pf_base + (at + step * pf_stride), o, s_unread + 256 * wid);
            };
            auto issue = [&](uint8_t* sa, uint8_t* sb, int step) {
#pragma unroll
                for (int u = 0; u < kLoads; ++u) issue1(sa, sb, step, u);
            };
            // Packed codes of two K blocks, the one being unpacked and the one being loaded.
            Codes ca[kUnits], cb[kUnits];
            // 4-bit: their first two blocks.
            if constexpr (BL == kCodes) {
                load_codes(0, ca);
                load_codes(1, cb);
                fence();
            }
            issue(s_a0, s_b0, 0);
            issue(s_a1, s_b1, 1);
            issue(s_a2, s_b2, 2);
            if constexpr (kPrefetch) prefetch(kAhead - 2);
            if constexpr (BL == kCodes) {
                store_codes(s_b0, ca, 0, 0);
                store_codes(s_b1, ca, 1, 1);
            }
            // Step c multiplies stage c % 4.  Its B operands and the first half of its A
            // operands (of 4-bit B, whose codes need the registers, one) are in registers
            // when it begins (they were read in step c - 1); the other A operands are read
            // at its start, behind the first products. In its middle, with half of its
            // products issued, comes the step's one barrier: this wave's own loads of step c
            // + 1 have landed (only what was issued after them may be in flight) and so has
            // every other wave's; and every wave is past its reads of stage (c - 1) % 4,
            // which takes step c + 3. The next step's operands are then read behind the
            // second half of the products, each A operand into the registers of one that the
            // first half has used, so that the matrix cores have work on both sides of the
            // barrier.  Waves in their second half go first (not with 4-bit B, where it is
            // no faster): their products are what the barrier of the next step waits for (dx
            // of 4096 x 4096 from 2 x 10240, bf16, the three in turn on one card: 549 to 559
            // us, 578 without, and 550 with one A operand read ahead instead of half).
            constexpr int kAfter = kLoads + (kPrefetch ? 1 : 0);
            // 4-bit: the next block's codes but one are asked for at the start of the third step
            // of four, which leaves them in flight as long as the loads into the stages; until
            // the fourth step's barrier they are among what was issued after.
            constexpr int kCodeLoads = BL == kCodes ? 2 * kUnits : 0;
            static_assert(kAfter + kCodeLoads < 64, "the wait count fits vmcnt");
            constexpr int kEarly = BL == kCodes ? 1 : TM / 2;
            uint4 a[TM], b[2][TN];  // b by parity of the step
            auto step = [&](const uint8_t* sa, const uint8_t* next_a, const uint8_t* next_b,
                            uint8_t* ahead_a, uint8_t* ahead_b, uint8_t* codes_b, int c, auto index,
                            Codes(&cur)[kUnits], const Codes(&nxt)[kUnits]) {
                constexpr int in_turn = decltype(index)::value;  // c % kTurn
                constexpr int s = in_turn % 4;
                constexpr int X = s & 1, Y = X ^ 1;
                // 4-bit: where the scales of the group that ends with the step before are.
                using Done = std::integral_constant<int, s % kGroup == 0 ? (in_turn + 8 - kGroup) % 8 : -1>;
                fence();
                if constexpr (BL == kCodes && s == 2) load_codes(c / 4 + 2, cur);
                fence();
#pragma unroll
                for (int i = kEarly; i < TM; ++i) a[i] = rd_a(sa, i);
                fence();
                if constexpr (BL == kCodes) {
                    code_products(Row0{}, RowMid{}, a, b[X], Done{});
                } else {
#pragma unroll
                    for (int i = 0; i < TM / 2; ++i)
#pragma unroll
                        for (int j = 0; j < TN; ++j) acc[i][j] = Ops::mma(b[X][j], a[i], acc[i][j]);
                }
                fence();
                constexpr int kFlying = kAfter + (s >= 2 ? kCodeLoads : 0);
                __builtin_amdgcn_s_waitcnt((kFlying & 15) | ((kFlying >> 4) << 14) |
                                           (BL == kCodes ? 0x0070 : 0x0F70));
                __builtin_amdgcn_s_barrier();
                fence();
#pragma unroll
                for (int j = 0; j < TN; ++j) b[Y][j] = rd_b(next_b, j);
#pragma unroll
                for (int i = 0; i < kEarly; ++i) a[i] = rd_a(next_a, i);
                if constexpr (BL != kCodes) __builtin_amdgcn_s_setprio(1);
                fence();
                if constexpr (BL == kCodes) {
                    code_products(RowMid{}, RowEnd{}, a, b[X], Done{});
                    fence();
                    issue(ahead_a, ahead_b, c + 3);
                    fence();
                } else {
#pragma unroll
                    for (int i = TM / 2; i < TM; ++i) {
#pragma unroll
                        for (int j = 0; j < TN; ++j) acc[i][j] = Ops::mma(b[X][j], a[i], acc[i][j]);
#pragma unroll
                        for (int u = 2 * kLoads * (i - TM / 2) / TM; u < 2 * kLoads * (i + 1 - TM / 2) / TM; ++u) {
                            fence();
                            issue1(ahead_a, ahead_b, c + 3, u);
                            fence();
                        }
                    }
                }
                if constexpr (BL != kCodes) __builtin_amdgcn_s_setprio(0);
                if constexpr (kPrefetch && s % 2 == 0) prefetch(c + kAhead);
                if constexpr (BL == kCodes) {  // step c + 2, read after the next barrier
                    if (s < 2) store_codes(codes_b, cur, s + 2, in_turn + 2);
                    else store_codes(codes_b, nxt, s - 2, (in_turn + 2) % 8);
                }
                fence();
            };
            auto four = [&](int c, auto first, Codes(&cur)[kUnits], Codes(&nxt)[kUnits]) {
                constexpr int h = decltype(first)::value;  // c % kTurn
                step(s_a0, s_a1, s_b1, s_a3, s_b3, s_b2, c, std::integral_constant<int, h>{}, cur, nxt);
                step(s_a1, s_a2, s_b2, s_a0, s_b0, s_b3, c + 1, std::integral_constant<int, h + 1>{}, cur, nxt);
                step(s_a2, s_a3, s_b3, s_a1, s_b1, s_b0, c + 2, std::integral_constant<int, h + 2>{}, cur, nxt);
                step(s_a3, s_a0, s_b0, s_a2, s_b2, s_b1, c + 3, std::integral_constant<int, h + 3>{}, cur, nxt);
            };
            fence();
            __builtin_amdgcn_s_waitcnt(kWaitSteps);  // step 0 has landed
            __builtin_amdgcn_s_barrier();
            fence();
#pragma unroll
            for (int j = 0; j < TN; ++j) b[0][j] = rd_b(s_b0, j);
#pragma unroll
            for (int i = 0; i < kEarly; ++i) a[i] = rd_a(s_a0, i);
            for (int c = 0; c < nsteps; c += kTurn) {
                four(c, std::integral_constant<int, 0>{}, ca, cb);
                if constexpr (kTurn == 8) four(c + 4, std::integral_constant<int, 4>{}, cb, ca);
            }
            __builtin_amdgcn_s_waitcnt(0x0070);  // no load is left in flight to the stages
            finish_parts(8 - kGroup);
        }
    }

    // ---- epilogue -------------------------------------------------------------
    T* out = (T*)g.out[kSegs > 1 && g.in_ranges ? 0 : z];
    constexpr int TNO = kGated ? TN / 2 : TN;
    const int nw = n0 + wc * (16 * TNO) + 4 * lg;  // this lane's first columns
    float bias[kGated ? 1 : TNO][4] = {};
    if constexpr (!kGated) {
        if (g.add[0]) {
#pragma unroll
            for (int j = 0; j < TNO; ++j)
                if (nw + 16 * j < N)
                    load4f<DT>((const T*)g.add[0] + nw + 16 * j, N - nw - 16 * j, g.yvec, bias[j]);
        }
    }
    // Row by row: a store instruction writes 32 bytes of each of 16 rows, and the
    // stores that complete its lines come next.  Column by column, L2 passed
    // lines on half written (both 10240 x 4096 weights' gradients: 397 MB written
    // for 168; of 11008 rows, 620 us against 578).
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int m = m0 + wr0 + 16 * i + lr;
        if (m >= M) continue;
#pragma unroll
        for (int j = 0; j < TNO; ++j) {
            const int n = nw + 16 * j, left = N - n;
            if (n >= N) continue;
            const long long at = (long long)m * N + n;
            float o[4];
            if constexpr (kGated) {
                float v[2][4];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[q][c] = acc[i][q * TNO + j][c];
                    if (g.add[q]) {
                        float b[4];
                        load4f<DT>((const T*)g.add[q] + at, left, g.yvec, b);
#pragma unroll
                        for (int c = 0; c < 4; ++c) v[q][c] += b[c];
                    }
                    if (g.save[q] && g.save_f32) {
                        store4f<F32>((float*)g.save[q] + at, left, g.yvec, v[q]);
                    } else if (g.save[q]) {
                        float k[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) k[c] = kept<DT>(v[q][c]);
                        store4f<DT>((T*)g.save[q] + at, left, g.yvec, k);
                    }
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) o[c] = act_value(g.act, v[0][c]) * v[1][c];
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) o[c] = acc[i][j][c] + bias[j][c];
            }
            if (kSegs > 1 && g.partial)
                store4f<F32>(g.partial + z * g.partial_stride + at, left, N % 4 == 0, o);
            else
                store4f<DT>(out + at, left, g.yvec, o);
        }
    }
}

// ---------------------------------------------------------------------------
// dg = dh u a'(g), du = dh a(g), element by element (three reads, two
// writes).  n is the element count; `vec`: every array is 16-byte aligned.
// Bound: HBM; 4096 x 11008 bf16, 451 MB: 87 us, 5.2 TB/s.
// kFull: g and u come in float32, and what dg and du lose by their rounding goes on to
// the matrix products too, as second parts (lo), 16 and 22 bits in all: gradients are
// off by their own rounding, 0.0017 of their size (bf16, root mean square over a
// training step's).  4096 x 11008 bf16 moves 811 MB then, 180 us, and the products take
// twice as long.  Without it, where the caller chooses that, g, u, dg and du are held in
// the activations' type: 0.0031.
// ---------------------------------------------------------------------------
template <typename DT, bool kFull>
__global__ __launch_bounds__(256) void gated_grad_kernel(
    typename DT::storage* __restrict__ dg, typename DT::storage* __restrict__ du,
    typename DT::storage* __restrict__ dg_lo, typename DT::storage* __restrict__ du_lo,
    const typename DT::storage* __restrict__ dh, const void* __restrict__ gs,
    const void* __restrict__ us, long long n, int act, int vec) {
    using KT = std::conditional_t<kFull, F32, DT>;  // of g and u
    using K = typename KT::storage;
    constexpr int V = DT::kVec;
    const K* const gk = (const K*)gs;
    const K* const uk = (const K*)us;
    auto unpack = [](const K* p, float* f) {
#pragma unroll
        for (int i = 0; i < V; i += KT::kVec) KT::unpack(load16(p + i), f + i);
    };
    const long long stride = (long long)gridDim.x * 256 * V;
    for (long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * V; i < n; i += stride) {
        float h[V], a[V], b[V];
        const bool whole = vec && i + V <= n;
        if (whole) {
            DT::unpack(load16(dh + i), h);
            unpack(gk + i, a);
            unpack(uk + i, b);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const bool in = i + e < n;
                h[e] = in ? DT::load1(dh + i + e) : 0.f;
                a[e] = in ? KT::load1(gk + i + e) : 0.f;
                b[e] = in ? KT::load1(uk + i + e) : 0.f;
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float v, d;
            act_value_grad(act, a[e], v, d);
            a[e] = h[e] * b[e] * d;
            b[e] = h[e] * v;
        }
        auto put = [&](typename DT::storage* hi, typename DT::storage* lo, const float* f) {
            if (whole) {
                store16(hi + i, DT::pack(f));
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (i + e < n) hi[i + e] = DT::from_float(f[e]);
            }
            if constexpr (kFull) {
                float r[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const typename DT::storage one = DT::from_float(f[e]);
                    const float rounded = DT::load1(&one);
                    // Past the type's range (and for NaN) the first part says it all.
                    r[e] = __builtin_isfinite(rounded) ? f[e] - rounded : 0.f;
                }
                if (whole) {
                    store16(lo + i, DT::pack(r));
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (i + e < n) lo[i + e] = DT::from_float(r[e]);
                }
            }
        };
        put(dg, dg_lo, a);
        put(du, du_lo, b);
    }
}

// ---------------------------------------------------------------------------
// y = the sum of `count` arrays of n float32 sums, in their order, rounded
// once.  `stride` floats apart, a multiple of 4, each 16-byte aligned; `vec`: y
// is too.  The sums were written just before and are mostly read from the
// caches.
// ---------------------------------------------------------------------------
template <typename DT>
__global__ __launch_bounds__(256) void join_kernel(typename DT::storage* __restrict__ y,
                                                   const float* __restrict__ parts, int count,
                                                   long long stride, long long n, int vec) {
    const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < count; ++c) {
        float v[4];
        F32::unpack(load16(parts + c * stride + i), v);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += v[e];
    }
    store4f<DT>(y + i, (int)min(n - i, 4ll), vec, sum);
}

}  // namespace sgmv
