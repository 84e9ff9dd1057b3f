// kv_cache.hpp -- writing K and V into the quantized cache by slots, and reading
// them back (format and layout: kv_format.hpp).
//
// Bound: HBM at prompt sizes (16-bit rows in, codes out, or the reverse), the
// launch at decode sizes: 8000 rows of 8 heads of 128, float16, 4 bits, written in 13 us and read in 11 (42 MB
// either way: 8 at a copy's rate), 48 rows in 5 and 6.  A workgroup takes RT rows of one head, of K or of V; 8
// elements a lane, the group's largest magnitude by lane moves.  K rows go out as they
// are.  V lies with tokens innermost, so its codes pass through LDS: rows whose slots
// follow one another fill whole 16-token lines (16-byte stores, consecutive lines
// adjacent) or quarters of them, lone tokens go out byte by byte.
#pragma once

#include "kv_format.hpp"
#include "sgmv_device.hpp"

namespace sgmv {

constexpr int kKvThreads = 256;

struct KvArgs {
    uint8_t *codes[2], *scales[2];      // of K and V
    const void* in[2];                  // write
    void* out[2];                       // read
    long long row[2], head[2];          // strides of in or out, in elements
    const void* slots;
    int wide_slots;                     // int64
    long long num_slots;                // pages x page_size, below 2^35
    int page_size, rows, heads, D;
    int lo, hi;                         // exponents allowed
    int vec;                            // rows take 16-byte accesses
};

// Codes of 8 floats at scale 2^e, whose magnitudes are at most M 2^e: 8 bytes or 4.
template <int BITS>
__device__ __forceinline__ uint2 kv_encode(const float* f, float scale) {
    typedef short s2_t __attribute__((ext_vector_type(2)));
    if constexpr (BITS == 8) {
        s2_t a = {0, 0}, b = {0, 0};
        a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, f[0], f[1], scale, false);
        a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, f[2], f[3], scale, true);
        b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, f[4], f[5], scale, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, f[6], f[7], scale, true);
        return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
    } else {
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[0], f[1], scale, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2], f[3], scale, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4], f[5], scale, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[6], f[7], scale, 3);
        return make_uint2(w, 0);
    }
}

template <int BITS>
__device__ __forceinline__ void kv_decode(uint2 c, float scale, float* f) {
    typedef float f2_t __attribute__((ext_vector_type(2)));
    f2_t v[4];
    if constexpr (BITS == 8) {
        v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.x, scale, false);
        v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.x, scale, true);
        v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.y, scale, false);
        v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.y, scale, true);
    } else {
        v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, scale, 0);
        v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, scale, 1);
        v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, scale, 2);
        v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, scale, 3);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = v[i].x;
        f[2 * i + 1] = v[i].y;
    }
}

// Scale byte as the float 2^(b - 127); 255 gives an infinity, which the conversions
// take for NaN.
__device__ __forceinline__ float kv_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// 4-bit codes of V: a token's 8 codes in the low halves of 8 bytes.
__device__ __forceinline__ uint2 spread_nibbles(uint32_t w) {
    auto four = [](uint32_t x) {
        x = (x | (x << 8)) & 0x00FF00FFu;
        return (x | (x << 4)) & 0x0F0F0F0Fu;
    };
    return make_uint2(four(w & 0xFFFFu), four(w >> 16));
}
// ... and back: the halves at `shift` (0 or 4) of 8 bytes as 8 codes.
__device__ __forceinline__ uint32_t gather_nibbles(uint2 b, int shift) {
    auto four = [&](uint32_t x) {
        x = (x >> shift) & 0x0F0F0F0Fu;
        x = (x | (x >> 4)) & 0x00FF00FFu;
        return (x | (x >> 8)) & 0xFFFFu;
    };
    return four(b.x) | (four(b.y) << 16);
}

// Sizes of a kernel: P the padded head, RT its rows.
template <int BITS, int P, int RT>
struct KvTile {
    static constexpr int kBytes = P * BITS / 8;       // of a token's codes; lines of V
    static constexpr int kGroups = BITS == 8 ? 1 : P / 32;
    static constexpr int kUnits = P / 8;              // of 8 elements
    static constexpr int kLanes = kUnits <= 8 ? 8 : kUnits <= 16 ? 16 : 32;  // of a row
    static constexpr int kPass = kKvThreads / kLanes; // rows at once
    static constexpr int kPiece = BITS;               // bytes of a unit's codes: 8 or 4
};

// Places of the tile's rows into LDS (-1: none), and the order in which V's lines are
// accessed: entries (row, n) of n = 16 or 4 rows whose slots follow one another from a
// multiple of n, or of one row.  Returns after a barrier.
template <int RT>
__device__ __forceinline__ int kv_slots(const KvArgs& a, int row0, long long* s_place, int* s_ops, int* s_count) {
    static_assert(RT <= kWave, "a wave looks at all rows");
    if (threadIdx.x < kWave) {
        const int i = threadIdx.x;
        long long s = -1;
        if (i < RT && row0 + i < a.rows) {
            s = a.wide_slots ? ((const long long*)a.slots)[row0 + i] : (long long)((const int*)a.slots)[row0 + i];
            if (s < 0 || s >= a.num_slots) s = -1;
        }
        if (i < RT) {
            // block of head 0, counted over pages and heads, and the token in it
            const uint32_t b = (uint32_t)(s >> 4), per = (uint32_t)a.page_size >> 4;
            const uint32_t page = s < 0 ? 0 : b / per;
            s_place[i] = s < 0 ? -1 : (((long long)page * a.heads * per + (b - page * per)) << 4) | (s & 15);
        }
        const long long next = __shfl(s, i + 1 < kWave ? i + 1 : i);
        // bit i: row i + 1 has the next slot
        const uint64_t follows = __ballot(s >= 0 && i + 1 < RT && next == s + 1);
        const bool h16 = s >= 0 && (s & 15) == 0 && ((follows >> i) & 0x7FFF) == 0x7FFF;
        uint64_t in16 = __ballot(h16);
        in16 |= in16 << 1;
        in16 |= in16 << 2;
        in16 |= in16 << 4;
        in16 |= in16 << 8;
        const bool rest = s >= 0 && !((in16 >> i) & 1);
        const bool h4 = rest && (s & 3) == 0 && ((follows >> i) & 7) == 7;
        uint64_t in4 = __ballot(h4);
        in4 |= in4 << 1;
        in4 |= in4 << 2;
        const bool h1 = rest && !((in4 >> i) & 1);
        const uint64_t starts = __ballot(h16 || h4 || h1);
        if (h16 || h4 || h1)
            s_ops[__popcll(starts & ((1ull << i) - 1))] = i | (h16 ? 16 : h4 ? 4 : 1) << 8;
        if (i == 0) *s_count = __popcll(starts);
    }
    __syncthreads();
    return *s_count;
}

struct KvPlace {
    long long block;  // of 16 tokens, counted over pages and heads
    int token;        // in it
};
__device__ __forceinline__ KvPlace kv_place(const KvArgs& a, long long place, int head) {
    return {(place >> 4) + (long long)head * (a.page_size >> 4), (int)(place & 15)};
}

// The 8 elements from 8 u on of a row of D; zeros past D.
template <typename DT>
__device__ __forceinline__ void kv_load8(const typename DT::storage* p, int at, int D, bool vec, float* f) {
    if (vec && at + 8 <= D) {
        DT::unpack(load16(p + at), f);
        if constexpr (DT::kBytes == 4) DT::unpack(load16(p + at + 4), f + 4);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = at + i < D ? DT::load1(p + at + i) : 0.f;
}
template <typename DT>
__device__ __forceinline__ void kv_store8(typename DT::storage* p, int at, int D, bool vec, const float* f) {
    if (vec && at + 8 <= D) {
        store16(p + at, DT::pack(f));
        if constexpr (DT::kBytes == 4) store16(p + at + 4, DT::pack(f + 4));
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (at + i < D) p[at + i] = DT::from_float(f[i]);
}

// Largest over the lanes of a group (4: 32 elements; else all lanes of a row).
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#pragma unroll
    for (int m = 1; m < LANES; m *= 2) {
        const uint32_t o = (uint32_t)__shfl_xor((int)v, m);
        v = v > o ? v : o;
    }
    return v;
}

// grid (row tiles, heads, 2): z = 0 writes K, 1 writes V.
template <typename DT, int BITS, int P, int RT>
__global__ __launch_bounds__(kKvThreads) void kv_write_kernel(KvArgs a) {
    using Tile = KvTile<BITS, P, RT>;
    using T = typename DT::storage;
    __shared__ long long s_place[RT];
    __shared__ int s_ops[RT], s_count;
    __shared__ __align__(16) uint8_t s_codes[RT * Tile::kBytes];
    const int row0 = blockIdx.x * RT, head = blockIdx.y, which = blockIdx.z;
    const int ops = kv_slots<RT>(a, row0, s_place, s_ops, &s_count);
    const int lane = threadIdx.x & (Tile::kLanes - 1);
    const T* in = (const T*)a.in[which] + (long long)head * a.head[which];
    for (int i = threadIdx.x / Tile::kLanes; i < RT; i += Tile::kPass) {
        const long long place = s_place[i];
        const bool held = place >= 0;  // the same for all lanes of a row
        float f[8] = {};
        if (held && lane < Tile::kUnits)
            kv_load8<DT>(in + (long long)(row0 + i) * a.row[which], lane * 8, a.D, a.vec, f);
        uint32_t most = 0;  // magnitudes' bits order like the magnitudes; NaN and infinity above all
#pragma unroll
        for (int k = 0; k < 8; ++k) most = max(most, __float_as_uint(f[k]) & 0x7FFFFFFFu);
        if constexpr (BITS == 4) most = lanes_max<4>(most);
        const uint32_t head_most = BITS == 4 ? lanes_max<Tile::kLanes>(most) : (most = lanes_max<Tile::kLanes>(most));
        // least e with most <= 1.75 2^8 2^e, or 1.5 2^2 2^e
        constexpr uint32_t kBump = BITS == 8 ? 0x1FFFFF : 0x3FFFFF;
        constexpr float kMost = BITS == 8 ? 448.f : 6.f;
        const bool finite = head_most < 0x7F800000u;  // of all the head
        int e = (int)((most + kBump) >> 23) - 127 - (BITS == 8 ? 8 : 2);
        e = min(max(e, a.lo), a.hi);
        const float scale = __uint_as_float((uint32_t)(e + 127) << 23);
        const float limit = kMost * scale;
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = finite ? __builtin_amdgcn_fmed3f(f[k], -limit, limit) : 0.f;
        uint2 c = kv_encode<BITS>(f, scale);
        const uint8_t byte = finite ? (uint8_t)(e + 127) : (uint8_t)kKvNaN;
        const KvPlace p = kv_place(a, held ? place : 0, head);
        if (held && lane < Tile::kUnits && (BITS == 8 ? lane == 0 : (lane & 3) == 0))
            a.scales[which][(p.block * Tile::kGroups + (BITS == 8 ? 0 : lane / 4)) * 16 + p.token] = byte;
        if (which == 0) {
            if (held && lane < Tile::kUnits) {
                uint8_t* out = a.codes[0] + (p.block * 16 + p.token) * Tile::kBytes + lane * Tile::kPiece;
                if constexpr (BITS == 8) *reinterpret_cast<uint2*>(out) = c;
                else *reinterpret_cast<uint32_t*>(out) = c.x;
            }
        } else if constexpr (BITS == 8) {
            if (lane < Tile::kUnits) *reinterpret_cast<uint2*>(s_codes + i * Tile::kBytes + lane * 8) = c;
        } else {
            // Elements 32 g + 8 q + j and 16 further share a byte: lanes 4 g + q and 4 g + q + 2.
            const uint32_t other = (uint32_t)__shfl_xor((int)c.x, 2);
            const uint2 low = spread_nibbles(c.x), high = spread_nibbles(other);
            if (lane < Tile::kUnits && (lane & 2) == 0)
                *reinterpret_cast<uint2*>(s_codes + i * Tile::kBytes + (lane / 4) * 16 + (lane & 1) * 8) =
                    make_uint2(low.x | high.x << 4, low.y | high.y << 4);
        }
    }
    if (which == 0) return;
    __syncthreads();
    for (int w = threadIdx.x; w < ops * Tile::kBytes; w += kKvThreads) {
        const int op = s_ops[w / Tile::kBytes], line = w % Tile::kBytes;
        const int i = op & 255, n = op >> 8;
        const KvPlace p = kv_place(a, s_place[i], head);
        uint8_t* out = a.codes[1] + (p.block * Tile::kBytes + line) * 16 + p.token;
        const uint8_t* src = s_codes + i * Tile::kBytes + line;
        auto four = [&](int r) {
            return (uint32_t)src[r * Tile::kBytes] | (uint32_t)src[(r + 1) * Tile::kBytes] << 8 |
                   (uint32_t)src[(r + 2) * Tile::kBytes] << 16 | (uint32_t)src[(r + 3) * Tile::kBytes] << 24;
        };
        if (n == 16) store16(out, make_uint4(four(0), four(4), four(8), four(12)));
        else if (n == 4) *reinterpret_cast<uint32_t*>(out) = four(0);
        else *out = *src;
    }
}

// The same grid; rows without a slot read as zeros.
template <typename DT, int BITS, int P, int RT>
__global__ __launch_bounds__(kKvThreads) void kv_read_kernel(KvArgs a) {
    using Tile = KvTile<BITS, P, RT>;
    using T = typename DT::storage;
    __shared__ long long s_place[RT];
    __shared__ int s_ops[RT], s_count;
    __shared__ __align__(16) uint8_t s_codes[RT * Tile::kBytes];
    const int row0 = blockIdx.x * RT, head = blockIdx.y, which = blockIdx.z;
    const int ops = kv_slots<RT>(a, row0, s_place, s_ops, &s_count);
    if (which == 1) {
        for (int w = threadIdx.x; w < ops * Tile::kBytes; w += kKvThreads) {
            const int op = s_ops[w / Tile::kBytes], line = w % Tile::kBytes;
            const int i = op & 255, n = op >> 8;
            const KvPlace p = kv_place(a, s_place[i], head);
            const uint8_t* src = a.codes[1] + (p.block * Tile::kBytes + line) * 16 + p.token;
            uint8_t* dst = s_codes + i * Tile::kBytes + line;
            auto four = [&](int r, uint32_t v) {
#pragma unroll
                for (int k = 0; k < 4; ++k) dst[(r + k) * Tile::kBytes] = (uint8_t)(v >> (8 * k));
            };
            if (n == 16) {
                const uint4 v = load16(src);
                four(0, v.x);
                four(4, v.y);
                four(8, v.z);
                four(12, v.w);
            } else if (n == 4) {
                four(0, *reinterpret_cast<const uint32_t*>(src));
            } else {
                *dst = *src;
            }
        }
        __syncthreads();
    }
    const int lane = threadIdx.x & (Tile::kLanes - 1);
    if (lane >= Tile::kUnits) return;
    T* out = (T*)a.out[which] + (long long)head * a.head[which];
    for (int i = threadIdx.x / Tile::kLanes; i < RT && row0 + i < a.rows; i += Tile::kPass) {
        const long long place = s_place[i];
        float f[8] = {};
        if (place >= 0) {
            const KvPlace p = kv_place(a, place, head);
            const float scale =
                kv_scale(a.scales[which][(p.block * Tile::kGroups + (BITS == 8 ? 0 : lane / 4)) * 16 + p.token]);
            uint2 c = make_uint2(0, 0);
            if (which == 0) {
                const uint8_t* src = a.codes[0] + (p.block * 16 + p.token) * Tile::kBytes + lane * Tile::kPiece;
                if constexpr (BITS == 8) c = *reinterpret_cast<const uint2*>(src);
                else c.x = *reinterpret_cast<const uint32_t*>(src);
            } else if constexpr (BITS == 8) {
                c = *reinterpret_cast<const uint2*>(s_codes + i * Tile::kBytes + lane * 8);
            } else {
                c = *reinterpret_cast<const uint2*>(s_codes + i * Tile::kBytes + (lane / 4) * 16 + (lane & 1) * 8);
                c.x = gather_nibbles(c, (lane & 2) ? 4 : 0);
            }
            kv_decode<BITS>(c, scale, f);
        }
        kv_store8<DT>(out + (long long)(row0 + i) * a.row[which], lane * 8, a.D, a.vec, f);
    }
}

}  // namespace sgmv
