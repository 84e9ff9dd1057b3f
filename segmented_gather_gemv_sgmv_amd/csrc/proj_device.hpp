// proj_device.hpp -- device-side pieces shared by the base projections'
// kernels (proj_rows.hpp, proj_tile.hpp): matrix-core products of 16-byte
// operand pieces for every element type, guarded piece loads, the
// activations of the gated block with their derivatives, and the unpacking
// of 4-bit weight codes.
#pragma once

#include <type_traits>

#include "sgmv_device.hpp"

namespace sgmv {

// One operand piece is 16 bytes per lane: lane (lr, lg) = (lane % 16, lane / 16)
// holds kPK consecutive K of row (or column) lr, starting at lg * kPK.  A
// piece of the wave therefore covers 4 kPK values of K.  16-bit types take
// one MFMA of K = 32; float32 takes four of K = 4, MFMA e multiplying
// element e of every lane's piece.  Both operands use the same order of K,
// which is all a sum over K needs.
typedef float acc4_t __attribute__((ext_vector_type(4)));

template <typename DT>
struct PieceOps;
template <>
struct PieceOps<F16> {
    static constexpr int kPK = 8;
    typedef _Float16 frag_t __attribute__((ext_vector_type(8)));
    __device__ static __forceinline__ acc4_t mma(const uint4& a, const uint4& b, acc4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(frag_t, a),
                                                      __builtin_bit_cast(frag_t, b), c, 0, 0, 0);
    }
};
template <>
struct PieceOps<BF16> {
    static constexpr int kPK = 8;
    typedef __bf16 frag_t __attribute__((ext_vector_type(8)));
    __device__ static __forceinline__ acc4_t mma(const uint4& a, const uint4& b, acc4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(frag_t, a),
                                                       __builtin_bit_cast(frag_t, b), c, 0, 0, 0);
    }
};
template <>
struct PieceOps<F32> {
    static constexpr int kPK = 4;
    __device__ static __forceinline__ acc4_t mma(const uint4& a, const uint4& b, acc4_t c) {
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.y), __uint_as_float(b.y), c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.z), __uint_as_float(b.z), c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.w), __uint_as_float(b.w), c, 0, 0, 0);
        return c;
    }
};

// What lanes past the end of K read in direct global-to-LDS loads.
__device__ const uint4 g_zero_piece = {0, 0, 0, 0};

__device__ __forceinline__ uint2 load_pair(const void* p) {
    return *reinterpret_cast<const uint2*>(p);
}
__device__ __forceinline__ void store_pair(void* p, const uint2& v) {
    *reinterpret_cast<uint2*>(p) = v;
}

// Two floats to two packed 16-bit values, nearest-even (gfx950 has a packed
// conversion to bf16; NaN stays NaN, overflow goes to infinity).
template <typename DT>
__device__ __forceinline__ uint32_t pack2_rne(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2_rne<F16>(float lo, float hi) {
    return F16::pack2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pack2_rne<BF16>(float lo, float hi) {
    typedef __bf16 b2_t __attribute__((ext_vector_type(2)));
    const b2_t v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

// Elements [k, k + kPK) of a row, zero at and past K.  `vec`: the row is
// 16-byte aligned and K a multiple of kPK, so the piece lies wholly inside
// or wholly outside.
template <typename DT>
__device__ __forceinline__ uint4 load_piece(const typename DT::storage* row, int k, int K,
                                            bool vec) {
    constexpr int PK = PieceOps<DT>::kPK;
    if (vec) return k < K ? load16(row + k) : make_uint4(0, 0, 0, 0);
    union {
        typename DT::storage e[PK];
        uint4 u;
    } p;
    p.u = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < PK; ++i)
        if (k + i < K) p.e[i] = row[k + i];
    return p.u;
}

// Four consecutive elements at p (the first n valid): one 8- or 16-byte
// access when `vec` (p aligned to it and n >= 4), element by element else.
template <typename DT>
__device__ __forceinline__ void load4f(const typename DT::storage* p, int n, bool vec, float* f) {
    if (vec && n >= 4) {
        if constexpr (DT::kBytes == 4) {
            DT::unpack(load16(p), f);
        } else {
            const uint2 u = load_pair(p);
            DT::unpack2(u.x, f);
            DT::unpack2(u.y, f + 2);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = i < n ? DT::load1(p + i) : 0.f;
}
template <typename DT>
__device__ __forceinline__ void store4f(typename DT::storage* p, int n, bool vec, const float* f) {
    if (vec && n >= 4) {
        if constexpr (DT::kBytes == 4)
            store16(p, DT::pack(f));
        else
            store_pair(p, make_uint2(pack2_rne<DT>(f[0], f[1]), pack2_rne<DT>(f[2], f[3])));
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) p[i] = DT::from_float(f[i]);
}

// A pre-activation as it is kept for the backward pass: what a 16-bit type cannot hold is
// kept as its largest finite value (an infinity as it is).  Rounded to infinity it
// would meet the zeros of dh and of act' there, as NaN.
template <typename DT>
__device__ __forceinline__ float kept(float v) {
    if constexpr (DT::kBytes == 4) {
        return v;
    } else {
        constexpr float kMost = std::is_same<DT, F16>::value ? 65504.f : 0x1.FEp127f;
        return __builtin_isfinite(v) ? __builtin_amdgcn_fmed3f(v, -kMost, kMost) : v;
    }
}

// ---------------------------------------------------------------------------
// Activations a(g) of the gated block and their derivatives.  `act` is
// uniform over the launch (SGMV_ACT_* of sgmv.h).
// ---------------------------------------------------------------------------
enum { kActSilu = 0, kActGelu = 1, kActGeluTanh = 2, kActRelu = 3, kActSigmoid = 4 };

__device__ __forceinline__ float sigmoid_f(float g) { return 1.f / (1.f + __expf(-g)); }

constexpr float kInvSqrt2 = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kSqrt2OverPi = 0.79788456080286536f;
constexpr float kGeluCubic = 0.044715f;

// (1 + tanh z) / 2 is the sigmoid of 2 z, z = sqrt(2 / pi) (g + c g^3).  Taken so, the
// left tail keeps its relative accuracy; from 1 + tanh z nothing is left of it at
// g = -5, where the value is -2.3e-7.
__device__ __forceinline__ float gelu_tanh_arg(float g) {
    return 2.f * kSqrt2OverPi * (g + kGeluCubic * g * g * g);
}

// From |g| = 128 on, silu and both gelus are g or 0 and their slopes 1 or 0 in float32.
// Their formulas are evaluated no further out, where a cube or a square overflows
// and infinity times zero would be NaN: a unit masked by the type's lowest value or
// by minus infinity gives 0 and has no gradient.  A NaN passes.
constexpr float kActFar = 128.f;
__device__ __forceinline__ float not_below(float g) { return g < -kActFar ? -kActFar : g; }
__device__ __forceinline__ float not_above(float g) { return g > kActFar ? kActFar : g; }

__device__ __forceinline__ float act_value(int act, float g) {
    switch (act) {
        case kActSilu: g = not_below(g); return g * sigmoid_f(g);
        case kActGelu: g = not_below(g); return g * 0.5f * erfcf(-g * kInvSqrt2);
        case kActGeluTanh: g = not_below(g); return g * sigmoid_f(gelu_tanh_arg(g));
        case kActRelu: return g < 0.f ? 0.f : g;  // a NaN stays one
        default: return sigmoid_f(g);
    }
}

__device__ __forceinline__ void act_value_grad(int act, float g, float& a, float& d) {
    switch (act) {
        case kActSilu: {
            g = not_below(g);
            const float n = not_above(g), s = sigmoid_f(n);
            a = g * s;
            d = s * (1.f + n * (1.f - s));
            return;
        }
        case kActGelu: {
            g = not_below(g);
            const float n = not_above(g), c = 0.5f * erfcf(-n * kInvSqrt2);
            a = g * c;
            d = c + n * __expf(-0.5f * n * n) * kInvSqrt2Pi;
            return;
        }
        case kActGeluTanh: {
            g = not_below(g);
            const float n = not_above(g), z2 = gelu_tanh_arg(n), s = sigmoid_f(z2);
            a = g * s;
            d = s + 2.f * n * s * sigmoid_f(-z2) * kSqrt2OverPi * (1.f + 3.f * kGeluCubic * n * n);
            return;
        }
        case kActRelu:
            a = g < 0.f ? 0.f : g;
            d = g > 0.f ? 1.f : 0.f;
            return;
        default: {
            const float s = sigmoid_f(g);
            a = s;
            d = s * (1.f - s);
            return;
        }
    }
}

// ---------------------------------------------------------------------------
// 4-bit weight codes.  A packed dword holds the codes of one lane's operand
// piece (8 consecutive K of one output feature): code 2 p in bits
// [4 p, 4 p + 4) and code 2 p + 1 in bits [16 + 4 p, 16 + 4 p + 4), so that
// one mask picks a pair that already sits in the two halves of a register.
// Put into the top mantissa bits of 16.0 (ulp 2^-6 in fp16, 2^-3 in bf16),
// a code q becomes the exact value 16 + q: a shift and an and-or per pair.
// ---------------------------------------------------------------------------
constexpr float kCodeBias = 16.f;

template <typename DT>
__device__ __forceinline__ uint4 codes_biased(uint32_t w) {
    uint4 o;
    if constexpr (std::is_same<DT, F16>::value) {
        constexpr uint32_t m = 0x03C003C0u, b = 0x4C004C00u;
        o.x = ((w << 6) & m) | b;
        o.y = ((w << 2) & m) | b;
        o.z = ((w >> 2) & m) | b;
        o.w = ((w >> 6) & m) | b;
    } else {
        constexpr uint32_t m = 0x00780078u, b = 0x41804180u;
        o.x = ((w << 3) & m) | b;
        o.y = ((w >> 1) & m) | b;
        o.z = ((w >> 5) & m) | b;
        o.w = ((w >> 9) & m) | b;
    }
    return o;
}

// A piece of ones.
template <typename DT>
__device__ __forceinline__ uint4 ones_piece() {
    const uint32_t o = std::is_same<DT, F16>::value ? 0x3C003C00u : 0x3F803F80u;
    return make_uint4(o, o, o, o);
}

}  // namespace sgmv
