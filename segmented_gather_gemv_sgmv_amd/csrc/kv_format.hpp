// kv_format.hpp -- how the quantized K / V cache lies in memory, and what a code is worth.
//
// Codes with power-of-two scales: code c with scale byte b is worth c 2^(b - 127).
//   fp8   e4m3 codes, one scale per token and head;
//   fp4   e2m1 codes, one scale per 32 elements of a token's head.
// Such a value is exact in bfloat16, and the scale costs nothing to apply: gfx950
// converts two codes to two 16-bit operands, scaled, in one instruction.  The exponent is
// the least one with |x| <= M 2^e over the group (M = 448, 6), held where code and
// scale stay exact in the cache's type (float16: between 2^-24 and 65504); what lies
// above the largest exponent's reach saturates.  Scale byte 255, in all groups of a token's
// head, marks one that held a NaN or an infinity: all of it reads as NaN.
//
// Layout, for attention (prefix_attention.hpp): a head of head_dim elements is padded to
// P (64, 96, 128, 192 or 256).  Pages are cut into blocks of 16 tokens.
//   K codes  [page][head][token][P]          the 16-byte pieces of a token feed the
//                                            product over d as they lie;
//   V codes  [page][head][block][line][16]   tokens innermost: the product over
//                                            tokens reads 16 of them in one load.  fp8: a
//                                            line is one d.  fp4: a byte holds d = 32 g + i
//                                            (low half) and 32 g + 16 + i (high half) of
//                                            one token, line 16 g + i, so that a
//                                            token is written without reading its neighbour;
//   scales   [page][head][block][group][16]
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "sgmv.h"

namespace sgmv {

constexpr int kKvBlock = 16;      // tokens of a block
constexpr int kKvMaxDim = 256;    // head_dim
constexpr int kKvNaN = 255;       // scale byte

inline int kv_padded(int head_dim) {
    return head_dim <= 64 ? 64 : head_dim <= 96 ? 96 : head_dim <= 128 ? 128 : head_dim <= 192 ? 192 : 256;
}
inline int kv_bits(int kind) { return kind == SGMV_KV_FP8 ? 8 : 4; }
// Bytes of a token's codes of one head (K: a row; V: the number of lines).
inline int kv_code_bytes(int head_dim, int kind) { return kv_padded(head_dim) * kv_bits(kind) / 8; }
inline int kv_groups(int head_dim, int kind) { return kind == SGMV_KV_FP8 ? 1 : kv_padded(head_dim) / 32; }

// Exponents allowed for a scale.
inline void kv_exponents(int kind, int dtype, int* lo, int* hi) {
    if (dtype == SGMV_F16) {
        *lo = kind == SGMV_KV_FP8 ? -15 : -23;
        *hi = kind == SGMV_KV_FP8 ? 7 : 13;
    } else {
        *lo = kind == SGMV_KV_FP8 ? -116 : -124;
        *hi = kind == SGMV_KV_FP8 ? 119 : 125;
    }
}

}  // namespace sgmv
