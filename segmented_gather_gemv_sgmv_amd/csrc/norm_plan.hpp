// norm_plan.hpp -- how the normed rotation's kernels are cut (host code without HIP, shared
// with the kernels for its constants).
#pragma once

#include <algorithm>

namespace sgmv {

constexpr int kNormThreads = 256;
constexpr int kNormMaxDim = 1024;    // of a head
constexpr int kNormAngles = 512;     // of a workgroup's rows: rows x rot / 2
constexpr int kNormGradBlocks = 1024;  // workgroups of the gradients, at most: what 4 waves a SIMD can hold

struct NormShape {
    int units, lanes, per_lane;  // units of a head, lanes that hold it, units of a lane (1, 2, 4 or 16)
};

// v: elements of a unit's piece (16 bytes, or 1 where those do not fit).
inline NormShape norm_shape(int head_dim, int rotary_dim, bool interleaved, int v) {
    NormShape s;
    s.units = (interleaved ? (v > 1 ? rotary_dim / v : rotary_dim / 2) : rotary_dim / 2 / v) +
              (head_dim - rotary_dim) / v;
    s.lanes = 1;
    while (s.lanes < s.units && s.lanes < 64) s.lanes *= 2;
    const int each = (s.units + s.lanes - 1) / s.lanes;
    s.per_lane = each <= 1 ? 1 : each <= 2 ? 2 : each <= 4 ? 4 : 16;
    return s;
}

// Rows a workgroup takes at once: as many as give its threads an angle each and whole
// passes over heads, but no more than leave the chip without work (4 workgroups per CU), and no
// fewer than make one round of them (1400 rows of 12 + 4 heads of 64, float16: 5.3 us, with one row each 6.4).
inline int norm_rows_per_block(long long rows, int rotary_dim) {
    const long long most = std::min(8, kNormAngles / (rotary_dim / 2));
    return (int)std::min(most, (rows + 1023) / 1024);
}

// The gradients of one tensor: each of at most `most` workgroups takes ceil(rows / most) rows, in turns of as many as
// its angles have room for.
struct NormGradShape {
    int block_rows, workgroups;
};
inline NormGradShape norm_grad_shape(long long rows, int rotary_dim, int most) {
    const long long room = std::min(8, kNormAngles / (rotary_dim / 2));
    const long long each = std::max(1ll, (rows + most - 1) / most);
    const long long turns = (each + room - 1) / room;
    NormGradShape s;
    s.block_rows = (int)((each + turns - 1) / turns);
    s.workgroups = (int)((rows + s.block_rows * turns - 1) / (s.block_rows * turns));
    return s;
}
// The share of the workgroups that w (0: queries, 1: keys) gets.
inline int norm_grad_share(int q_heads, int k_heads, int w) {
    const int heads = w ? k_heads : q_heads;
    return heads ? std::max(1, (int)((long long)kNormGradBlocks * heads / ((long long)q_heads + k_heads))) : 0;
}

// Heads of a workgroup in the forward pass: all of them once the blocks of rows are half a round, else
// split down to one pass (1003 rows of 5 + 5 heads of 80, float32: 6.5 us, in two groups 8.8).
inline int norm_heads_per_group(long long blocks, long long heads, int lanes) {
    const long long pass = std::max(1, kNormThreads / lanes);
    const long long want = std::max(1ll, 1024 / blocks);
    return (int)std::min(heads, std::max(pass, (heads + want - 1) / want));
}

}  // namespace sgmv
