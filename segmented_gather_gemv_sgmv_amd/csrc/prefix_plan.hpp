// prefix_plan.hpp -- how attention over the cache is cut into work, and where its plan and
// workspace keep it (host code without HIP; the kernels share the constants).
//
// A stack is a run of q rows that meet the same keys: all rows of the sequences that
// share a prefix over that prefix, or the rows of one sequence over its own tokens.  The
// heads that share a K / V head lie on top of each other, so a stack has
// M = rows * q_heads / kv_heads rows per K / V head.  An item is a tile of these rows (16, 32,
// 64 or, with two tiles a wave, 128) over a chunk of the keys; its results go to the
// workspace and are joined per row.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "kv_format.hpp"

namespace sgmv {

constexpr int kAttnWaves = 4;            // of an item's workgroup
constexpr int kAttnThreads = 64 * kAttnWaves;
constexpr int kAttnKeys = 64;            // keys of a wave's step
constexpr int kAttnTarget = 768;        // items to aim at
constexpr int kAttnLeast = 4;            // steps of an item, at least
constexpr int kPlanHeader = 16;          // ints: items, slots, chunk
constexpr int kStackInts = 8, kItemInts = 8;

// Row tiles of 16 that a wave keeps at once: two halve the conversions of codes per
// row, where the registers hold them (heads of up to 128; float32 has three terms of q).
inline int attn_tiles(int padded, int dtype) { return padded <= 128 && dtype != SGMV_F32 ? 2 : 1; }
inline int attn_tile_most(int padded, int dtype) { return 16 * attn_tiles(padded, dtype) * kAttnWaves; }

struct AttnSizes {
    long long items, slots;  // at most
    size_t plan_ints;
};

inline AttnSizes attn_sizes(long long rows, long long seqs, long long prefixes, int q_heads, int kv_heads,
                            int padded, int dtype) {
    const long long rep = q_heads / kv_heads, most = attn_tile_most(padded, dtype), stacks = seqs + prefixes;
    AttnSizes s;
    // Every row is in at most one prefix's stack and one sequence's.  A stack has one tile, or one
    // more than M / most; chunks beyond a tile's first are at most the target.
    s.items = kAttnTarget + kv_heads * (stacks + 2 * rows * rep / most);
    s.slots = kAttnTarget * most + kv_heads * (16 * stacks + 4 * rows * rep);
    s.plan_ints = (size_t)(kPlanHeader + kStackInts * stacks + kItemInts * s.items + rows + seqs);
    return s;
}

// Offsets into the plan's ints.
struct PlanLayout {
    long long stacks, items, row_seq, seq_prefix;
};
inline PlanLayout plan_layout(long long rows, long long seqs, long long prefixes, long long items) {
    PlanLayout l;
    l.stacks = kPlanHeader;
    l.items = l.stacks + kStackInts * (seqs + prefixes);
    l.row_seq = l.items + kItemInts * items;
    l.seq_prefix = l.row_seq + rows;
    return l;
}

}  // namespace sgmv
