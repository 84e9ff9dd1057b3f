// prefix_plan.hpp -- how attention over the cache is cut into work, and where its plan and
// workspace keep it (host code without HIP; the kernels share the constants).
//
// A stack is a run of q rows that meet the same keys: all rows of the sequences that
// share a prefix over that prefix, or the rows of one sequence over its own tokens.  The
// heads that share a K / V head lie on top of each other, so a stack has
// M = rows * q_heads / kv_heads rows per K / V head.  An item is a tile of these rows (16, 32,
// 64 or, with two tiles a wave, 128) over a chunk of the keys.  Where every sequence of a run fills the
// largest tile (prompts), the prefix is put in front of each sequence's own tokens instead: the prefix is read
// by each tile either way.  A row whose keys are one item's has its output from there; the results of the others
// go to the workspace and are joined per row.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "kv_format.hpp"

namespace sgmv {

constexpr int kAttnWaves = 4;            // of an item's workgroup
constexpr int kAttnThreads = 64 * kAttnWaves;
constexpr int kAttnKeys = 64;            // keys of a wave's step
// Items to aim at, most of what two workgroups a CU can take: what is too much costs partial results, what is too
// little leaves CUs waiting.  Kernel and join at 384, 448, 512: 64 sequences behind 16384 tokens, 32 / 8 heads of
// 128: 60, 55, 61 us; 24 behind 6000, 40 heads of 128, 4 bits: 54, 54, 54; 32 of up to 4000 tokens without a prefix,
// 32 / 8 heads of 128: 45, 42, 40; four prompts of up to 600 rows, 16 / 4 heads of 128, 4 bits: 51, 48, 47.
// A stack is cut into chunks of about work / target, or not at all below 1.7 of
// that.  Work is counted in steps of 64 keys of a tile; a step of 64 or 128 rows takes about twice as long as
// one of up to 32.
constexpr int kAttnTarget = 448;
// Work of an item, at least.  Kernel and join at 4, 6, 8: 40 sequences behind 450 to 1350 tokens, 12 / 4 heads of 96,
// float32: 19.5, 18.4, 19.1 us; 12 of up to 800 behind 250 to 750, 16 / 4 heads of 64, bfloat16: 13.2, 14.0, 14.3;
// 16 of up to 2000 behind 1500, 8 / 2 heads of 256, float16: 24, 25, 27; three short ones: 10.8 at each.
constexpr int kAttnLeast = 6;
constexpr int kPlanHeader = 16;          // ints: items, slots, work of a chunk

// Records of the plan, in ints.
enum { kStackRow0, kStackRows, kStackLen, kStackItem0, kStackChunks, kStackTiles, kStackTile, kStackSlot0,
       kStackBlocks, kStackFront, kStackPrefix, kStackDone, kStackInts };
enum { kItemTile, kItemHead, kItemM0, kItemBlk0, kItemBlk1, kItemSlot, kItemRow0, kItemM, kItemLen, kItemHidden,
       kItemTable, kItemOwn, kItemFrontLen, kItemFrontTable, kItemFrontBlocks, kItemFinal, kItemInts };

// Lanes that join a row's results, four elements each.
constexpr int attn_join_lanes(int padded) { return padded <= 64 ? 16 : padded <= 128 ? 32 : 64; }

// Row tiles of 16 that a wave keeps at once: two halve the conversions of codes per
// row, where the registers hold them (heads of up to 128; float32 has three terms of q).
inline int attn_tiles(int padded, int dtype) { return padded <= 128 && dtype != SGMV_F32 ? 2 : 1; }
inline int attn_tile_most(int padded, int dtype) { return 16 * attn_tiles(padded, dtype) * kAttnWaves; }

struct AttnSizes {
    long long items, slots;  // at most; a slot is a row's result of one item, to be joined
    size_t plan_ints;
};

// Slots of the first chunks of n stacks that share `rows` rows (of one K / V head), at most: a stack of M rows has
// tiles of M + tile - 1 rows in all, and of 16 + 2 M.
inline long long attn_first_slots(long long n, long long rows, long long tile) {
    const long long a = rows + n * (tile - 1), b = 16 * n + 2 * rows;
    return a < b ? a : b;
}

inline AttnSizes attn_sizes(long long rows, long long seqs, long long prefixes, int q_heads, int kv_heads,
                            int padded, int dtype) {
    const long long rep = q_heads / kv_heads, most = attn_tile_most(padded, dtype), stacks = seqs + prefixes;
    AttnSizes s;
    // Every row is in at most one prefix's stack and one sequence's.  A stack has one tile, or one
    // more than M / most.  A tile of work w has at most w / chunk + 0.3 chunks: beyond the first of each tile
    // these are no more than the target.
    s.items = kAttnTarget + kv_heads * (stacks + (prefixes ? 2 : 1) * rows * rep / most);
    long long tile = 16;  // of any stack, at most
    while (tile < rows * rep && tile < most) tile *= 2;
    s.slots = kAttnTarget * tile + kv_heads * (attn_first_slots(seqs, rows * rep, tile) +
                                               (prefixes ? attn_first_slots(prefixes, rows * rep, tile) : 0));
    // Without prefixes only stacks that are cut have slots: from a work of 1.7 chunks on, so c chunks stand for a
    // work of c / (1 + 0.3 / 1.7) of them.
    const long long cut = (kAttnTarget * 20 / 17 + 1) * tile;
    if (prefixes == 0 && cut < s.slots) s.slots = cut;
    s.plan_ints = (size_t)(kPlanHeader + kStackInts * stacks + kItemInts * s.items + rows + seqs + prefixes);
    return s;
}

// Offsets into the plan's ints.
struct PlanLayout {
    long long stacks, items, row_seq, seq_prefix, apart;
};
inline PlanLayout plan_layout(long long rows, long long seqs, long long prefixes, long long items) {
    PlanLayout l;
    l.stacks = kPlanHeader;
    l.items = l.stacks + kStackInts * (seqs + prefixes);
    l.row_seq = l.items + kItemInts * items;
    l.seq_prefix = l.row_seq + rows;
    l.apart = l.seq_prefix + seqs;
    return l;
}

}  // namespace sgmv
