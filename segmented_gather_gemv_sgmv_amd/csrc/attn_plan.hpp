// attn_plan.hpp -- the plan of attention over the cache, made on the device from lengths and
// row tables that only it knows: stacks, items, and which sequence a row belongs to
// (prefix_plan.hpp).  One workgroup; a step of a model makes it once for all layers.
#pragma once

#include "prefix_plan.hpp"
#include "sgmv_device.hpp"

namespace sgmv {

struct PlanArgs {
    int* plan;
    PlanLayout at;
    const int *lengths, *row_indptr, *prefix_lengths, *prefix_indptr;
    int rows, seqs, prefixes, kv_heads, rep;
    long long own_tokens, prefix_tokens;  // that a page table's row holds
    long long items, slots;               // at most
    int tiles;                            // R
};

constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int plan_row(const PlanArgs& a, int s) {
    const int r = a.row_indptr ? a.row_indptr[s] : s;
    return min(max(r, 0), a.rows);
}
__device__ __forceinline__ int plan_rows(const PlanArgs& a, int lo, int hi) {
    return max(plan_row(a, hi) - plan_row(a, lo), 0);
}
// Sequences [lo, hi) of prefix g.
__device__ __forceinline__ void plan_run(const PlanArgs& a, int g, int& lo, int& hi) {
    lo = a.prefix_indptr ? min(max(a.prefix_indptr[g], 0), a.seqs) : 0;
    hi = a.prefix_indptr ? min(max(a.prefix_indptr[g + 1], lo), a.seqs) : a.seqs;
}
__device__ __forceinline__ int plan_length(int len, long long most) {
    return (int)min((long long)max(len, 0), most);
}
__device__ __forceinline__ int plan_blocks(int len) { return (len + kAttnKeys - 1) / kAttnKeys; }
__device__ __forceinline__ int plan_weight(int tile) { return tile >= 64 ? 2 : 1; }

__device__ __forceinline__ long long block_sum64(long long v, long long* s) {
    for (int m = 1; m < 64; m *= 2) v += __shfl_xor(v, m);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x / 64] = v;
    __syncthreads();
    long long t = 0;
    for (int i = 0; i < kPlanThreads / 64; ++i) t += s[i];
    return t;
}

// Inclusive prefix sum over the workgroup; `total` receives the sum.
__device__ __forceinline__ long long block_scan64(long long v, long long* s, long long& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    for (int m = 1; m < 64; m *= 2) {
        const long long t = __shfl_up(v, m);
        if (lane >= m) v += t;
    }
    __syncthreads();
    if (lane == 63) s[wave] = v;
    __syncthreads();
    total = 0;
    for (int i = 0; i < kPlanThreads / 64; ++i) {
        if (i < wave) v += s[i];
        total += s[i];
    }
    return v;
}

__global__ __launch_bounds__(kPlanThreads) void attn_plan_kernel(PlanArgs a) {
    __shared__ long long s_sum[kPlanThreads / 64];
    __shared__ int s_key[kPlanThreads], s_order[kPlanThreads];
    const int n = a.prefixes + a.seqs, tid = threadIdx.x, lane = tid & 63, wave = tid / 64;
    constexpr int kWaves = kPlanThreads / 64;
    const int wide = 16 * a.tiles * kAttnWaves;
    int* seq_prefix = a.plan + a.at.seq_prefix;
    int* apart = a.plan + a.at.apart;  // prefixes that are read apart from their sequences' tokens
    // Which prefix a sequence has (-1: none); rows of no sequence.
    for (int s = tid; s < a.seqs; s += kPlanThreads) seq_prefix[s] = -1;
    for (int g = tid; g < a.prefixes; g += kPlanThreads) apart[g] = 0;
    const int first = plan_row(a, 0), last = plan_row(a, a.seqs);
    for (int r = tid; r < a.rows; r += kPlanThreads)
        if (r < first || r >= last) a.plan[a.at.row_seq + r] = -1;
    __syncthreads();
    for (int g = wave; g < a.prefixes; g += kWaves) {
        int lo, hi;
        plan_run(a, g, lo, hi);
        for (int s = lo + lane; s < hi; s += 64) seq_prefix[s] = g;
    }
    __syncthreads();
    for (int s = tid; s < a.seqs; s += kPlanThreads) {
        const int M = plan_rows(a, s, s + 1) * a.rep, g = seq_prefix[s];
        if (g >= 0 && M > 0 && M < wide) apart[g] = 1;
    }
    __syncthreads();
    // The stacks and the work in all.
    long long work = 0;
    for (int i = tid; i < n; i += kPlanThreads) {
        int row0, rows, len, front = 0, prefix = -1, only = 0;  // only: no other stack has keys of its rows
        if (i < a.prefixes) {
            int lo, hi;
            plan_run(a, i, lo, hi);
            row0 = plan_row(a, lo);
            rows = plan_rows(a, lo, hi);
            len = plan_length(a.prefix_lengths[i], a.prefix_tokens);
            if (!apart[i]) rows = 0;  // in front of its sequences' tokens
        } else {
            const int s = i - a.prefixes;
            row0 = plan_row(a, s);
            rows = plan_rows(a, s, s + 1);
            len = plan_length(a.lengths[s], a.own_tokens);
            prefix = seq_prefix[s];
            const int before = prefix >= 0 ? plan_length(a.prefix_lengths[prefix], a.prefix_tokens) : 0;
            if (prefix >= 0 && !apart[prefix]) front = before;
            only = front == before;
        }
        const int M = rows * a.rep;
        int tile = 16;
        while (tile < M && tile < wide) tile *= 2;
        const int tiles = (M + tile - 1) / tile, blocks = plan_blocks(front) + plan_blocks(len);
        int* r = a.plan + a.at.stacks + (long long)i * kStackInts;
        r[kStackRow0] = row0;
        r[kStackRows] = rows;
        r[kStackLen] = len;
        r[kStackTiles] = tiles;
        r[kStackTile] = tile;
        r[kStackBlocks] = blocks;
        r[kStackFront] = front;
        r[kStackPrefix] = prefix;
        r[kStackDone] = only;
        work += (long long)a.kv_heads * tiles * blocks * plan_weight(tile);
    }
    work = block_sum64(work, s_sum);
    const long long chunk = max((long long)kAttnLeast, (work + kAttnTarget - 1) / kAttnTarget);
    auto record = [&](int i) { return a.plan + a.at.stacks + (long long)i * kStackInts; };
    auto chunks_of = [&](const int* r) {
        if (r[kStackRows] == 0 || r[kStackBlocks] == 0) return 0;
        const long long w = (long long)r[kStackBlocks] * plan_weight(r[kStackTile]);
        return (int)max(1ll, (10 * w + 3 * chunk) / (10 * chunk));
    };
    // One chunk, and no prefix apart: the rows' outputs come from their items, and need no slots.
    auto alone = [&](const int* r, int chunks) { return chunks == 1 && r[kStackDone] != 0; };
    // Row tables whose sequences overlap could ask for more than there is: no work then.
    long long items = 0, slots = 0;
    for (int i = tid; i < n; i += kPlanThreads) {
        const int* r = record(i);
        const int chunks = chunks_of(r);
        const long long mine = (long long)a.kv_heads * r[kStackTiles] * chunks;
        items += mine;
        if (!alone(r, chunks)) slots += mine * r[kStackTile];
    }
    items = block_sum64(items, s_sum);
    slots = block_sum64(slots, s_sum);
    const bool fits = items <= a.items && slots <= a.slots;
    // Stacks of the longest items first, so that short ones even out the end (24 sequences of 1 to 2000 tokens
    // behind 6000, 40 heads of 128 in 4 bits: 49 against 54 us).  More stacks than threads stay in their order: no
    // one of so many is long against all.
    const bool sorted = n <= kPlanThreads;
    if (sorted) {
        __syncthreads();
        int key = 0;
        if (tid < n) {
            const int* r = record(tid);
            key = r[kStackBlocks] * plan_weight(r[kStackTile]) / max(chunks_of(r), 1);
        }
        s_key[tid] = key;
        __syncthreads();
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += s_key[j] > key || (s_key[j] == key && j < tid);
        if (tid < n) s_order[rank] = tid;
        __syncthreads();
    }
    // Where every stack's items and slots begin.
    long long item_base = 0, slot_base = 0;
    for (int base = 0; base < n; base += kPlanThreads) {
        const bool live = base + tid < n;
        const int i = !live ? 0 : sorted ? s_order[tid] : base + tid;
        int* r = record(i);
        const int chunks = live && fits ? chunks_of(r) : 0;
        const long long mine = live ? (long long)a.kv_heads * r[kStackTiles] * chunks : 0;
        const bool done = live && alone(r, chunks);
        const long long size = live && !done ? mine * r[kStackTile] : 0;
        long long all_items, all_slots;
        const long long i1 = block_scan64(mine, s_sum, all_items);
        const long long s1 = block_scan64(size, s_sum, all_slots);
        if (live) {
            r[kStackItem0] = (int)(item_base + i1 - mine);
            r[kStackChunks] = chunks;
            r[kStackSlot0] = (int)(slot_base + s1 - size);
            r[kStackDone] = done;
        }
        item_base += all_items;
        slot_base += all_slots;
    }
    if (tid == 0) {
        a.plan[0] = fits ? (int)items : 0;
        a.plan[1] = fits ? (int)slots : 0;
        a.plan[2] = (int)min(chunk, 0x7FFFFFFFll);
    }
    __syncthreads();
    // Items, one stack a wave, later tiles (which see more keys) first; rows of the stack.
    for (int i = wave; i < n; i += kWaves) {
        const int* r = record(i);
        const bool own = i >= a.prefixes;
        const int row0 = r[kStackRow0], rows = r[kStackRows], len = r[kStackLen], chunks = r[kStackChunks];
        const int tiles = r[kStackTiles], tile = r[kStackTile], front = r[kStackFront];
        const int M = rows * a.rep, hidden = len - rows;
        for (int j = lane; j < a.kv_heads * tiles * chunks; j += 64) {
            const int t = j / chunks, part = j - t * chunks;
            const int mt = tiles - 1 - t / a.kv_heads, head = t % a.kv_heads;
            // Steps that the tile's last row sees, shared out over its chunks.
            const int end = min((mt + 1) * tile, M) - 1;
            const int seen = own ? min(max(hidden + end / a.rep + 1, 0), len) : len;
            const int blocks = plan_blocks(front) + plan_blocks(seen);
            int* e = a.plan + a.at.items + (long long)(r[kStackItem0] + j) * kItemInts;
            e[kItemTile] = tile;
            e[kItemHead] = head;
            e[kItemM0] = mt * tile;
            e[kItemBlk0] = (int)((long long)blocks * part / chunks);
            e[kItemBlk1] = (int)((long long)blocks * (part + 1) / chunks);
            e[kItemSlot] = r[kStackSlot0] + ((head * tiles + mt) * chunks + part) * tile;
            e[kItemRow0] = row0;
            e[kItemM] = M;
            e[kItemLen] = len;
            e[kItemHidden] = hidden;
            e[kItemTable] = own ? i - a.prefixes : i;
            e[kItemOwn] = own;
            e[kItemFrontLen] = front;
            e[kItemFrontTable] = r[kStackPrefix];
            e[kItemFrontBlocks] = plan_blocks(front);
            e[kItemFinal] = r[kStackDone];
        }
        if (own)
            for (int j = lane; j < rows; j += 64) a.plan[a.at.row_seq + row0 + j] = i - a.prefixes;
    }
}

}  // namespace sgmv
