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

struct Stack {
    int row0, rows, len;
    int tile, mtiles, blocks;  // rows of a tile, tiles per K / V head, steps of 64 keys
};

__device__ __forceinline__ int plan_row(const PlanArgs& a, int s) {
    const int r = a.row_indptr ? a.row_indptr[s] : s;
    return min(max(r, 0), a.rows);
}

__device__ __forceinline__ Stack plan_stack(const PlanArgs& a, int i) {
    Stack k;
    int lo, hi;
    long long len, most;
    if (i < a.prefixes) {
        const int s0 = a.prefix_indptr ? a.prefix_indptr[i] : 0;
        const int s1 = a.prefix_indptr ? a.prefix_indptr[i + 1] : a.seqs;
        lo = min(max(s0, 0), a.seqs);
        hi = min(max(s1, lo), a.seqs);
        len = a.prefix_lengths[i];
        most = a.prefix_tokens;
    } else {
        lo = i - a.prefixes;
        hi = lo + 1;
        len = a.lengths[lo];
        most = a.own_tokens;
    }
    k.row0 = plan_row(a, lo);
    k.rows = max(plan_row(a, hi) - k.row0, 0);
    k.len = (int)min(max(len, 0ll), most);
    const int M = k.rows * a.rep;
    const int wide = 16 * a.tiles * kAttnWaves;
    k.tile = 16;
    while (k.tile < M && k.tile < wide) k.tile *= 2;
    k.mtiles = (M + k.tile - 1) / k.tile;
    k.blocks = (k.len + kAttnKeys - 1) / kAttnKeys;
    return k;
}

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
    const int n = a.prefixes + a.seqs, tid = threadIdx.x, lane = tid & 63;
    // Steps of 64 keys in all, and from them those of a chunk.
    long long work = 0;
    for (int i = tid; i < n; i += kPlanThreads) {
        const Stack k = plan_stack(a, i);
        work += (long long)a.kv_heads * k.mtiles * k.blocks;
    }
    work = block_sum64(work, s_sum);
    const int chunk = (int)min(max((long long)kAttnLeast, (work + kAttnTarget - 1) / kAttnTarget), 0x3FFFFFFFll);
    auto items_of = [&](const Stack& k) {
        return (long long)a.kv_heads * k.mtiles * ((k.blocks + chunk - 1) / chunk);
    };
    // Row tables whose sequences overlap could ask for more than there is: no work then.
    long long items = 0, slots = 0;
    for (int i = tid; i < n; i += kPlanThreads) {
        const Stack k = plan_stack(a, i);
        items += items_of(k);
        slots += items_of(k) * k.tile;
    }
    items = block_sum64(items, s_sum);
    slots = block_sum64(slots, s_sum);
    const bool fits = items <= a.items && slots <= a.slots;
    // Where every stack's items and slots begin.
    long long item_base = 0, slot_base = 0;
    for (int base = 0; base < n; base += kPlanThreads) {
        const int i = base + tid;
        Stack k{};
        long long mine = 0;
        if (i < n && fits) {
            k = plan_stack(a, i);
            mine = items_of(k);
        }
        long long all_items, all_slots;
        const long long i1 = block_scan64(mine, s_sum, all_items);
        const long long s1 = block_scan64(mine * k.tile, s_sum, all_slots);
        if (i < n) {
            k = plan_stack(a, i);
            int* r = a.plan + a.at.stacks + (long long)i * kStackInts;
            r[0] = k.row0;
            r[1] = k.rows;
            r[2] = k.len;
            r[3] = (int)(item_base + i1 - mine);
            r[4] = mine ? (k.blocks + chunk - 1) / chunk : 0;
            r[5] = k.mtiles;
            r[6] = k.tile;
            r[7] = (int)(slot_base + s1 - mine * k.tile);
        }
        item_base += all_items;
        slot_base += all_slots;
    }
    if (tid == 0) {
        a.plan[0] = fits ? (int)items : 0;
        a.plan[1] = fits ? (int)slots : 0;
        a.plan[2] = chunk;
    }
    __syncthreads();  // the stacks' records are read below by other threads of this workgroup
    // Rows of no sequence.
    const int first = plan_row(a, 0), last = plan_row(a, a.seqs);
    for (int r = tid; r < a.rows; r += kPlanThreads)
        if (r < first || r >= last) a.plan[a.at.row_seq + r] = -1;
    // Items, one stack a wave; rows and sequences of the stack.
    for (int i = tid / 64; i < n; i += kPlanThreads / 64) {
        const Stack k = plan_stack(a, i);
        const int* r = a.plan + a.at.stacks + (long long)i * kStackInts;
        const int item0 = r[3], chunks = r[4], slot0 = r[7];
        for (int j = lane; j < a.kv_heads * k.mtiles * chunks; j += 64) {
            const int t = j / chunks, part = j - t * chunks;  // (head, tile), chunk
            const int head = t / k.mtiles, mt = t - head * k.mtiles;
            int* e = a.plan + a.at.items + (long long)(item0 + j) * kItemInts;
            e[0] = i;
            e[1] = head;
            e[2] = mt * k.tile;
            e[3] = (int)((long long)k.blocks * part / chunks);  // chunks of a stack alike in length
            e[4] = (int)((long long)k.blocks * (part + 1) / chunks);
            e[5] = slot0 + j * k.tile;
            e[6] = k.tile;
            e[7] = 0;
        }
        if (i >= a.prefixes) {
            for (int j = lane; j < k.rows; j += 64) a.plan[a.at.row_seq + k.row0 + j] = i - a.prefixes;
        } else {
            const int s0 = a.prefix_indptr ? min(max(a.prefix_indptr[i], 0), a.seqs) : 0;
            const int s1 = a.prefix_indptr ? min(max(a.prefix_indptr[i + 1], s0), a.seqs) : a.seqs;
            for (int s = s0 + lane; s < s1; s += 64) a.plan[a.at.seq_prefix + s] = i;
        }
    }
}

}  // namespace sgmv
