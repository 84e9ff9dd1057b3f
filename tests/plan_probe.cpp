// The choice rules of proj_plan.hpp as C functions, for test_projection_choices.py.
#include "proj_plan.hpp"

using namespace sgmv;

extern "C" {

int probe_q4_path(long long R, long long N, int flushes, int gated, int bytes, int vec) {
    return q4_path(R, N, flushes, gated, bytes, vec);
}
int probe_q4_strip(long long R, long long N, int flushes, int gated) {
    return q4_strip_block(R, N, flushes, gated);
}
int probe_ffn_path(long long R, long long N, int bytes, int vec) { return ffn_path(R, N, bytes, vec); }
int probe_ffn_wide(long long N) { return ffn_wide_strips(N); }

// Kinds of tile of a 16-bit product: of the first whole rounds (-1: not split off)
// and of the rest, or of all.  flushes: of 4-bit weights, else 0.
void probe_tiles(long long M, long long N, int batches, int gated, int flushes, int* kinds) {
    const TilePlan p = plan_tiles(M, N, batches, gated, flushes);
    kinds[0] = p.big.m_end > 0 ? (int)p.big_kind : -1;
    kinds[1] = p.kind;
}
int probe_f32_tiles(long long M, long long N, int batches, int gated) {
    return f32_kind(M, N, batches, gated);
}
// dx's sums: the kind of tile, and how many ranges of K.
int probe_sum(long long M, long long N, long long K, int segments, int dtype, int* ranges) {
    const SumPlan p = plan_sum(M, N, K, segments, dtype);
    *ranges = p.ranges;
    return p.kind;
}
int probe_rope(long long rows, long long heads, int head_dim, int rotary_dim, int interleaved, int v) {
    const RopeGrid g = rope_grid(rows, heads, head_dim, rotary_dim, interleaved != 0, v);
    return rope_units_per_thread(g.heads_per_group, g.units);
}

}  // extern "C"
