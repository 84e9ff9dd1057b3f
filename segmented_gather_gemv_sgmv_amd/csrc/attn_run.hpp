// attn_run.hpp -- the launches of attention over the cache for one type of q; every type has a
// source file of its own, so that they compile side by side.
#pragma once

#include "prefix_attention.hpp"
#include "sgmv_host.hpp"

namespace sgmv {

void run_attn_f32(const AttnArgs& a, int kind, int items, hipStream_t st);
void run_attn_f16(const AttnArgs& a, int kind, int items, hipStream_t st);
void run_attn_bf16(const AttnArgs& a, int kind, int items, hipStream_t st);

template <typename QT, int P>
void run_attn_padded(const AttnArgs& a, int kind, int items, hipStream_t st) {
    constexpr int R = P <= 128 && QT::kBytes == 2 ? 2 : 1;  // attn_tiles
    const dim3 grid((unsigned)items), block(kAttnThreads);
    if (kind == SGMV_KV_FP8) launch(&attn_kernel<QT, 8, P, R>, grid, block, st, a);
    else launch(&attn_kernel<QT, 4, P, R>, grid, block, st, a);
    constexpr int kLanes = attn_join_lanes(P);
    const long long pairs = (long long)a.rows * a.q_heads;
    launch(&attn_join_kernel<QT, P>, dim3((unsigned)((pairs + 256 / kLanes - 1) / (256 / kLanes))), dim3(256),
           st, a);
}

template <typename QT>
void run_attn(const AttnArgs& a, int kind, int items, hipStream_t st) {
    const int p = kv_padded(a.D);
    if (p == 64) run_attn_padded<QT, 64>(a, kind, items, st);
    else if (p == 96) run_attn_padded<QT, 96>(a, kind, items, st);
    else if (p == 128) run_attn_padded<QT, 128>(a, kind, items, st);
    else if (p == 192) run_attn_padded<QT, 192>(a, kind, items, st);
    else run_attn_padded<QT, 256>(a, kind, items, st);
}

}  // namespace sgmv
