// attn_f32.hip -- attention over the quantized cache, f32 queries.
#include "attn_run.hpp"

namespace sgmv {

void run_attn_f32(const AttnArgs& a, int kind, int items, hipStream_t st) { run_attn<F32>(a, kind, items, st); }

}  // namespace sgmv
