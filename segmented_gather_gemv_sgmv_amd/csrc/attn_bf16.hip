// attn_bf16.hip -- attention over the quantized cache, bf16 queries.
#include "attn_run.hpp"

namespace sgmv {

void run_attn_bf16(const AttnArgs& a, int kind, int items, hipStream_t st) { run_attn<BF16>(a, kind, items, st); }

}  // namespace sgmv
