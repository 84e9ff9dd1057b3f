// attn_f16.hip -- attention over the quantized cache, f16 queries.
#include "attn_run.hpp"

namespace sgmv {

void run_attn_f16(const AttnArgs& a, int kind, int items, hipStream_t st) { run_attn<F16>(a, kind, items, st); }

}  // namespace sgmv
