// q4_bf16.hip -- the 4-bit projections' kernels for BF16 activations.
#include "q4_run.hpp"

namespace sgmv {

template int run_q4<BF16, false>(const RowsArgs&, int, hipStream_t);
template int run_q4<BF16, true>(const RowsArgs&, int, hipStream_t);

}  // namespace sgmv
