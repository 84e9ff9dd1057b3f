// q4_f32.hip -- the 4-bit projections' kernels for F32 activations.
#include "q4_run.hpp"

namespace sgmv {

template int run_q4<F32, false>(const RowsArgs&, int, hipStream_t);
template int run_q4<F32, true>(const RowsArgs&, int, hipStream_t);

}  // namespace sgmv
