// ragged_f16.hip -- the grouped products' kernels for f16 operands.
#include "ragged_float.inc"

namespace fp32gemm {
hipError_t ragged_f16(int form, int shape, const RaggedArgs& a, long long grid, hipStream_t s) {
  return launch_float<kElemF16>(form, shape, a, grid, s);
}
}  // namespace fp32gemm
