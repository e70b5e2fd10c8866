// ragged_bf16.hip -- the grouped products' kernels for bf16 operands.
#include "ragged_float.inc"

namespace fp32gemm {
hipError_t ragged_bf16(int form, int shape, const RaggedArgs& a, long long grid, hipStream_t s) {
  return launch_float<kElemBF16>(form, shape, a, grid, s);
}
}  // namespace fp32gemm
