// norm.hpp -- what layer_api.hip hands to the kernels of norm.hip.
#pragma once

#include <hip/hip_runtime.h>

namespace fp32gemm {

struct NormArgs {
  const char* x;
  const char* r;  // or null
  const char* w;  // or null: ones
  char* h;        // or null
  char* y;        // or null
  signed char* q;
  float* scale;   // or null: no codes
  long long ldx, ldr, ldh, ldy, ldq;  // elements
  double inv_k;
  float eps;
  int M, K, out32;  // out32: y holds 32-bit floats
};

struct NormGradArgs {
  const char* dy;
  const char* h;
  const char* w;   // or null: ones
  const char* dh;  // or null
  char* dx;
  float* partial;  // teams rows of K sums, or null
  long long lddy, ldh, lddh, lddx;  // elements
  double inv_k;
  float eps;
  int M, K, teams;
};

// Teams that a gradient over M rows is divided among, each with a row of sums.
int norm_teams(long long M);

hipError_t rms_norm_launch(int type, bool w32, const NormArgs& a, hipStream_t s);
hipError_t rms_norm_grad_launch(int type, bool w32, int dw_type, char* dw, const NormGradArgs& a, hipStream_t s);

}  // namespace fp32gemm
