// expert_layer.hpp -- what layer_api.hip hands to the kernels of expert_layer.hip.
#pragma once

#include <hip/hip_runtime.h>

namespace fp32gemm {

struct LayerArgs {
  const char* x;
  const int* ids;      // T x top
  const float* share;  // T x top
  const char* w_in;    // experts of (gated ? 2 F : F) rows of D
  const char* w_out;   // experts of D rows of F
  const void* scale_in;   // 8-bit weights: floats, a row each; 4-bit: bytes, a block each
  const void* scale_out;
  char* h;        // workspace: T * top rows of F values of 32 bits, ldh apart (16-bit x: pairs, rows of a multiple of 8),
  float* z;       // T * top rows of D, ldz apart,
  int* finished;  // and how often each 32 columns of those are done
  char* y;
  long long ldx, ldw_in, ldw_out, ldh;   // bytes
  long long stride_in, stride_out;       // bytes between experts
  long long ldy, ldz;                    // elements
  int T, D, F, experts, top, gated, out32;
  int few, sets_in, sets_out;  // set by expert_layer_launch
};

// Tokens, and tokens times experts of each, that one call takes.
constexpr int kLayerTokens = 64, kLayerPairs = 512, kLayerExperts = 1024;

// type: Elem of x and h; weights: Elem of the weights (type, kElemI8 or kElemM4).
hipError_t expert_layer_launch(int type, int weights, const LayerArgs& a, hipStream_t s);

}  // namespace fp32gemm
