// ragged_mx4.hip -- the product in microscaled 4-bit floats, and the kernel that
// brings rows to them.
//
// A block of 32 values that follow one another in a row shares a power of two,
// 2^(scale - 127), and each value is a code: sign, two bits of exponent and one
// of mantissa (0, 1/2, 1, 3/2, 2, 3, 4, 6).  Two codes a byte, the even column's
// in the low half.
//
// The product is ragged_kernel on the bytes that 8-bit operands would be, with the
// matrix instruction that scales.  8192 x 8192 x 8192: 265 us, 4150 TFLOP/s, where the
// card's power bounds it (1.86 GHz under load, matrix units 55 % busy); 16 experts of
// 16 rows, 4096 to 2048: 13 us, reading the weights at 5.3 TB/s.
#include "ragged_kernels.hpp"

namespace fp32gemm {

hipError_t ragged_m4(int, int shape, const RaggedArgs& a, long long grid, hipStream_t s) {
  return launch_shape<kElemM4, kFormNT>(shape, a, grid, s);
}

namespace {

// Eight values a thread, four threads a block of 32, 2^log2_threads threads a
// row.  The largest magnitude is an integer maximum over the bits without the
// sign, whose exponent is the block's: with the largest in [4, 8) times 2^e no
// value needs more than the saturation at 6.  Infinities and NaN exceed every
// number there; such a block gets the scale NaN.  x * 2^-e is exact but for
// values far below the smallest code, so each code is the value's one rounding.
// Memory-bound: bf16 8192 x 8192 36 to 38 us, 4.5 to 4.7 TB/s.
constexpr int kQuantBlocks = 1 << 23;  // workgroups in x; more rows go on in y
template <int ELEM>
__global__ __launch_bounds__(256) void quantize_mx4_kernel(const char* x, long long ldx, unsigned char* q,
                                                           long long ldq, unsigned char* scale, int M, int K,
                                                           int log2_threads) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int ES = elem_size(ELEM);
  const int in = threadIdx.x & ((1 << log2_threads) - 1);
  const long long block = static_cast<long long>(blockIdx.y) * kQuantBlocks + blockIdx.x;
  const long long row = block * (256 >> log2_threads) + (threadIdx.x >> log2_threads);
  if (row >= M) return;
  const int blocks = (K + 31) / 32;
  const char* src = x + row * ldx * ES;
  unsigned char* dst = q + row * ldq;
  unsigned char* sc = scale + row * blocks;
  for (int c = (blockIdx.z << log2_threads) + in; c / 4 < blocks; c += gridDim.z << log2_threads) {
    float v[8];
    const int left = K - c * 8;
    if (left >= 8) {
      if constexpr (ELEM == kElemF32) {
        rf4 w[2];
        __builtin_memcpy(w, src + static_cast<long long>(c) * 32, 32);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = w[i / 4][i % 4];
      } else {
        ri4 w;
        __builtin_memcpy(&w, src + static_cast<long long>(c) * 16, 16);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if constexpr (ELEM == kElemBF16) v[i] = static_cast<float>(__builtin_bit_cast(rb8, w)[i]);
          else v[i] = static_cast<float>(__builtin_bit_cast(rh8, w)[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const long long at = static_cast<long long>(c) * 8 + i;
        v[i] = 0.0f;
        if (i < left) {
          if constexpr (ELEM == kElemF32) v[i] = reinterpret_cast<const float*>(src)[at];
          else if constexpr (ELEM == kElemBF16) v[i] = static_cast<float>(reinterpret_cast<const __bf16*>(src)[at]);
          else v[i] = static_cast<float>(reinterpret_cast<const _Float16*>(src)[at]);
        }
      }
    }
    int top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __builtin_bit_cast(int, v[i]) & 0x7FFFFFFF);
    top = max(top, __builtin_amdgcn_update_dpp(0, top, 0xB1, 0xF, 0xF, false));  // of the thread beside,
    top = max(top, __builtin_amdgcn_update_dpp(0, top, 0x4E, 0xF, 0xF, false));  // of the pair beside
    const int exponent = top >> 23;
    const bool usable = exponent < 255;
    const int byte = usable ? max(exponent - 2, 0) : 255;
    const float inv = __builtin_bit_cast(float, usable ? (254 - byte) << 23 : 0);
    unsigned code = 0;
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[0] * inv, v[1] * inv, 1.0f, 0);
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[2] * inv, v[3] * inv, 1.0f, 1);
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[4] * inv, v[5] * inv, 1.0f, 2);
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[6] * inv, v[7] * inv, 1.0f, 3);
    if (!usable) code = 0;
    if (left >= 8) {
      __builtin_memcpy(dst + static_cast<long long>(c) * 4, &code, 4);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (2 * i < left) dst[static_cast<long long>(c) * 4 + i] = static_cast<unsigned char>(code >> (8 * i));
    }
    if (c % 4 == 0) sc[c / 4] = static_cast<unsigned char>(byte);
  }
#endif
}

}  // namespace

hipError_t quantize_mx4_launch(int type, const char* x, long long ldx, unsigned char* q, long long ldq,
                               unsigned char* scale, int M, int K, hipStream_t s) {
  const int pieces = (K + 31) / 32 * 4;
  int log2_threads = 2;
  while (log2_threads < 8 && (1 << log2_threads) < pieces) ++log2_threads;
  const unsigned rows = 256u >> log2_threads, blocks = (static_cast<unsigned>(M) + rows - 1) / rows;
  const unsigned parts = (static_cast<unsigned>(pieces) + 255) / 256;
  const dim3 grid(blocks < kQuantBlocks ? blocks : kQuantBlocks, (blocks + kQuantBlocks - 1) / kQuantBlocks,
                  parts < 1024 ? parts : 1024);
  void* values[] = {&x, &ldx, &q, &ldq, &scale, &M, &K, &log2_threads};
  const void* const kernel = type == kElemF32    ? reinterpret_cast<const void*>(&quantize_mx4_kernel<kElemF32>)
                             : type == kElemBF16 ? reinterpret_cast<const void*>(&quantize_mx4_kernel<kElemBF16>)
                                                 : reinterpret_cast<const void*>(&quantize_mx4_kernel<kElemF16>);
  return hipLaunchKernel(kernel, grid, dim3(256), values, 0, s);
}

}  // namespace fp32gemm
