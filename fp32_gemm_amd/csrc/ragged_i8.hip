// ragged_i8.hip -- the 8-bit integer product's kernels, and the kernels that
// bring rows to 8 bits.
#include "ragged_kernels.hpp"

namespace fp32gemm {

hipError_t ragged_i8(int, int shape, const RaggedArgs& a, long long grid, hipStream_t s) {
  return launch_shape<kElemI8, kFormNT>(shape, a, grid, s);
}

namespace {

template <int ELEM>
__device__ __forceinline__ float as_float(const char* p, long long i) {
  if constexpr (ELEM == kElemF32) return reinterpret_cast<const float*>(p)[i];
  else if constexpr (ELEM == kElemBF16) return static_cast<float>(reinterpret_cast<const __bf16*>(p)[i]);
  else return static_cast<float>(reinterpret_cast<const _Float16*>(p)[i]);
}

// The code of x: the integer nearest to 127 x / top, ties to even.  The
// product with 127 / top is off by at most 2^-44 in 64 bits, while a value that
// is no tie lies at least 2^-33 from one (|x| >= top / 254 there, so both are
// multiples of 2^-32 top): rounding it to multiples of 2^-36 first puts exact
// ties back on the tie and moves nothing across.
__device__ __forceinline__ int code_of(float x, double inv) {
  constexpr double kSnap = 1.5 * 65536.0;
  const double t = static_cast<double>(x) * inv;
  return static_cast<int>(__builtin_rint((t + kSnap) - kSnap));
}

// One row by THREADS threads of a 256-thread workgroup.  The largest magnitude
// is an integer maximum over the bits without the sign, in which infinities
// and NaN exceed every number: such a row gets the scale NaN and codes 0.
// VEC: rows are whole, aligned 16-byte pieces of x and aligned groups of q;
// up to KEEP pieces a thread stay in registers, longer rows are read twice.
constexpr int kQuantKeep = 8;
template <int ELEM, int THREADS, bool VEC>
__global__ __launch_bounds__(256) void quantize_kernel(const char* x, long long ldx, signed char* q,
                                                       long long ldq, float* scale, int M, int K) {
  constexpr int ES = elem_size(ELEM), PER = VEC ? 16 / ES : 1;
  const int in = threadIdx.x % THREADS;
  const long long row = static_cast<long long>(blockIdx.x) * (256 / THREADS) + threadIdx.x / THREADS;
  const bool live = row < M;
  const char* src = x + (live ? row : 0) * ldx * ES;
  signed char* dst = q + (live ? row : 0) * ldq;
  const int pieces = live ? K / PER : 0;

  float keep[kQuantKeep][PER];
  unsigned top = 0;
  auto load = [&](int c, float* v) {
    if constexpr (VEC) {
      const ri4 w = reinterpret_cast<const ri4*>(src)[c];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if constexpr (ELEM == kElemF32) v[i] = __builtin_bit_cast(rf4, w)[i];
        else if constexpr (ELEM == kElemBF16) v[i] = static_cast<float>(__builtin_bit_cast(rb8, w)[i]);
        else v[i] = static_cast<float>(__builtin_bit_cast(rh8, w)[i]);
      }
    } else {
      v[0] = as_float<ELEM>(src, c);
    }
  };
  auto raise = [&](const float* v) {
#pragma unroll
    for (int i = 0; i < PER; ++i) top = max(top, __builtin_bit_cast(unsigned, v[i]) & 0x7FFFFFFFu);
  };
#pragma unroll
  for (int j = 0; j < kQuantKeep; ++j) {
    const int c = in + j * THREADS;
    if (c < pieces) {
      load(c, keep[j]);
      raise(keep[j]);
    }
  }
  for (int c = in + kQuantKeep * THREADS; c < pieces; c += THREADS) {
    float v[PER];
    load(c, v);
    raise(v);
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) top = max(top, static_cast<unsigned>(__shfl_xor(static_cast<int>(top), d)));
  if constexpr (THREADS > 64) {
    __shared__ unsigned tops[THREADS / 64];
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) top = max(top, tops[i]);
  }
  const float largest = __builtin_bit_cast(float, top);
  const bool usable = top != 0 && top < 0x7F800000u;
  const double inv = usable ? 127.0 / static_cast<double>(largest) : 0.0;
  if (live && in == 0)
    scale[row] = top >= 0x7F800000u ? __builtin_nanf("") : static_cast<float>(static_cast<double>(largest) / 127.0);
  auto write = [&](int c, const float* v) {
    if constexpr (VEC) {
      unsigned w[PER / 4];
#pragma unroll
      for (int i = 0; i < PER / 4; ++i) {
        w[i] = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          w[i] |= (usable ? static_cast<unsigned>(code_of(v[4 * i + b], inv)) & 255u : 0u) << (8 * b);
      }
      if constexpr (PER == 8) reinterpret_cast<ri2*>(dst)[c] = ri2{static_cast<int>(w[0]), static_cast<int>(w[1])};
      else reinterpret_cast<unsigned*>(dst)[c] = w[0];
    } else {
      dst[c] = static_cast<signed char>(usable ? code_of(v[0], inv) : 0);
    }
  };
#pragma unroll
  for (int j = 0; j < kQuantKeep; ++j) {
    const int c = in + j * THREADS;
    if (c < pieces) write(c, keep[j]);
  }
  for (int c = in + kQuantKeep * THREADS; c < pieces; c += THREADS) {
    float v[PER];
    load(c, v);
    write(c, v);
  }
}

template <int ELEM>
void launch_quantize(const char* x, long long ldx, signed char* q, long long ldq, float* scale, int M,
                     int K, hipStream_t s) {
  constexpr int ES = elem_size(ELEM), PER = 16 / ES;
  const bool vec = K % PER == 0 && ldx % PER == 0 && ldq % PER == 0 &&
                   reinterpret_cast<uintptr_t>(x) % 16 == 0 && reinterpret_cast<uintptr_t>(q) % PER == 0;
  // A wave takes rows of up to two pieces a lane; longer ones go to four waves.
  const bool wave = (vec ? K / PER : K) <= 128;
  const dim3 grid(static_cast<unsigned>(wave ? (M + 3) / 4 : M));
  if (vec && wave) quantize_kernel<ELEM, 64, true><<<grid, 256, 0, s>>>(x, ldx, q, ldq, scale, M, K);
  else if (vec) quantize_kernel<ELEM, 256, true><<<grid, 256, 0, s>>>(x, ldx, q, ldq, scale, M, K);
  else if (wave) quantize_kernel<ELEM, 64, false><<<grid, 256, 0, s>>>(x, ldx, q, ldq, scale, M, K);
  else quantize_kernel<ELEM, 256, false><<<grid, 256, 0, s>>>(x, ldx, q, ldq, scale, M, K);
}

}  // namespace

hipError_t quantize_launch(int type, const char* x, long long ldx, signed char* q, long long ldq,
                           float* scale, int M, int K, hipStream_t s) {
  if (type == kElemF32) launch_quantize<kElemF32>(x, ldx, q, ldq, scale, M, K, s);
  else if (type == kElemBF16) launch_quantize<kElemBF16>(x, ldx, q, ldq, scale, M, K, s);
  else launch_quantize<kElemF16>(x, ldx, q, ldq, scale, M, K, s);
  return hipGetLastError();
}

}  // namespace fp32gemm
