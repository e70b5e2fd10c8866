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

// The code of x: the integer nearest to 127 x / top, ties to even.  In 32 bits
// x * (127 / top) is off by at most 127 * 2^-23 < 2^-16, so it decides unless it
// lies within kNear of a tie.  The product in 64 bits is off by at most 2^-44,
// while a value that is no tie lies at least 2^-33 from one (|x| >= top / 254
// there, so both are multiples of 2^-32 top): rounding it to multiples of 2^-36
// first puts exact ties back on the tie and moves nothing across.
constexpr float kNear = 0x1p-14f;
__device__ __forceinline__ bool near_tie(float t) {
  return __builtin_fabsf(__builtin_fabsf(t - __builtin_rintf(t)) - 0.5f) < kNear;
}
__device__ __forceinline__ int code_of(float x, double inv) {
  constexpr double kSnap = 1.5 * 65536.0;
  const double t = static_cast<double>(x) * inv;
  return static_cast<int>(__builtin_rint((t + kSnap) - kSnap));
}

// One row by THREADS threads of a 256-thread workgroup.  The largest magnitude
// is an integer maximum over the bits without the sign, in which infinities
// and NaN exceed every number: such a row gets the scale NaN and codes 0.
// Rows are read in pieces of 16 bytes from any element on, their last few
// elements one a thread.  Up to KEEP pieces a thread stay in registers as they
// came, longer rows are read twice.  Memory-bound: bf16 8192 x 8192 in 38.6 us,
// 5.2 TB/s, as a copy runs (59.6 with every code in 64 bits).
constexpr int kQuantKeep = 8;
// Workgroups in x; more rows go on in y (HIP holds 2^32 threads a dimension).
constexpr int kQuantBlocks = 1 << 23;
template <int ELEM, int THREADS>
__global__ __launch_bounds__(256) void quantize_kernel(const char* x, long long ldx, signed char* q,
                                                       long long ldq, float* scale, int M, int K) {
  constexpr int ES = elem_size(ELEM), PER = 16 / ES;
  const int in = threadIdx.x % THREADS;
  const long long block = static_cast<long long>(blockIdx.y) * kQuantBlocks + blockIdx.x;
  const long long row = block * (256 / THREADS) + threadIdx.x / THREADS;
  const bool live = row < M;
  const char* src = x + (live ? row : 0) * ldx * ES;
  signed char* dst = q + (live ? row : 0) * ldq;
  const int pieces = live ? K / PER : 0, rest = live ? K % PER : 0;
  const bool one = in < rest;  // this thread takes an element of the rest

  ri4 keep[kQuantKeep];
  unsigned top = 0;
  auto load = [&](int c) {
    ri4 w;
    __builtin_memcpy(&w, src + static_cast<long long>(c) * 16, 16);
    return w;
  };
  auto value = [&](const ri4& w, int i) -> float {
    if constexpr (ELEM == kElemF32) return __builtin_bit_cast(rf4, w)[i];
    else if constexpr (ELEM == kElemBF16) return static_cast<float>(__builtin_bit_cast(rb8, w)[i]);
    else return static_cast<float>(__builtin_bit_cast(rh8, w)[i]);
  };
  auto lift = [&](float v) { top = max(top, __builtin_bit_cast(unsigned, v) & 0x7FFFFFFFu); };
  auto raise = [&](const ri4& w) {
#pragma unroll
    for (int i = 0; i < PER; ++i) lift(value(w, i));
  };
#pragma unroll
  for (int j = 0; j < kQuantKeep; ++j) {
    const int c = in + j * THREADS;
    keep[j] = c < pieces ? load(c) : ri4{};
  }
  const float last = one ? as_float<ELEM>(src, static_cast<long long>(pieces) * PER + in) : 0.0f;
#pragma unroll
  for (int j = 0; j < kQuantKeep; ++j) raise(keep[j]);
  lift(last);
  for (int c = in + kQuantKeep * THREADS; c < pieces; c += THREADS) raise(load(c));
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
  // Below 2^-100 the quotient may pass 32 bits: all in 64 then.
  const bool small = largest < 0x1p-100f;
  const float inv32 = small ? 0.0f : static_cast<float>(inv);
  if (live && in == 0)
    scale[row] = top >= 0x7F800000u ? __builtin_nanf("") : static_cast<float>(static_cast<double>(largest) / 127.0);
  auto write = [&](int c, const ri4& w) {
    int code[PER];
    bool near = small;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const float t = value(w, i) * inv32;
      near |= near_tie(t);
      code[i] = static_cast<int>(__builtin_rintf(t));
    }
    if (near)
#pragma unroll
      for (int i = 0; i < PER; ++i) code[i] = code_of(value(w, i), inv);
    unsigned o[PER / 4];
#pragma unroll
    for (int i = 0; i < PER / 4; ++i)
      o[i] = usable ? (code[4 * i] & 255u) | (code[4 * i + 1] & 255u) << 8 | (code[4 * i + 2] & 255u) << 16 |
                          static_cast<unsigned>(code[4 * i + 3]) << 24
                    : 0u;
    __builtin_memcpy(dst + static_cast<long long>(c) * PER, o, PER);
  };
#pragma unroll
  for (int j = 0; j < kQuantKeep; ++j) {
    const int c = in + j * THREADS;
    if (c < pieces) write(c, keep[j]);
  }
  if (one)
    dst[static_cast<long long>(pieces) * PER + in] = static_cast<signed char>(usable ? code_of(last, inv) : 0);
  for (int c = in + kQuantKeep * THREADS; c < pieces; c += THREADS) write(c, load(c));
}

template <int ELEM>
hipError_t launch_quantize(const char* x, long long ldx, signed char* q, long long ldq, float* scale, int M,
                           int K, hipStream_t s) {
  // A wave takes rows of up to two pieces a lane, and of up to eight where there
  // are rows enough for all waves (bf16 8192 x 4097: 20.5 us, 25.1 by four); longer
  // ones go to four waves.
  const int pieces = K / (16 / elem_size(ELEM));
  const bool wave = pieces <= 128 || (pieces <= 64 * kQuantKeep && M >= 4096);
  const unsigned blocks = static_cast<unsigned>(wave ? (M + 3) / 4 : M);
  const dim3 grid(blocks < kQuantBlocks ? blocks : kQuantBlocks, (blocks + kQuantBlocks - 1) / kQuantBlocks);
  void* values[] = {&x, &ldx, &q, &ldq, &scale, &M, &K};
  return hipLaunchKernel(wave ? reinterpret_cast<const void*>(&quantize_kernel<ELEM, 64>)
                              : reinterpret_cast<const void*>(&quantize_kernel<ELEM, 256>),
                         grid, dim3(256), values, 0, s);
}

}  // namespace

hipError_t quantize_launch(int type, const char* x, long long ldx, signed char* q, long long ldq,
                           float* scale, int M, int K, hipStream_t s) {
  return type == kElemF32    ? launch_quantize<kElemF32>(x, ldx, q, ldq, scale, M, K, s)
         : type == kElemBF16 ? launch_quantize<kElemBF16>(x, ldx, q, ldq, scale, M, K, s)
                             : launch_quantize<kElemF16>(x, ldx, q, ldq, scale, M, K, s);
}

}  // namespace fp32gemm
