// ragged_api.hip -- the C ABI of include/grouped_gemm.h: argument checks, the
// choice of a tile, and the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/fp32_gemm.h"
#include "../../include/grouped_gemm.h"
#include "ragged_host_wave.hpp"
#include "ragged_kernels.hpp"
#include "windows.hpp"

namespace fp32gemm {

hipError_t quantize_launch(int type, const char* x, long long ldx, signed char* q, long long ldq,
                           float* scale, int M, int K, hipStream_t s);
hipError_t quantize_mx4_launch(int type, const char* x, long long ldx, unsigned char* q, long long ldq,
                               unsigned char* scale, int M, int K, hipStream_t s);
void set_last_hip_error(hipError_t e);  // sgemm_api.hip

namespace {

constexpr long long kMaxDim = 1LL << 30, kMaxStride = 1LL << 40, kMaxGroups = 1 << 16;
constexpr double kMaxThreads = 4294967295.0;  // of a launch: HIP holds workgroups x threads in 32 bits
constexpr long long kMaxIntegerK = 131071;  // 131071 * 128 * 128 < 2^31

struct Plan {
  int shape;
  int bm, bn;
  bool longest_first;
  long long grid;  // workgroups; 0: more than a launch holds
};

// What a tile costs, in microseconds as measured: a slice of 128 bytes of the
// reduction on a busy compute unit and on one that holds no other tile, and a
// tile's start and end with results of 2 and of 4 bytes.  32-bit floats take
// four times the matrix instructions a slice.  8-bit and 4-bit operands are planned by
// the costs of 16-bit ones, which those of 4 bits do not quite follow: at 8192 x 8192 x
// 8192 a slice of the widest tile takes some 1.8.
struct TileCost { double busy, alone, ends2, ends4; };
constexpr TileCost kCost16[kShapes] = {{1.4, 1.4, 7.2, 8.5}, {.50, .64, 2.0, 2.5}, {.54, .52, 2.3, 3},
                                       {.19, .28, .9, .9},    {.135, .2, .5, .5},   {.09, .11, .5, .5}};
constexpr TileCost kCost32[kShapes] = {{7.1, 7.1, 8.5, 8.5}, {1.9, 1.93, 2.5, 2.5}, {1.95, 1.93, 3, 3},
                                       {.52, .62, .8, .8},   {.14, .22, .5, .5},    {.09, .11, .5, .5}};

long long tiles(long long n, int t) { return (n + t - 1) / t; }

// Workgroups of a shape for any split of the rows, as a double: queries may ask
// for more than 64 bits hold.
double workgroups(int form, int shape, int groups, long long M, long long N, long long K) {
  const int bm = kRaggedRows[shape], bn = kRaggedCols[shape];
  if (form == kFormTN) return groups * std::ceil(static_cast<double>(tiles(K, bm)) * tiles(N, bn) / 8) * 8;
  // Every used group may leave one row tile partly filled; the dies take whole
  // tiles, and partly filled ones kDeal columns at a time, in eights.
  const long long used = std::min<long long>(groups, M);
  return static_cast<double>((M + used * (bm - 1)) / bm) * tiles(N, bn) + used * (kDeal - 1) + 8 + 8 * kDeal;
}

// Slices of 128 bytes of a reduction; the offsets are on the device, so groups
// are taken as equal.
double slices_of(int form, int type, int groups, long long M, long long K) {
  const double steps = form == kFormTN ? static_cast<double>(M) / groups : static_cast<double>(K);
  return std::max(1.0, std::ceil(steps * elem_size(type) / 128));
}
// Looking up the order of the lengths takes some 0.4 us of every tile.
constexpr double kLongSlices = 8;
bool longest_first(int form, double slices) { return form == kFormTN && slices >= kLongSlices; }

// The shape whose tiles, spread over the compute units, are done first by these
// costs.  Groups are taken as equal but for the last row tile of each, which is
// half full.
Plan plan(int form, int type, int out, int groups, long long M, long long N, long long K) {
  constexpr double kUnits = 256;
  const long long used = std::min<long long>(groups, M);
  const TileCost* cost = type == kElemF32 ? kCost32 : kCost16;
  const double slices = slices_of(form, type, groups, M, K);
  Plan p{};
  double best = 0;
  for (int shape = 0; shape < kShapes; ++shape) {
    if (!ragged_compiled(type, form, shape)) continue;
    const int bm = kRaggedRows[shape], bn = kRaggedCols[shape];
    if (workgroups(form, shape, groups, M, N, K) * kRaggedThreads[shape] > kMaxThreads) continue;
    const TileCost& c = cost[shape];
    double count;  // tiles
    if (form == kFormTN) count = static_cast<double>(groups) * tiles(K, bm) * tiles(N, bn);
    else if (groups == 1) count = static_cast<double>(tiles(M, bm)) * tiles(N, bn);
    else if (shape == kWide) count = (static_cast<double>(M) / bm + used / 8.0) * tiles(N, bn);
    else count = std::max<double>(used, static_cast<double>(M) / bm + used / 2.0) * tiles(N, bn);
    // Tiles of the fullest compute unit.  Wide ones of ragged groups come in
    // all sizes and leave some 0.4 of one idle, small ones half of one.
    double n = count / kUnits;
    if (shape == kWide && form != kFormTN && groups > 1) n = n <= 1 ? 1 : n + 0.4;
    else if (shape <= kDeep) n = std::ceil(n);
    // Long reductions of ragged groups: where all tiles are resident at once,
    // long ones share a unit to the end; one at a time, the longest first, they
    // even out.  Over 13 sizes of 257 to 512 tiles, with lengths up to six times
    // apart and with equal ones, kMid takes on average 1.17 and .95 of kDeep's
    // time in f32 (8000 rows over 8, 1024 x 1024: 172 us and 144; equal groups
    // 135 and 138), but 1.01 to 1.03 and .88 to .90 in bf16, whose slices are
    // short beside a tile's ends (35.3 and 34.5; equal groups 30.5 and 35.1).
    if (form == kFormTN && type == kElemF32 && groups > 1 && shape == kMid && n == 2 && slices >= kLongSlices)
      n = 2.5;
    if (shape == kSmall && n > 1) n += 0.5;
    const double busy = c.busy * (form == kFormNN && shape == kThin ? 1.5 : 1.0);
    const double time = std::max(n * busy, c.alone) * slices +
                        std::max(n, 1.0) * (out == kElemF32 ? c.ends4 : c.ends2);
    if (best == 0 || time < best) {
      best = time;
      p.shape = shape;
    }
  }
  p.longest_first = longest_first(form, slices);
  if (best == 0) return Plan{};  // no tile's workgroups fit a launch
  p.bm = kRaggedRows[p.shape];
  p.bn = kRaggedCols[p.shape];
  p.grid = static_cast<long long>(workgroups(form, p.shape, groups, M, N, K));
  return p;
}

// The tile that workgroup w takes, as the kernel finds it.
TileAt host_tile(int form, int shape, const Groups& g, int w, int K, int tiles_n, bool longest) {
  const HostWave wave;
  auto one = [&](auto bm) {
    constexpr int BM = decltype(bm)::value;
    return form == kFormTN ? tile_of_group<BM>(wave, g, w, static_cast<int>(tiles(K, BM)), tiles_n, longest)
                           : tile_of_rows<BM>(wave, g, w, tiles_n);
  };
  switch (kRaggedRows[shape]) {
    case 256: return one(std::integral_constant<int, 256>{});
    case 128: return one(std::integral_constant<int, 128>{});
    case 64: return one(std::integral_constant<int, 64>{});
    default: return one(std::integral_constant<int, 16>{});
  }
}

int launch(int type, int form, const RaggedArgs& a, long long M, long long N, long long K,
           void* stream) {
  const Plan p = plan(form, type, a.out, a.groups, M, N, K);
  if (p.grid == 0) return SGEMM_ERR_UNSUPPORTED;
  RaggedArgs args = a;
  args.longest_first = p.longest_first;
  const int rc = sgemm_device_check();
  if (rc != SGEMM_OK) return rc;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t err = type == kElemF32    ? ragged_f32(form, p.shape, args, p.grid, s)
                         : type == kElemBF16 ? ragged_bf16(form, p.shape, args, p.grid, s)
                         : type == kElemF16  ? ragged_f16(form, p.shape, args, p.grid, s)
                         : type == kElemM4   ? ragged_m4(form, p.shape, args, p.grid, s)
                                             : ragged_i8(form, p.shape, args, p.grid, s);
  if (err != hipSuccess) {
    set_last_hip_error(err);
    return SGEMM_ERR_LAUNCH;
  }
  return SGEMM_OK;
}

bool float_type(int t) { return t == GEMM_F32 || t == GEMM_BF16 || t == GEMM_F16; }
long long at_least(long long n) { return n > 1 ? n : 1; }

bool plan_arguments(int form, int type, int out_type, int groups, long long M, long long N, long long K) {
  const bool typed = float_type(type) || ((type == kElemI8 || type == kElemM4) && form == kFormNT);
  return form >= kFormNT && form <= kFormTN && typed && float_type(out_type) && groups >= 1 && groups <= kMaxGroups &&
         M >= 0 && N >= 0 && K >= 0 && M <= kMaxDim && N <= kMaxDim && K <= kMaxDim;
}

}  // namespace
}  // namespace fp32gemm

using namespace fp32gemm;

extern "C" {

int gemm_grouped(int32_t type, int32_t out_type, int32_t transpose_w, int32_t groups,
                 const int32_t* offsets, int64_t M, int64_t N, int64_t K, float alpha, const void* X,
                 int64_t ldx, const void* W, int64_t ldw, int64_t stride_w, float beta, void* Y,
                 int64_t ldy, void* stream) {
  if (!float_type(type)) return -1;
  if (out_type != type && out_type != GEMM_F32) return -2;
  if (transpose_w != 0 && transpose_w != 1) return -3;
  if (groups < 1 || (offsets == nullptr && groups != 1)) return -4;
  if (M < 0) return -6;
  if (N < 0) return -7;
  if (K < 0) return -8;
  if (X == nullptr && M > 0 && K > 0) return -10;
  if (ldx < at_least(K)) return -11;
  if (W == nullptr && N > 0 && K > 0) return -12;
  if (ldw < at_least(transpose_w ? K : N)) return -13;
  if (stride_w < 0) return -14;
  if (Y == nullptr && M > 0 && N > 0) return -16;
  if (ldy < at_least(N)) return -17;
  if (M > kMaxDim || N > kMaxDim || K > kMaxDim || ldx >= kRaggedMaxLd || ldw >= kRaggedMaxLd ||
      ldy >= kRaggedMaxLd || stride_w > kMaxStride || groups > kMaxGroups)
    return SGEMM_ERR_UNSUPPORTED;
  const int es = elem_size(type), os = elem_size(out_type);
  const long long y = extent(M, N, ldy, os);
  const long long w = extent(transpose_w ? N : K, transpose_w ? K : N, ldw, es);
  if (overlap(Y, y, X, extent(M, K, ldx, es)) ||
      overlap(Y, y, W, w ? (groups - 1) * stride_w * es + w : 0) ||
      (offsets && overlap(Y, y, offsets, 4LL * (groups + 1))))
    return SGEMM_ERR_OVERLAP;
  if (M == 0 || N == 0) return SGEMM_OK;
  RaggedArgs a{};
  a.A = static_cast<const char*>(X);
  a.B = static_cast<const char*>(W);
  a.C = static_cast<char*>(Y);
  a.offsets = offsets;
  a.lda = ldx * es;
  a.ldb = ldw * es;
  a.ldc = ldy;
  a.stride_b = stride_w * es;
  a.groups = groups;
  a.rows = static_cast<int>(M);
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.out = out_type;
  a.alpha = alpha;
  a.beta = beta;
  return launch(type, transpose_w ? kFormNT : kFormNN, a, M, N, K, stream);
}

int gemm_grouped_wgrad(int32_t type, int32_t out_type, int32_t groups, const int32_t* offsets,
                       int64_t M, int64_t N, int64_t K, float alpha, const void* X, int64_t ldx,
                       const void* dY, int64_t lddy, float beta, void* dW, int64_t lddw,
                       int64_t stride_dw, void* stream) {
  if (!float_type(type)) return -1;
  if (out_type != type && out_type != GEMM_F32) return -2;
  if (groups < 1 || (offsets == nullptr && groups != 1)) return -3;
  if (M < 0) return -5;
  if (N < 0) return -6;
  if (K < 0) return -7;
  if (X == nullptr && M > 0 && K > 0) return -9;
  if (ldx < at_least(K)) return -10;
  if (dY == nullptr && M > 0 && N > 0) return -11;
  if (lddy < at_least(N)) return -12;
  if (dW == nullptr && K > 0 && N > 0) return -14;
  if (lddw < at_least(N)) return -15;
  if (M > kMaxDim || N > kMaxDim || K > kMaxDim || ldx >= kRaggedMaxLd || lddy >= kRaggedMaxLd ||
      lddw >= kRaggedMaxLd || stride_dw > kMaxStride || groups > kMaxGroups)
    return SGEMM_ERR_UNSUPPORTED;
  if (stride_dw < 0 || (groups > 1 && K > 0 && N > 0 && stride_dw < (K - 1) * lddw + N)) return -16;
  const int es = elem_size(type), os = elem_size(out_type);
  const long long one = extent(K, N, lddw, os), w = one ? (groups - 1) * stride_dw * os + one : 0;
  if (overlap(dW, w, X, extent(M, K, ldx, es)) || overlap(dW, w, dY, extent(M, N, lddy, es)) ||
      (offsets && overlap(dW, w, offsets, 4LL * (groups + 1))))
    return SGEMM_ERR_OVERLAP;
  if (K == 0 || N == 0) return SGEMM_OK;
  RaggedArgs a{};
  a.A = static_cast<const char*>(X);
  a.B = static_cast<const char*>(dY);
  a.C = static_cast<char*>(dW);
  a.offsets = offsets;
  a.lda = ldx * es;
  a.ldb = lddy * es;
  a.ldc = lddw;
  a.stride_c = stride_dw;
  a.groups = groups;
  a.rows = static_cast<int>(M);
  a.M = static_cast<int>(K);
  a.N = static_cast<int>(N);
  a.out = out_type;
  a.alpha = alpha;
  a.beta = beta;
  return launch(type, kFormTN, a, M, N, K, stream);
}

int quantize_rows(int32_t type, int64_t M, int64_t K, const void* X, int64_t ldx, int8_t* Q,
                  int64_t ldq, float* scale, void* stream) {
  if (!float_type(type)) return -1;
  if (M < 0) return -2;
  if (K < 0) return -3;
  if (X == nullptr && M > 0 && K > 0) return -4;
  if (ldx < at_least(K)) return -5;
  if (Q == nullptr && M > 0 && K > 0) return -6;
  if (ldq < at_least(K)) return -7;
  if (scale == nullptr && M > 0) return -8;
  if (M > kMaxDim || K > kMaxDim || ldx > kMaxDim || ldq > kMaxDim) return SGEMM_ERR_UNSUPPORTED;
  const long long x = extent(M, K, ldx, elem_size(type)), q = extent(M, K, ldq, 1);
  if (overlap(Q, q, X, x) || overlap(scale, 4 * M, X, x) || overlap(scale, 4 * M, Q, q))
    return SGEMM_ERR_OVERLAP;
  if (M == 0) return SGEMM_OK;
  const int rc = sgemm_device_check();
  if (rc != SGEMM_OK) return rc;
  const hipError_t err =
      quantize_launch(type, static_cast<const char*>(X), ldx, reinterpret_cast<signed char*>(Q), ldq,
                      scale, static_cast<int>(M), static_cast<int>(K), static_cast<hipStream_t>(stream));
  if (err != hipSuccess) {
    set_last_hip_error(err);
    return SGEMM_ERR_LAUNCH;
  }
  return SGEMM_OK;
}

int igemm(int32_t out_type, int32_t groups, const int32_t* offsets, int64_t M, int64_t N, int64_t K,
          const int8_t* A, int64_t lda, const float* scale_a, const int8_t* B, int64_t ldb,
          int64_t stride_b, const float* scale_b, const float* bias, void* C, int64_t ldc, void* stream) {
  if (!float_type(out_type)) return -1;
  if (groups < 1 || (offsets == nullptr && groups != 1)) return -2;
  if (M < 0) return -4;
  if (N < 0) return -5;
  if (K < 0) return -6;
  if (A == nullptr && M > 0 && K > 0) return -7;
  if (lda < at_least(K)) return -8;
  if (scale_a == nullptr && M > 0) return -9;
  if (B == nullptr && N > 0 && K > 0) return -10;
  if (ldb < at_least(K)) return -11;
  if (stride_b < 0) return -12;
  if (scale_b == nullptr && N > 0) return -13;
  if (C == nullptr && M > 0 && N > 0) return -15;
  if (ldc < at_least(N)) return -16;
  if (M > kMaxDim || N > kMaxDim || K > kMaxIntegerK || lda >= kRaggedMaxLd || ldb >= kRaggedMaxLd ||
      ldc >= kRaggedMaxLd || stride_b > kMaxStride || groups > kMaxGroups)
    return SGEMM_ERR_UNSUPPORTED;
  const long long c = extent(M, N, ldc, elem_size(out_type)), b = extent(N, K, ldb, 1);
  if (overlap(C, c, A, extent(M, K, lda, 1)) || overlap(C, c, B, b ? (groups - 1) * stride_b + b : 0) ||
      overlap(C, c, scale_a, 4 * M) || overlap(C, c, scale_b, 4LL * groups * N) ||
      (bias && overlap(C, c, bias, 4LL * groups * N)) ||
      (offsets && overlap(C, c, offsets, 4LL * (groups + 1))))
    return SGEMM_ERR_OVERLAP;
  if (M == 0 || N == 0) return SGEMM_OK;
  RaggedArgs a{};
  a.A = reinterpret_cast<const char*>(A);
  a.B = reinterpret_cast<const char*>(B);
  a.C = static_cast<char*>(C);
  a.offsets = offsets;
  a.scale_a = scale_a;
  a.scale_b = scale_b;
  a.bias = bias;
  a.lda = lda;
  a.ldb = ldb;
  a.ldc = ldc;
  a.stride_b = stride_b;
  a.groups = groups;
  a.rows = static_cast<int>(M);
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.out = out_type;
  return launch(kElemI8, kFormNT, a, M, N, K, stream);
}

int quantize_mx4(int32_t type, int64_t M, int64_t K, const void* X, int64_t ldx, uint8_t* Q, int64_t ldq,
                 uint8_t* scale, void* stream) {
  if (!float_type(type)) return -1;
  if (M < 0) return -2;
  if (K < 0) return -3;
  if (X == nullptr && M > 0 && K > 0) return -4;
  if (ldx < at_least(K)) return -5;
  if (Q == nullptr && M > 0 && K > 0) return -6;
  if (ldq < at_least((K + 1) / 2)) return -7;
  if (scale == nullptr && M > 0 && K > 0) return -8;
  if (M > kMaxDim || K > kMaxDim || ldx > kMaxDim || ldq > kMaxDim) return SGEMM_ERR_UNSUPPORTED;
  const long long x = extent(M, K, ldx, elem_size(type)), q = extent(M, (K + 1) / 2, ldq, 1);
  const long long blocks = M * ((K + 31) / 32);
  if (overlap(Q, q, X, x) || overlap(scale, blocks, X, x) || overlap(scale, blocks, Q, q))
    return SGEMM_ERR_OVERLAP;
  if (M == 0 || K == 0) return SGEMM_OK;
  const int rc = sgemm_device_check();
  if (rc != SGEMM_OK) return rc;
  const hipError_t err = quantize_mx4_launch(type, static_cast<const char*>(X), ldx, Q, ldq, scale,
                                             static_cast<int>(M), static_cast<int>(K),
                                             static_cast<hipStream_t>(stream));
  if (err != hipSuccess) {
    set_last_hip_error(err);
    return SGEMM_ERR_LAUNCH;
  }
  return SGEMM_OK;
}

int gemm_mx4(int32_t out_type, int32_t groups, const int32_t* offsets, int64_t M, int64_t N, int64_t K,
             const uint8_t* A, int64_t lda, const uint8_t* scale_a, const uint8_t* B, int64_t ldb,
             int64_t stride_b, const uint8_t* scale_b, const float* bias, void* C, int64_t ldc, void* stream) {
  if (!float_type(out_type)) return -1;
  if (groups < 1 || (offsets == nullptr && groups != 1)) return -2;
  if (M < 0) return -4;
  if (N < 0) return -5;
  if (K < 0) return -6;
  if (A == nullptr && M > 0 && K > 0) return -7;
  const long long bytes = (K + 1) / 2, blocks = (K + 31) / 32;  // of a row
  if (lda < at_least(bytes)) return -8;
  if (scale_a == nullptr && M > 0 && K > 0) return -9;
  if (B == nullptr && N > 0 && K > 0) return -10;
  if (ldb < at_least(bytes)) return -11;
  if (stride_b < 0) return -12;
  if (scale_b == nullptr && N > 0 && K > 0) return -13;
  if (C == nullptr && M > 0 && N > 0) return -15;
  if (ldc < at_least(N)) return -16;
  if (M > kMaxDim || N > kMaxDim || K > kMaxDim || lda >= kRaggedMaxLd || ldb >= kRaggedMaxLd ||
      ldc >= kRaggedMaxLd || stride_b > kMaxStride || groups > kMaxGroups)
    return SGEMM_ERR_UNSUPPORTED;
  const long long c = extent(M, N, ldc, elem_size(out_type)), b = extent(N, bytes, ldb, 1);
  if (overlap(C, c, A, extent(M, bytes, lda, 1)) || overlap(C, c, B, b ? (groups - 1) * stride_b + b : 0) ||
      overlap(C, c, scale_a, M * blocks) || overlap(C, c, scale_b, groups * N * blocks) ||
      (bias && overlap(C, c, bias, 4LL * groups * N)) ||
      (offsets && overlap(C, c, offsets, 4LL * (groups + 1))))
    return SGEMM_ERR_OVERLAP;
  if (M == 0 || N == 0) return SGEMM_OK;
  RaggedArgs a{};
  a.A = reinterpret_cast<const char*>(A);
  a.B = reinterpret_cast<const char*>(B);
  a.C = static_cast<char*>(C);
  a.offsets = offsets;
  a.block_a = scale_a;
  a.block_b = scale_b;
  a.bias = bias;
  a.lda = lda;
  a.ldb = ldb;
  a.ldc = ldc;
  a.stride_b = stride_b;
  a.groups = groups;
  a.rows = static_cast<int>(M);
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(bytes);
  a.out = out_type;
  return launch(kElemM4, kFormNT, a, M, N, bytes, stream);
}

int64_t gemm_grouped_plan(int32_t form, int32_t type, int32_t out_type, int32_t groups, int64_t M,
                          int64_t N, int64_t K, int32_t tile[2]) {
  if (tile == nullptr || !plan_arguments(form, type, out_type, groups, M, N, K)) return -1;
  const Plan p = plan(form, type, out_type, groups, M, N, K);
  if (p.grid == 0) return -1;
  tile[0] = p.bm;
  tile[1] = p.bn;
  return p.grid;
}

int32_t gemm_grouped_tile(int32_t form, int32_t type, int32_t out_type, int32_t groups, int64_t M,
                          int64_t N, int64_t K) {
  if (!plan_arguments(form, type, out_type, groups, M, N, K)) return -1;
  const Plan p = plan(form, type, out_type, groups, M, N, K);
  return p.grid == 0 ? -1 : p.shape;
}

int32_t gemm_grouped_tiles(int32_t form, int32_t type) {
  if (!plan_arguments(form, type, GEMM_F32, 1, 0, 0, 0)) return -1;
  int32_t bits = 0;
  for (int shape = 0; shape < kShapes; ++shape) bits |= ragged_compiled(type, form, shape) << shape;
  return bits;
}

int64_t gemm_grouped_tile_order(int32_t form, int32_t type, int32_t tile, int32_t groups,
                                const int32_t* offsets, int64_t M, int64_t N, int64_t K, int64_t first,
                                int64_t count, int32_t* order) {
  if (!plan_arguments(form, type, GEMM_F32, groups, M, N, K) || tile < 0 || tile >= kShapes ||
      !ragged_compiled(type, form, tile) || (offsets == nullptr && groups != 1) || first < 0 || count < 0 ||
      (count > 0 && order == nullptr))
    return -1;
  const double grid = M == 0 && form != kFormTN ? 0 : workgroups(form, tile, groups, M, N, K);
  if (grid * kRaggedThreads[tile] > kMaxThreads) return -1;
  const Groups g{offsets, groups, static_cast<int>(M)};
  const bool longest = longest_first(form, slices_of(form, type, groups, M, K));
  for (int64_t w = first; w < std::min<int64_t>(first + count, grid); ++w) {
    const TileAt at = host_tile(form, tile, g, static_cast<int>(w), static_cast<int>(K),
                                static_cast<int>(tiles(N, kRaggedCols[tile])), longest);
    const int32_t four[4] = {at.group, at.row, at.hi, at.n};
    std::copy(four, four + 4, order + 4 * (w - first));
  }
  return static_cast<int64_t>(grid);
}

const char* gemm_grouped_status_string(int status) {
  static const char* const kArguments[] = {
      "argument 1 is illegal",  "argument 2 is illegal",  "argument 3 is illegal",
      "argument 4 is illegal",  "argument 5 is illegal",  "argument 6 is illegal",
      "argument 7 is illegal",  "argument 8 is illegal",  "argument 9 is illegal",
      "argument 10 is illegal", "argument 11 is illegal", "argument 12 is illegal",
      "argument 13 is illegal", "argument 14 is illegal", "argument 15 is illegal",
      "argument 16 is illegal", "argument 17 is illegal"};
  if (status < 0 && status >= -17) return kArguments[-status - 1];
  switch (status) {
    case SGEMM_ERR_OVERLAP: return "an output overlaps an input";
    case SGEMM_ERR_UNSUPPORTED: return "size beyond the supported limits";
    default: return sgemm_status_string(status);
  }
}

}  // extern "C"
