// layer_api.hip -- the C ABI of include/layer_ops.h: argument checks and launches.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/fp32_gemm.h"
#include "../../include/grouped_gemm.h"
#include "../../include/layer_ops.h"
#include "expert_layer.hpp"
#include "norm.hpp"
#include "ragged_kernels.hpp"
#include "windows.hpp"

namespace fp32gemm {

void set_last_hip_error(hipError_t e);  // sgemm_api.hip

namespace {

constexpr long long kMaxDim = 1LL << 30, kMaxStride = 1LL << 40, kMaxWidth = 1LL << 19;  // 512 rows of h within a buffer offset

bool float_type(int t) { return t == GEMM_F32 || t == GEMM_BF16 || t == GEMM_F16; }
bool own_or_f32(int t, int type) { return t == type || t == GEMM_F32; }
long long at_least(long long n) { return n > 1 ? n : 1; }

int launched(hipError_t err) {
  if (err == hipSuccess) return SGEMM_OK;
  set_last_hip_error(err);
  return SGEMM_ERR_LAUNCH;
}

// The workspace of a layer: rows of h, rows of products and a counter for each run
// of columns, each part and row at a multiple of 128 bytes, a line of the L2's.
constexpr long long kLine = 128;
struct LayerRoom {
  long long h_row, z_row, z, counters, all;  // bytes
  LayerRoom(int type, long long T, long long D, long long F, long long top) {
    const auto lines = [](long long n) { return (n + kLine - 1) / kLine * kLine; };
    h_row = lines(4 * (type == kElemF32 ? F : (F + 7) / 8 * 8));
    z_row = lines(4 * D);
    z = T * top * h_row;
    counters = z + T * top * z_row;
    all = counters + lines(4 * ((D + 31) / 32));
  }
};

}  // namespace
}  // namespace fp32gemm

using namespace fp32gemm;

extern "C" {

int rms_norm(int32_t type, int32_t weight_type, int32_t out_type, int64_t M, int64_t K, float eps,
             const void* X, int64_t ldx, const void* R, int64_t ldr, const void* weight, void* H,
             int64_t ldh, void* Y, int64_t ldy, int8_t* Q, int64_t ldq, float* scale, void* stream) {
  if (!float_type(type)) return -1;
  if (!own_or_f32(weight_type, type)) return -2;
  if (!own_or_f32(out_type, type)) return -3;
  if (M < 0) return -4;
  if (K < 0) return -5;
  if (!(eps >= 0.0f)) return -6;
  if (X == nullptr && M > 0 && K > 0) return -7;
  if (ldx < at_least(K)) return -8;
  if (R != nullptr && ldr < at_least(K)) return -10;
  if (H != nullptr && ldh < at_least(K)) return -13;
  const bool some = M > 0 && K > 0;
  if (some && Y == nullptr && Q == nullptr) return -15;
  if (Y != nullptr && ldy < at_least(K)) return -15;
  if (Q == nullptr && scale != nullptr && some) return -16;
  if (Q != nullptr && ldq < at_least(K)) return -17;
  if (scale == nullptr && Q != nullptr && M > 0) return -18;
  if (M > kMaxDim || K > kMaxDim || ldx > kMaxDim || (R && ldr > kMaxDim) || (H && ldh > kMaxDim) ||
      (Y && ldy > kMaxDim) || (Q && ldq > kMaxDim))
    return SGEMM_ERR_UNSUPPORTED;
  const int es = elem_size(type);
  const Window x{X, extent(M, K, ldx, es)}, r{R, R ? extent(M, K, ldr, es) : 0},
      w{weight, weight ? K * elem_size(weight_type) : 0}, h{H, H ? extent(M, K, ldh, es) : 0},
      y{Y, Y ? extent(M, K, ldy, elem_size(out_type)) : 0}, q{Q, Q ? extent(M, K, ldq, 1) : 0},
      sc{scale, scale ? 4 * M : 0};
  const bool in_place_x = H == X && (ldh == ldx || M <= 1), in_place_r = H == R && (ldh == ldr || M <= 1);
  if ((meet(h, x) && !in_place_x) || (meet(h, r) && !in_place_r) || meet(h, w) || meet(y, x) || meet(y, r) ||
      meet(y, w) || meet(y, h) || meet(q, x) || meet(q, r) || meet(q, w) || meet(q, h) || meet(q, y) ||
      meet(sc, x) || meet(sc, r) || meet(sc, w) || meet(sc, h) || meet(sc, y) || meet(sc, q))
    return SGEMM_ERR_OVERLAP;
  if (M == 0 || (K == 0 && scale == nullptr)) return SGEMM_OK;  // empty rows have scales
  const int rc = sgemm_device_check();
  if (rc != SGEMM_OK) return rc;
  NormArgs a{};
  a.x = static_cast<const char*>(X);
  a.r = static_cast<const char*>(R);
  a.w = static_cast<const char*>(weight);
  a.h = static_cast<char*>(H);
  a.y = static_cast<char*>(Y);
  a.q = reinterpret_cast<signed char*>(Q);
  a.scale = scale;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldh = ldh;
  a.ldy = ldy;
  a.ldq = ldq;
  a.inv_k = K > 0 ? 1.0 / static_cast<double>(K) : 0.0;
  a.eps = K > 0 ? eps : 1.0f;  // empty rows: scale 0, whatever eps
  a.M = static_cast<int>(M);
  a.K = static_cast<int>(K);
  a.out32 = out_type == GEMM_F32;
  return launched(rms_norm_launch(type, weight != nullptr && weight_type != type, a, static_cast<hipStream_t>(stream)));
}

int rms_norm_grad(int32_t type, int32_t weight_type, int32_t dw_type, int64_t M, int64_t K, float eps,
                  const void* dY, int64_t lddy, const void* H, int64_t ldh, const void* weight,
                  const void* dH, int64_t lddh, void* dX, int64_t lddx, void* dweight,
                  void* workspace, int64_t workspace_bytes, void* stream) {
  if (!float_type(type)) return -1;
  if (!own_or_f32(weight_type, type)) return -2;
  if (!own_or_f32(dw_type, type)) return -3;
  if (M < 0) return -4;
  if (K < 0) return -5;
  if (!(eps >= 0.0f)) return -6;
  const bool some = M > 0 && K > 0;
  if (dY == nullptr && some) return -7;
  if (lddy < at_least(K)) return -8;
  if (H == nullptr && some) return -9;
  if (ldh < at_least(K)) return -10;
  if (dH != nullptr && lddh < at_least(K)) return -13;
  if (dX == nullptr && some) return -14;
  if (lddx < at_least(K)) return -15;
  if (M > kMaxDim || K > kMaxDim || lddy > kMaxDim || ldh > kMaxDim || (dH && lddh > kMaxDim) || lddx > kMaxDim)
    return SGEMM_ERR_UNSUPPORTED;
  const long long room = dweight && some ? rms_norm_grad_workspace(M, K) : 0;
  if (room > 0 && (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 4 != 0)) return -17;
  if (workspace_bytes < room) return -18;
  const int es = elem_size(type);
  const Window dy{dY, extent(M, K, lddy, es)}, h{H, extent(M, K, ldh, es)},
      w{weight, weight ? K * elem_size(weight_type) : 0}, dh{dH, dH ? extent(M, K, lddh, es) : 0},
      dx{dX, extent(M, K, lddx, es)}, dw{dweight, dweight ? K * elem_size(dw_type) : 0}, ws{workspace, room};
  const bool in_place_dy = dX == dY && (lddx == lddy || M <= 1), in_place_dh = dX == dH && (lddx == lddh || M <= 1);
  if ((meet(dx, dy) && !in_place_dy) || meet(dx, h) || meet(dx, w) || (meet(dx, dh) && !in_place_dh) ||
      meet(dw, dy) || meet(dw, h) || meet(dw, w) || meet(dw, dh) || meet(dw, dx) || meet(ws, dy) || meet(ws, h) ||
      meet(ws, w) || meet(ws, dh) || meet(ws, dx) || meet(ws, dw))
    return SGEMM_ERR_OVERLAP;
  if (K == 0 || (M == 0 && dweight == nullptr)) return SGEMM_OK;
  const int rc = sgemm_device_check();
  if (rc != SGEMM_OK) return rc;
  NormGradArgs a{};
  a.dy = static_cast<const char*>(dY);
  a.h = static_cast<const char*>(H);
  a.w = static_cast<const char*>(weight);
  a.dh = static_cast<const char*>(dH);
  a.dx = static_cast<char*>(dX);
  a.partial = dweight ? static_cast<float*>(workspace) : nullptr;
  a.lddy = lddy;
  a.ldh = ldh;
  a.lddh = lddh;
  a.lddx = lddx;
  a.inv_k = 1.0 / static_cast<double>(K);
  a.eps = eps;
  a.M = static_cast<int>(M);
  a.K = static_cast<int>(K);
  a.teams = norm_teams(M);
  return launched(rms_norm_grad_launch(type, weight != nullptr && weight_type != type, dw_type,
                                       static_cast<char*>(dweight), a, static_cast<hipStream_t>(stream)));
}

int64_t rms_norm_grad_workspace(int64_t M, int64_t K) {
  if (M < 0 || K < 0 || M > kMaxDim || K > kMaxDim) return -1;
  return 4LL * norm_teams(M) * K;
}

int expert_layer(int32_t type, int32_t weights, int32_t out_type, int32_t gated, int64_t T, int64_t D,
                 int64_t F, int32_t experts, int32_t top, const void* X, int64_t ldx, const int32_t* ids,
                 const float* share, const void* W_in, int64_t ldw_in, int64_t stride_in,
                 const void* scale_in, const void* W_out, int64_t ldw_out, int64_t stride_out,
                 const void* scale_out, void* Y, int64_t ldy, void* workspace, int64_t workspace_bytes,
                 void* stream) {
  if (!float_type(type)) return -1;
  const bool i8 = weights == kElemI8, m4 = weights == kElemM4;
  if (weights != type && !i8 && !m4) return -2;
  if (!own_or_f32(out_type, type)) return -3;
  if (gated != 0 && gated != 1) return -4;
  if (T < 0) return -5;
  if (D < 0) return -6;
  if (F < 0) return -7;
  if (experts < 1) return -8;
  if (top < 1) return -9;
  const bool some = T > 0 && D > 0, work = some && F > 0;
  const long long in_row = m4 ? (D + 1) / 2 : D, out_row = m4 ? (F + 1) / 2 : F;  // elements; 4 bits: bytes
  if (X == nullptr && work) return -10;
  if (ldx < at_least(D)) return -11;
  if (ids == nullptr && work) return -12;
  if (share == nullptr && work) return -13;
  if (W_in == nullptr && work) return -14;
  if (ldw_in < at_least(in_row)) return -15;
  if (stride_in < 0) return -16;
  if ((i8 || m4) ? scale_in == nullptr && work : scale_in != nullptr) return -17;
  if (W_out == nullptr && work) return -18;
  if (ldw_out < at_least(out_row)) return -19;
  if (stride_out < 0) return -20;
  if ((i8 || m4) ? scale_out == nullptr && work : scale_out != nullptr) return -21;
  if (Y == nullptr && some) return -22;
  if (ldy < at_least(D)) return -23;
  if (T > kLayerTokens || T * top > kLayerPairs || experts > kLayerExperts || D > kMaxWidth || F > kMaxWidth ||
      ldx >= kRaggedMaxLd || ldw_in >= kRaggedMaxLd || ldw_out >= kRaggedMaxLd || ldy >= kRaggedMaxLd ||
      stride_in > kMaxStride || stride_out > kMaxStride)
    return SGEMM_ERR_UNSUPPORTED;
  const long long room = some ? expert_layer_workspace(type, T, D, F, top) : 0;
  if (room > 0 && (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 16 != 0)) return -24;
  if (workspace_bytes < room) return -25;
  const int es = elem_size(type), wes = i8 || m4 ? 1 : es;
  const long long rows = gated ? 2 * F : F;
  const long long w_in = extent(rows, in_row, ldw_in, wes), w_out = extent(D, out_row, ldw_out, wes);
  const long long in_scales = i8 ? 4 * rows : m4 ? rows * ((D + 31) / 32) : 0,
                  out_scales = i8 ? 4 * D : m4 ? D * ((F + 31) / 32) : 0;
  const Window inputs[] = {{X, extent(T, D, ldx, es)},
                           {ids, 4 * T * top},
                           {share, 4 * T * top},
                           {W_in, w_in ? (experts - 1) * stride_in * wes + w_in : 0},
                           {W_out, w_out ? (experts - 1) * stride_out * wes + w_out : 0},
                           {scale_in, experts * in_scales},
                           {scale_out, experts * out_scales}};
  const Window y{Y, extent(T, D, ldy, elem_size(out_type))}, ws{workspace, room};
  for (const Window& in : inputs)
    if (meet(y, in) || meet(ws, in)) return SGEMM_ERR_OVERLAP;
  if (meet(y, ws)) return SGEMM_ERR_OVERLAP;
  if (!some) return SGEMM_OK;
  const int rc = sgemm_device_check();
  if (rc != SGEMM_OK) return rc;
  LayerArgs a{};
  a.x = static_cast<const char*>(X);
  a.ids = ids;
  a.share = share;
  a.w_in = static_cast<const char*>(W_in);
  a.w_out = static_cast<const char*>(W_out);
  a.scale_in = scale_in;
  a.scale_out = scale_out;
  const LayerRoom parts(type, T, D, F, top);
  a.h = static_cast<char*>(workspace);
  a.z = reinterpret_cast<float*>(a.h + parts.z);
  a.finished = reinterpret_cast<int*>(a.h + parts.counters);
  a.y = static_cast<char*>(Y);
  a.ldx = ldx * es;
  a.ldw_in = ldw_in * wes;
  a.ldw_out = ldw_out * wes;
  a.ldh = parts.h_row;
  a.ldz = parts.z_row / 4;
  a.stride_in = stride_in * wes;
  a.stride_out = stride_out * wes;
  a.ldy = ldy;
  a.T = static_cast<int>(T);
  a.D = static_cast<int>(D);
  a.F = static_cast<int>(F);
  a.experts = experts;
  a.top = work ? top : 0;  // without a hidden width nothing is read, and Y is zeros
  a.gated = gated;
  a.out32 = out_type == GEMM_F32;
  return launched(expert_layer_launch(type, weights, a, static_cast<hipStream_t>(stream)));
}

int64_t expert_layer_workspace(int32_t type, int64_t T, int64_t D, int64_t F, int32_t top) {
  if (!float_type(type) || T < 0 || D < 0 || F < 0 || top < 1 || T > kLayerTokens || T * top > kLayerPairs ||
      D > kMaxWidth || F > kMaxWidth)
    return -1;
  return T == 0 || D == 0 ? 0 : LayerRoom(type, T, D, F, top).all;
}

const char* layer_status_string(int status) {
  static const char* const kMore[] = {"argument 18 is illegal", "argument 19 is illegal", "argument 20 is illegal",
                                      "argument 21 is illegal", "argument 22 is illegal", "argument 23 is illegal",
                                      "argument 24 is illegal", "argument 25 is illegal"};
  if (status <= -18 && status >= -25) return kMore[-status - 18];
  return gemm_grouped_status_string(status);
}

}  // extern "C"
