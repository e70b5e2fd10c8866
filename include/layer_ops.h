/*
 * layer_ops.h -- C ABI of libfp32_gemm_amd.so: what stands around the products of
 * a layer: the root-mean-square norm in front of it, with the residual's addition,
 * an 8-bit output for igemm and a gradient, and a whole layer of experts for the
 * few tokens of a decoding step, on one AMD Instinct MI355X (gfx950).
 *
 * Conventions are those of grouped_gemm.h: row-major matrices with leading
 * dimensions in elements, DEVICE pointers owned by the caller, any alignment of
 * their element's size, nothing read outside the operands and nothing written
 * outside the outputs' windows.  The library allocates nothing and keeps no
 * pointer; where a call needs a workspace, the caller passes it, its content does not
 * matter before or after, and calls that may run at the same time need one each.
 * Calls enqueue one or two kernels on `stream` (a hipStream_t; NULL = default
 * stream) and may be captured into a graph.  Results do not depend on the run.
 *
 * Errors: validation happens before anything is enqueued; a status -i names the
 * i-th argument, positive ones are SGEMM_ERR_* of fp32_gemm.h.  Element types are
 * the GEMM_* of grouped_gemm.h.
 */
#ifndef LAYER_OPS_H
#define LAYER_OPS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Limits (SGEMM_ERR_UNSUPPORTED beyond): M, K, leading dimensions <= 2^30 for the
 * norms; for expert_layer T <= 64, T * top <= 512, experts <= 1024, D, F <= 2^19,
 * leading dimensions < 2^21, strides <= 2^40. */

/* H = X + R,  Y[r,k] = H[r,k] * s_r * weight[k] with s_r = 1 / sqrt(mean_k H[r,k]^2 + eps),
 * and the same rows in 8 bits, as quantize_rows would bring Y to them before it is
 * rounded: scale[r] = max_k |Y[r,k]| / 127, Q[r,k] = the integer nearest to 127 * Y[r,k] /
 * max_k |Y[r,k]|, ties to even.  A row whose values are all zero gets codes 0, a row
 * with a value that is not finite scale NaN and codes 0.  A sum of finite values past the
 * largest float makes H infinite, and neither Y nor Q.
 * X, R and H are M x K of `type`; R may be NULL (H = X).  H, Y and Q may each be NULL
 * when not wanted, but not Y and Q both.  Y and Q are made from the sum before it is
 * rounded to H.  weight: K values of weight_type, `type` or GEMM_F32, or NULL for
 * ones.  out_type: Y's, `type` or GEMM_F32.  H may be X or R itself, with the same
 * leading dimension; no other operands may overlap an output.
 * -1 type  -2 weight_type  -3 out_type  -4 M  -5 K negative  -6 eps negative or
 * not a number  -7 X NULL while not empty  -8 ldx  -10 ldr  -13 ldh smaller than a row (of
 * an operand that is given)  -15 ldy so, or Y and Q both NULL  -16 Q NULL with scale while
 * not empty  -17 ldq smaller than a row  -18 scale NULL with Q */
int rms_norm(int32_t type, int32_t weight_type, int32_t out_type, int64_t M, int64_t K, float eps,
             const void* X, int64_t ldx, const void* R, int64_t ldr, const void* weight, void* H,
             int64_t ldh, void* Y, int64_t ldy, int8_t* Q, int64_t ldq, float* scale, void* stream);

/* The gradient of Y = norm(H) * weight: with s_r as above, N = H * s_r and G = dY * weight,
 *   dX[r,k] = s_r * (G[r,k] - N[r,k] * mean_k(G[r,k] * N[r,k])) + dH[r,k]
 *   dweight[k] = sum_r dY[r,k] * N[r,k]
 * dY, H, dH and dX are M x K of `type`; dH, what reaches H by other ways, may be NULL.
 * dX may be dY or dH itself, with the same leading dimension.  dweight: K values of
 * dw_type, `type` or GEMM_F32, or NULL when not wanted; it is overwritten, by zeros
 * where M == 0.  Sums are 32-bit floats or wider, in a fixed order.
 * With dweight, the workspace holds rms_norm_grad_workspace(M, K) bytes, aligned to 4.
 * -1 type  -2 weight_type  -3 dw_type  -4 M  -5 K negative  -6 eps negative or not a
 * number  -7 dY  -9 H  -14 dX NULL while not empty  -8 lddy  -10 ldh  -13 lddh  -15
 * lddx smaller than a row  -17 workspace NULL or misaligned  -18 too small */
int rms_norm_grad(int32_t type, int32_t weight_type, int32_t dw_type, int64_t M, int64_t K, float eps,
                  const void* dY, int64_t lddy, const void* H, int64_t ldh, const void* weight,
                  const void* dH, int64_t lddh, void* dX, int64_t lddx, void* dweight,
                  void* workspace, int64_t workspace_bytes, void* stream);
int64_t rms_norm_grad_workspace(int64_t M, int64_t K); /* -1 for sizes out of range */

/* A layer of experts for T tokens, each of which names `top` experts:
 *   Y[t] = sum_j share[t,j] * W_out[e] * h(W_in[e] * X[t]),  e = ids[t,j]
 * With gated == 1, W_in[e] is 2 F x D, F rows of the gate and F more, and h(u) =
 * silu(u[0:F]) * u[F:2F]; with gated == 0 it is F x D and h = silu.  W_out[e] is D x F.
 * X is T x D of `type`, Y T x D of out_type, `type` or GEMM_F32.  ids and share are
 * T x top, tight, on the device.  An id outside 0 .. experts - 1 names no expert; a token
 * without any gets zeros.  A token may name an expert more than once.  Where F == 0 Y is
 * zeros and nothing is read.
 * weights: the weights' format.  `type` itself; 3: 8-bit integers with a float scale for each
 * row (scale_in experts x 2 F or F, scale_out experts x D), as quantize_rows writes
 * them; 5: microscaled 4-bit floats (leading dimensions and strides in bytes, scales
 * tight, a byte for each block of 32), as quantize_mx4 writes them.  Else the scales
 * are NULL.  Products are exact, sums 32-bit floats; for 8 and 4 bits, 32-bit values are
 * sums of three bfloat16 (what lies below 2^-133 is lost), and 4-bit weights are bfloat16
 * (those past 2^128, of scale bytes 253 and 254, are infinite).  h is held in 32 bits:
 * a float, or for 16-bit types a sum of two bfloat16, which is off by at most 2^-17 of
 * it and has a float's range.  Only the weights of experts that are named are read.
 * The workspace holds expert_layer_workspace(type, T, D, F, top) bytes, aligned to 16.
 * -1 type  -2 weights  -3 out_type  -4 gated not 0 or 1  -5 T  -6 D  -7 F negative
 * -8 experts < 1  -9 top < 1  -10 X  -12 ids  -13 share  -14 W_in  -17 scale_in  -18 W_out
 * -21 scale_out  -22 Y NULL while not empty (scales: or given with weights in `type`)
 * -11 ldx  -15 ldw_in  -19 ldw_out  -23 ldy smaller than a row  -16 stride_in
 * -20 stride_out negative  -24 workspace NULL or misaligned  -25 too small */
int expert_layer(int32_t type, int32_t weights, int32_t out_type, int32_t gated, int64_t T, int64_t D,
                 int64_t F, int32_t experts, int32_t top, const void* X, int64_t ldx,
                 const int32_t* ids, const float* share, const void* W_in, int64_t ldw_in,
                 int64_t stride_in, const void* scale_in, const void* W_out, int64_t ldw_out,
                 int64_t stride_out, const void* scale_out, void* Y, int64_t ldy, void* workspace,
                 int64_t workspace_bytes, void* stream);
int64_t expert_layer_workspace(int32_t type, int64_t T, int64_t D, int64_t F, int32_t top); /* -1: out of range */

/* Static string for a status of these calls (never NULL). */
const char* layer_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* LAYER_OPS_H */
