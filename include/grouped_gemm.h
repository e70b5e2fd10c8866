/*
 * grouped_gemm.h -- C ABI of libfp32_gemm_amd.so: matrix products grouped by
 * expert with ragged sizes, their weight gradient, the product in 8-bit
 * integers with a scale for each token and channel, and the product in
 * microscaled 4-bit floats, on one AMD Instinct MI355X (gfx950).
 *
 * Groups.  The rows of X (A) are sorted by group: group e owns the rows
 * offsets[e] .. offsets[e+1]-1, and is multiplied by its own weights W_e.
 * `offsets` is a DEVICE array of groups + 1 increasing int32 row numbers
 * between 0 and M, read by the kernels when they run, so a router's counts need
 * not come back to the host.  Groups may be empty; rows that no group owns are
 * left as they are.  Offsets out of that range or order give wrong results or none, but
 * no access outside the operands.  offsets == NULL means one group of all M
 * rows.
 *
 * Matrices are row-major with leading dimensions in elements, as in
 * fp32_gemm.h; strides between the groups' weights are in elements too.  All
 * pointers are DEVICE pointers owned by the caller.  Inputs are only read, and
 * only the outputs' windows are written; bytes between an operand's rows may be
 * read (never used), none before its first or past its last.  The library allocates
 * nothing, uses no workspace and keeps no pointer.  Outputs must not overlap
 * inputs: an operand counts from its first byte to its last, so column ranges of
 * one buffer are refused too (SGEMM_ERR_OVERLAP).
 *
 * Asynchrony, thread safety, graph capture: each call enqueues one kernel on
 * `stream` (a hipStream_t; NULL = default stream) and nothing else; it may be
 * captured.  Results do not depend on the run: sums are made in a fixed order.
 *
 * Alignment.  Pointers, leading dimensions and group strides need no more than
 * their element's alignment.  Rows that start at multiples of 128 bytes and hold
 * whole slices of 128 bytes (64 halves, 128 integers) are the fastest.
 *
 * Errors: as fp32_gemm.h: validation happens before anything is enqueued; a
 * status -i names the i-th argument, positive ones are SGEMM_ERR_*.
 */
#ifndef GROUPED_GEMM_H
#define GROUPED_GEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define GEMM_F32 0
#define GEMM_BF16 1
#define GEMM_F16 2

/* Limits (SGEMM_ERR_UNSUPPORTED beyond): M, N, K <= 2^30, leading dimensions
 * < 2^21, group strides <= 2^40, groups <= 65536, and K <= 131071 for igemm,
 * whose 32-bit sums could pass their range there.  A launch holds fewer than
 * 2^32 threads, which is 2^23 tiles of 256 x 256 outputs; the partly filled last
 * tiles of a group count whole. */

/* Y_r = alpha * X_r * W_e + beta * Y_r for every row r of every group e.
 * X is M x K, Y is M x N.  W_e = W + e * stride_w is K x N, or N x K when
 * transpose_w is 1 (the form of the input gradient dX = dY * W_e^T).
 * type: X's and W's; out_type: Y's, the same or GEMM_F32.  Sums, alpha and
 * beta are 32-bit floats and the result is rounded once.  Y is not read when
 * beta == 0.  K == 0 gives beta * Y.  stride_w == 0 shares one W.
 * -1 type  -2 out_type  -3 transpose_w not 0 or 1  -4 groups < 1, or not 1
 * without offsets  -6 M  -7 N  -8 K negative  -10 X  -12 W  -16 Y NULL while
 * not empty  -11 ldx  -13 ldw  -17 ldy smaller than a row  -14 stride_w < 0 */
int gemm_grouped(int32_t type, int32_t out_type, int32_t transpose_w, int32_t groups,
                 const int32_t* offsets, int64_t M, int64_t N, int64_t K, float alpha,
                 const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t stride_w,
                 float beta, void* Y, int64_t ldy, void* stream);

/* dW_e = alpha * X_e^T * dY_e + beta * dW_e for every group e, over its rows.
 * X is M x K, dY is M x N, dW_e = dW + e * stride_dw is K x N (for weights
 * stored N x K pass dY and X in each other's place).  An empty group gets
 * beta * dW_e.  out_type: dW's, the same as type or GEMM_F32.
 * -1 type  -2 out_type  -3 groups < 1, or not 1 without offsets  -5 M  -6 N
 * -7 K negative  -9 X  -11 dY  -14 dW NULL while not empty  -10 ldx  -12 lddy
 * -15 lddw smaller than a row  -16 stride_dw smaller than a dW_e */
int gemm_grouped_wgrad(int32_t type, int32_t out_type, int32_t groups, const int32_t* offsets,
                       int64_t M, int64_t N, int64_t K, float alpha, const void* X, int64_t ldx,
                       const void* dY, int64_t lddy, float beta, void* dW, int64_t lddw,
                       int64_t stride_dw, void* stream);

/* Brings every row of X (M x K, of `type`) to 8 bits:
 * scale[r] = max_k |X[r,k]| / 127 and Q[r,k] = the integer nearest to
 * 127 * X[r,k] / max_k |X[r,k]|, ties to even, so X[r,k] ~ scale[r] * Q[r,k].
 * A row of zeros gets scale 0 and codes 0; a row that holds an infinity or a
 * NaN gets scale NaN and codes 0, so that its products are NaN throughout.
 * Weights are brought to 8 bits by the same call, a channel a row.
 * -1 type  -2 M  -3 K negative  -4 X  -6 Q  -8 scale NULL while not empty
 * -5 ldx  -7 ldq smaller than a row */
int quantize_rows(int32_t type, int64_t M, int64_t K, const void* X, int64_t ldx, int8_t* Q,
                  int64_t ldq, float* scale, void* stream);

/* C[r,n] = (sum_k A[r,k] * B_e[n,k]) * (scale_a[r] * scale_b[e,n]) + bias[e,n]
 * for every row r of every group e.  A is M x K and B_e = B + e * stride_b is
 * N x K, both int8; sums are exact 32-bit integers, rounded to a float once.
 * The two scales are multiplied first, as 32-bit floats.
 * scale_a has M entries, scale_b and bias (or NULL) groups x N, all tight.
 * out_type: C's.  K == 0 gives the bias.
 * -1 out_type  -2 groups < 1, or not 1 without offsets  -4 M  -5 N  -6 K
 * negative  -7 A  -9 scale_a  -10 B  -13 scale_b  -15 C NULL while not empty
 * -8 lda  -11 ldb  -16 ldc smaller than a row  -12 stride_b < 0 */
int igemm(int32_t out_type, int32_t groups, const int32_t* offsets, int64_t M, int64_t N, int64_t K,
          const int8_t* A, int64_t lda, const float* scale_a, const int8_t* B, int64_t ldb,
          int64_t stride_b, const float* scale_b, const float* bias, void* C, int64_t ldc,
          void* stream);

/* Microscaled 4-bit floats (the public OCP format MXFP4).  Every 32 values that
 * follow one another in a row share a scale byte s, which stands for 2^(s - 127)
 * (255: NaN), and are codes of 4 bits: a sign and one of 0, 1/2, 1, 3/2, 2, 3, 4,
 * 6.  A row of K values is (K + 1) / 2 bytes, the even column in a byte's low half,
 * and (K + 31) / 32 scales; rows of scales follow one another without gaps. */

/* Brings every row of X (M x K, of `type`) to microscaled 4-bit floats.  A block's
 * scale is 2^(floor(log2 max|X|) - 2), at least 2^-127, and its codes the nearest
 * to X / scale, ties to the even code, at most 6.  A block of zeros gets scale byte
 * 0, a block that holds an infinity or a NaN scale byte 255 and codes 0, so that
 * its products are NaN throughout.  Where K is odd, the last byte's high half is 0.
 * Weights are brought to 4 bits by the same call, a channel a row.
 * -1 type  -2 M  -3 K negative  -4 X  -6 Q  -8 scale NULL while not empty
 * -5 ldx  -7 ldq (bytes) smaller than a row */
int quantize_mx4(int32_t type, int64_t M, int64_t K, const void* X, int64_t ldx, uint8_t* Q,
                 int64_t ldq, uint8_t* scale, void* stream);

/* C[r,n] = sum_k A[r,k] * B_e[n,k] + bias[e,n] for every row r of every group e, A
 * (M x K) and B_e (N x K) in microscaled 4-bit floats.  lda, ldb and stride_b, the
 * distance of B_e and B_(e+1), are in bytes; scale_a is M rows of scales, scale_b
 * groups x N, bias (or NULL) groups x N, all tight.  Products are exact, sums 32-bit
 * floats, the result is rounded once.  out_type: C's.  K == 0 gives the bias.  Where
 * K is odd, the high half of a row's last byte counts as one more value.
 * -1 out_type  -2 groups < 1, or not 1 without offsets  -4 M  -5 N  -6 K
 * negative  -7 A  -9 scale_a  -10 B  -13 scale_b  -15 C NULL while not empty
 * -8 lda  -11 ldb  -16 ldc smaller than a row  -12 stride_b < 0 */
int gemm_mx4(int32_t out_type, int32_t groups, const int32_t* offsets, int64_t M, int64_t N, int64_t K,
             const uint8_t* A, int64_t lda, const uint8_t* scale_a, const uint8_t* B, int64_t ldb,
             int64_t stride_b, const uint8_t* scale_b, const float* bias, void* C, int64_t ldc,
             void* stream);

/* The tile a product would run with, without a device.  form: 0 gemm_grouped
 * and igemm with transposed weights, 1 gemm_grouped with K x N weights, 2
 * gemm_grouped_wgrad; type: GEMM_*, 3 for igemm, or 5 for gemm_mx4, whose K counts
 * bytes here; out_type: GEMM_*.  Fills
 * tile[0..1] with the output tile's rows and columns and returns the number of
 * workgroups, or -1 for arguments out of range. */
int64_t gemm_grouped_plan(int32_t form, int32_t type, int32_t out_type, int32_t groups, int64_t M,
                          int64_t N, int64_t K, int32_t tile[2]);

/* The same tile's index: 0 256x256, 1 128x128, 2 128x128 with more slices on
 * their way, 3 64x64, 4 16x32, 5 16x16; -1 for arguments out of range. */
int32_t gemm_grouped_tile(int32_t form, int32_t type, int32_t out_type, int32_t groups, int64_t M,
                          int64_t N, int64_t K);

/* The tiles that a form and type can run with: bit i for index i; -1 for
 * arguments out of range. */
int32_t gemm_grouped_tiles(int32_t form, int32_t type);

/* Which outputs each workgroup computes with the tile of index `tile`, without a
 * device: `offsets` is a HOST array here (NULL: one group).  For workgroups
 * first .. first + count - 1 of the launch, order[4 i ..] gets the group (-1:
 * none), the first row (form 2: the row tile), the end of the group's rows
 * (form 2: 0) and the tile's column.  Returns the number of workgroups, or -1
 * for arguments out of range or more workgroups than a launch holds. */
int64_t gemm_grouped_tile_order(int32_t form, int32_t type, int32_t tile, int32_t groups,
                                const int32_t* offsets, int64_t M, int64_t N, int64_t K, int64_t first,
                                int64_t count, int32_t* order);

/* Static string for a status of these calls (never NULL). */
const char* gemm_grouped_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* GROUPED_GEMM_H */
