/*
 * mxtrain.h -- C ABI of libmxtrain.so: the operators of a mixture-of-experts
 * layer's training step that stay in 16 or 32 bits next to the MXFP8 casts
 * and products of mxfp8.h, on MI355X (gfx950).
 *
 * Conventions shared by every call (those of mxfp8.h):
 *  - All data pointers are DEVICE pointers.  bf16 values are raw 16-bit
 *    patterns.  Dimensions, strides and leading dimensions (ld_*) are int64
 *    element counts.  Every matrix is row-major with unit column stride and
 *    the given row stride.
 *  - The caller owns and allocates every buffer, workspaces among them; the
 *    library never allocates, frees, synchronizes or reads device memory
 *    from the host.
 *  - Work is enqueued asynchronously on `stream` (a hipStream_t; NULL is the
 *    default stream), with the stream's device current.  A call that launches
 *    several kernels orders them on that stream.
 *  - Every argument is checked before any launch; a failed check returns a
 *    status and enqueues nothing.
 *  - Outputs and workspaces must not alias inputs or each other (not
 *    checked).  Equal calls give equal bits: nothing is summed in an order
 *    that changes from call to call.  (The order depends on the sizes, on
 *    whether rows start 16-byte aligned, and on the device's compute units.)
 *  - Calls are thread-safe; the library keeps no mutable global state.
 */
#ifndef MXTRAIN_H
#define MXTRAIN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mxtrain_status {
    MXTRAIN_OK = 0,
    MXTRAIN_ERR_NULL = 1,      /* a required pointer is NULL                        */
    MXTRAIN_ERR_SHAPE = 2,     /* a dimension is negative or out of its range       */
    MXTRAIN_ERR_STRIDE = 3,    /* ld smaller than the row, or not the multiple asked */
    MXTRAIN_ERR_ALIGN = 4,     /* a pointer lacks the alignment asked               */
    MXTRAIN_ERR_TYPE = 5,      /* a type code is not one the call takes             */
    MXTRAIN_ERR_OVERFLOW = 6,  /* an extent or the launch grid is too large         */
    MXTRAIN_ERR_LAUNCH = 7,    /* the HIP runtime refused the launch                */
    MXTRAIN_ERR_WORKSPACE = 8, /* the workspace is smaller than the call needs      */
    MXTRAIN_ERR_VALUE = 9      /* a scalar argument is not one the call takes       */
} mxtrain_status;

/* Element types. */
enum { MXTRAIN_BF16 = 0, MXTRAIN_F32 = 1 };

/*
 * Layer norm over the last axis, row i of x [M, N]:
 *   mean = sum_j x_ij / N,  rstd = 1 / sqrt(sum_j (x_ij - mean)^2 / N + eps),
 *   y_ij = (x_ij - mean) rstd weight_j + bias_j.
 *   x, y       : dtype (MXTRAIN_BF16 or MXTRAIN_F32), row strides ld_x, ld_y.
 *   weight, bias : param_dtype [N] each, either may be NULL (ones, zeros).
 *   mean, rstd : fp32 [M], what the backward pass reads; either may be NULL.
 * Computed in fp32, rounded once into y.  Pointers aligned to their element
 * size; rows that all start 16-byte aligned with N a multiple of 16 bytes'
 * worth of elements move 16 bytes at a time, others by element.  eps >= 0 and
 * finite (MXTRAIN_ERR_VALUE).  N >= 1 when M > 0; M, N < 2^31.
 * M == 0 returns MXTRAIN_OK and enqueues nothing.
 */
mxtrain_status mxtrain_layer_norm_fwd(const void *x, int64_t ld_x, const void *weight, const void *bias,
                                      int param_dtype, int64_t M, int64_t N, int dtype, float eps,
                                      void *y, int64_t ld_y, float *mean, float *rstd, void *stream);

/*
 * Gradients of the above for upstream dy [M, N], with xh = (x - mean) rstd
 * and g = dy weight:
 *   dx = rstd (g - sum_j g / N - xh sum_j (g xh) / N),
 *   dweight_j = sum_i dy_ij xh_ij,  dbias_j = sum_i dy_ij.
 *   dy, x, dx : dtype, row strides ld_dy, ld_x, ld_dx.
 *   mean, rstd : fp32 [M], as the forward pass wrote them.
 *   weight    : param_dtype [N] or NULL (ones).
 *   dweight, dbias : fp32 [N]; either may be NULL (not wanted).
 *   workspace : at least mxtrain_layer_norm_bwd_workspace(M, N) bytes (0 for
 *               few rows), 4-byte aligned; may be NULL where that is 0, or
 *               dweight and dbias both are NULL.
 * M == 0 writes zeros into dweight and dbias.
 */
int64_t mxtrain_layer_norm_bwd_workspace(int64_t M, int64_t N);
mxtrain_status mxtrain_layer_norm_bwd(const void *dy, int64_t ld_dy, const void *x, int64_t ld_x,
                                      const float *mean, const float *rstd, const void *weight, int param_dtype,
                                      int64_t M, int64_t N, int dtype, void *dx, int64_t ld_dx,
                                      float *dweight, float *dbias,
                                      void *workspace, int64_t workspace_bytes, void *stream);

/*
 * The experts' products in bf16: the high-precision form of mxfp8.h's grouped
 * products, over the same ragged token groups.  group_ends is a DEVICE int32
 * array of G cumulative end rows, read on the GPU only: group g is rows
 * [end_{g-1}, end_g), with end_g = min(max(group_ends[g], end_{g-1}, 0), M),
 * so that any values give ranges inside the matrices.  Groups may have any
 * number of rows, none among them.
 *
 *   mxtrain_grouped_gemm:    C_g = A_g B_g^T (forward, transpose_b = 1) or
 *                            C_g = A_g B_g (input gradient, transpose_b = 0)
 *   a : bf16 [M, K], row stride lda
 *   b : bf16, expert g at b + g * stride_b: [N, K] (transpose_b = 1) or [K, N]
 *       (transpose_b = 0), row stride ldb
 *   c : c_dtype (MXTRAIN_BF16 or MXTRAIN_F32) [M, N], row stride ldc; rows
 *       past the last group's end are not written.
 *
 *   mxtrain_grouped_gemm_k:  C_g = A_g^T B_g (weight gradient)
 *   a : bf16 [T, M], b : bf16 [T, N] (tokens along the rows; M above is T
 *       here), row strides lda, ldb
 *   c : c_dtype, C_g [M, N] at c + g * stride_c; an empty group gives zeros.
 *
 * Sums are fp32, rounded once into C.  Any dimensions; a and b 16-byte
 * aligned, lda, ldb and stride_b multiples of 8 (16 bytes) and below 2^22
 * (lda, ldb); a single row's stride, a single expert's and those of operands
 * without elements (K == 0) may be any; c aligned to its element.  Elements between a row's end and the
 * next multiple of 8 may be read (never used), nothing else outside the
 * matrices.  0 <= G <= 65535; G == 0, or an empty C, returns MXTRAIN_OK and
 * enqueues nothing.
 */
mxtrain_status mxtrain_grouped_gemm(const void *a, int64_t lda, const void *b, int64_t ldb, int64_t stride_b,
                                    int transpose_b, const int32_t *group_ends, int64_t G,
                                    int64_t M, int64_t N, int64_t K,
                                    void *c, int64_t ldc, int c_dtype, void *stream);
mxtrain_status mxtrain_grouped_gemm_k(const void *a, int64_t lda, const void *b, int64_t ldb,
                                      const int32_t *group_ends, int64_t G, int64_t M, int64_t N, int64_t T,
                                      void *c, int64_t ldc, int64_t stride_c, int c_dtype, void *stream);

/*
 * Orthogonalised updates (Newton-Schulz): for each of `batch` matrices
 * G [m, n],
 *   X = G / (|G| + eps),  |G| = sqrt(sum of squares),
 *   `steps` times  X <- a X + b (X X^T) X + c (X X^T)^2 X,
 * with coeffs = {a, b, c} (HOST memory, read during the call).  Every singular
 * value s of X goes to a s + b s^3 + c s^5 at each step; coefficients like
 * (3.4445, -4.7750, 2.0315) bring five steps' values near 1.
 *   g   : dtype, matrix i at g + i * stride_g, row stride ld_g
 *   out : out_dtype, likewise with stride_out, ld_out
 *   workspace : at least mxtrain_newton_schulz_workspace(...) bytes, 256-byte
 *         aligned.
 * Requires that the steps keep the singular values at most 2 (they start at
 * most 1); a step that leads past that overflows to infinities or NaN.  An
 * fp32 result is computed to about fp32's accuracy; for a bf16 result X is
 * held with 22 significant bits between the products, S = X X^T and the
 * polynomial of it with 11.  A matrix with NaN or infinite
 * entries gives NaN everywhere (steps >= 1); the others of the batch are not
 * touched by it.  A zero matrix gives zeros where eps > 0.
 * Any dimensions (the odd ones and single rows among them) and strides;
 * pointers aligned to their element.  0 <= steps <= 100, eps >= 0, finite
 * coefficients (MXTRAIN_ERR_VALUE); batch <= 65535, m, n < 2^22
 * (MXTRAIN_ERR_SHAPE).  An empty batch or matrix returns MXTRAIN_OK and
 * enqueues nothing.
 */
int64_t mxtrain_newton_schulz_workspace(int64_t batch, int64_t m, int64_t n, int out_dtype);
mxtrain_status mxtrain_newton_schulz(const void *g, int64_t ld_g, int64_t stride_g, int dtype,
                                     int64_t batch, int64_t m, int64_t n, int steps, const float *coeffs, float eps,
                                     void *out, int64_t ld_out, int64_t stride_out, int out_dtype,
                                     void *workspace, int64_t workspace_bytes, void *stream);

/* Static, NUL-terminated description of a status code (never NULL). */
const char *mxtrain_status_str(mxtrain_status status);

#ifdef __cplusplus
}
#endif

#endif /* MXTRAIN_H */
