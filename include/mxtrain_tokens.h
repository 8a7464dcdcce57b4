/*
 * mxtrain_tokens.h -- C ABI of libmxtrain.so, second part: the operators that
 * bring tokens to the experts of a layer and back, embedding lookup, and
 * dropout, forward and backward, on MI355X (gfx950).
 *
 * The conventions are those of mxtrain.h: device pointers, int64 element
 * counts and row strides (ld_*, unit column stride), the caller's workspaces,
 * work enqueued on `stream` with its device current, every argument checked
 * before any launch, no aliasing of outputs with inputs, equal calls give equal
 * bits, thread-safe.  Element types are MXTRAIN_BF16 and MXTRAIN_F32; all
 * sums are fp32, rounded once.  Pointers and strides need no more alignment than
 * their element.  Values of index arrays never lead outside the
 * matrices, whatever they are.
 */
#ifndef MXTRAIN_TOKENS_H
#define MXTRAIN_TOKENS_H

#include "mxtrain.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Integer types of expert and token numbers. */
enum { MXTRAIN_I32 = 0, MXTRAIN_I64 = 1 };

/*
 * Stable sort of token-expert pairs by expert.  Pair p = t k + j is choice j of
 * token t; it belongs to group g = ids[t][j] - first and is dropped where g is
 * not in [0, G) (an expert held elsewhere, or -1 for none).
 *   ids   : id_type [T, k], row stride ld_ids
 *   rank  : int32 [T k], the row of pair p among the kept pairs in order of
 *           (group, p), or -1 where it is dropped
 *   ends  : int32 [G], cumulative end rows of the groups: the group_ends of the
 *           grouped products
 *   order : int32 [T k], the pair in each row, -1 in rows past the last; may
 *           be NULL
 *   workspace : at least mxtrain_expert_sort_workspace(T k, G) bytes (0 for few
 *           pairs, then it may be NULL), 16-byte aligned
 * T k < 2^31, G <= 65535; G == 0 drops every pair, T k == 0 leaves zeros in ends.
 */
int64_t mxtrain_expert_sort_workspace(int64_t pairs, int64_t G);
mxtrain_status mxtrain_expert_sort(const void *ids, int64_t ld_ids, int id_type, int64_t T, int64_t k, int64_t first,
                                   int64_t G, int32_t *rank, int32_t *ends, int32_t *order, void *workspace,
                                   int64_t workspace_bytes, void *stream);

/*
 * Rows moved to the places that `rank` names: xs[rank[t][j]] = x[t].
 *   x    : dtype [T, H], row stride ld_x
 *   rank : int32 [T, k], adjacent; values outside [0, R) are dropped pairs, the
 *          others distinct
 *   xs   : dtype [R, H], row stride ld_xs; rows that no pair names are not written
 * mxtrain_sort_dispatch is the sort above and this in one call (R = T k; one
 * launch where there are few pairs); order may be NULL.
 * mxtrain_dispatch_bwd is the gradient: dx[t] = sum_j dxs[rank[t][j]], in the
 * order of j, zeros where every pair of a token is dropped.
 * T, k, H, R < 2^31, T k < 2^31.
 */
mxtrain_status mxtrain_dispatch_fwd(const void *x, int64_t ld_x, int dtype, const int32_t *rank, int64_t T, int64_t k,
                                    int64_t H, int64_t R, void *xs, int64_t ld_xs, void *stream);
mxtrain_status mxtrain_sort_dispatch(const void *x, int64_t ld_x, int dtype, const void *ids, int64_t ld_ids,
                                     int id_type, int64_t T, int64_t k, int64_t first, int64_t G, int64_t H, void *xs,
                                     int64_t ld_xs, int32_t *rank, int32_t *ends, int32_t *order, void *workspace,
                                     int64_t workspace_bytes, void *stream);
mxtrain_status mxtrain_dispatch_bwd(const void *dxs, int64_t ld_dxs, int dtype, const int32_t *rank, int64_t T,
                                    int64_t k, int64_t H, int64_t R, void *dx, int64_t ld_dx, void *stream);

/*
 * The experts' rows weighted and summed back:
 *   y[t] = residual[t] + sum_j weights[t][j] ys[rank[t][j]],
 * over the kept pairs in the order of j.
 *   ys       : dtype [R, H], row stride ld_ys; rows that no pair names are not read
 *   weights  : weight_type [T, k], adjacent
 *   residual : dtype [T, H], row stride ld_res, or NULL (zeros)
 *   y        : dtype [T, H], row stride ld_y
 * The gradients for upstream dy [T, H] (residual's is dy itself):
 *   dys[rank[t][j]] = weights[t][j] dy[t]; rows that no pair names are not written
 *   dweights[t][j]  = sum_h dy[t][h] ys[rank[t][j]][h], fp32 [T, k], 0 for dropped pairs
 */
mxtrain_status mxtrain_combine_fwd(const void *ys, int64_t ld_ys, int dtype, const int32_t *rank, const void *weights,
                                   int weight_type, const void *residual, int64_t ld_res, int64_t T, int64_t k,
                                   int64_t H, int64_t R, void *y, int64_t ld_y, void *stream);
mxtrain_status mxtrain_combine_bwd(const void *dy, int64_t ld_dy, const void *ys, int64_t ld_ys, int dtype,
                                   const int32_t *rank, const void *weights, int weight_type, int64_t T, int64_t k,
                                   int64_t H, int64_t R, void *dys, int64_t ld_dys, float *dweights, void *stream);

/*
 * Embedding lookup: y[t] = scale weight[ids[t] - first], zeros where
 * ids[t] - first is not in [0, V) (a word held elsewhere, or padding).
 *   weight : weight_type [V, H], row stride ld_w
 *   ids    : id_type [T], id_stride elements apart
 *   y      : y_type [T, H], row stride ld_y
 * Its gradient, dweight[v] = scale sum over t with ids[t] - first = v of dy[t]:
 *   accumulate == 0 writes every row of dweight (zeros where no token has that word),
 *   accumulate == 1 adds to the rows that tokens name and leaves the others alone.
 *   dy        : dy_type [T, H], row stride ld_dy
 *   dweight   : dw_type [V, H], row stride ld_dw
 *   workspace : at least mxtrain_embedding_bwd_workspace(T, V, H, dy_type, dw_type)
 *               bytes (0 for few tokens, then it may be NULL, and for sizes that are
 *               refused), 16-byte aligned
 * A word's rows are summed in a fixed order: parts of at most 64 rows, each in the
 * order of the tokens, then every fourth part, then the four sums, each in order.
 * scale is finite (MXTRAIN_ERR_VALUE).  T, V, H < 2^31; in the gradient
 * ceil(T / 64) times the strips of a row, 256 columns of fp32 into fp32, 512
 * otherwise, at most 2^23 - 1 (MXTRAIN_ERR_OVERFLOW).
 */
mxtrain_status mxtrain_embedding_fwd(const void *weight, int64_t ld_w, int weight_type, int64_t V, int64_t H,
                                     const void *ids, int64_t id_stride, int id_type, int64_t T, int64_t first,
                                     float scale, void *y, int64_t ld_y, int y_type, void *stream);
int64_t mxtrain_embedding_bwd_workspace(int64_t T, int64_t V, int64_t H, int dy_type, int dw_type);
mxtrain_status mxtrain_embedding_bwd(const void *dy, int64_t ld_dy, int dy_type, const void *ids, int64_t id_stride,
                                     int id_type, int64_t T, int64_t first, float scale, int64_t V, int64_t H,
                                     void *dweight, int64_t ld_dw, int dw_type, int accumulate, void *workspace,
                                     int64_t workspace_bytes, void *stream);

/*
 * Dropout: y = residual + (kept ? x 65536 / (65536 - t) : 0) with t = p 65536
 * rounded to a whole number (halves to even), so that an element is dropped with
 * probability t / 65536 and the mean of y is the input's.  Whether element
 * (i, c) is kept is never stored: it is when its 16 random bits are t or more,
 * which are half c % 2 (0: the low one) of word c / 2 % 4 of the
 * Philox4x32-10 block (Salmon, Moraes, Dror and Shaw, "Parallel random numbers:
 * as easy as 1, 2, 3", 2011) at
 *   counter = (c / 8, i, offset's low word, offset's high word),
 *   key     = (seed's low word, seed's high word).
 * So every call needs an offset of its own under one seed; calls with the same
 * seed, offset and p have the same mask, whatever type, strides or number of
 * rows.  The gradient is the same mask on dy (residual's gradient is dy).
 *   x, residual, y : dtype [M, N], row strides ld_*; residual may be NULL (zeros)
 *   state : NULL, or two uint64 on the DEVICE that are added to seed and offset
 *           (mod 2^64): a captured graph draws new masks when they change
 * 0 <= p <= 1 (MXTRAIN_ERR_VALUE); what is dropped counts as zero, also where it
 * is infinite or NaN.  M, N < 2^31.
 */
mxtrain_status mxtrain_dropout_fwd(const void *x, int64_t ld_x, const void *residual, int64_t ld_res, int dtype,
                                   int64_t M, int64_t N, double p, uint64_t seed, uint64_t offset,
                                   const uint64_t *state, void *y, int64_t ld_y, void *stream);
mxtrain_status mxtrain_dropout_bwd(const void *dy, int64_t ld_dy, int dtype, int64_t M, int64_t N, double p,
                                   uint64_t seed, uint64_t offset, const uint64_t *state, void *dx, int64_t ld_dx,
                                   void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MXTRAIN_TOKENS_H */
