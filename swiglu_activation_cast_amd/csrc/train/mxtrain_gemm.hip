// mxtrain_gemm.hip -- C ABI of the experts' products.
// Nothing is allocated, synchronized or read back, and no exception can leave
// an entry point (nothing here throws).
#include "tr_host.hpp"
#include "tr_gemm.hpp"

namespace mxt {
namespace {

// -------------------------------------------------- the experts' products
struct GroupKernel {
  const void *k;
  int bm, bn;
};

template <int MODE, int AL, int BL, int WI, int WJ, int BK, int RING>
GroupKernel group_kernel(bool f32) {
  return {f32 ? (const void *)&mxt::k_group_gemm<MODE, AL, BL, WI, WJ, BK, RING, true>
              : (const void *)&mxt::k_group_gemm<MODE, AL, BL, WI, WJ, BK, RING, false>,
          64 * WI, 64 * WJ};
}

// The tile for `groups` groups of about `rows` rows of C each (as if tokens
// were spread evenly: the real ends are on the device).
//  - 256 x 256 from two thirds of a tile per CU on, unless K is so short that
//    the time is C's (the weight gradient of 61 groups without tokens, 6808 x
//    360: 79 us, with 128 x 128 tiles, two to a CU, 57; at depth 156 they are
//    within 5% of each other, at depth 250 90 us against 107);
//  - 128 x 128 where there is one per CU, or two per CU of groups that fill only
//    half of its rows (32 groups of 47 rows, 2048 x 2048: 70 us, with 64 rows
//    72; input gradient 55 against 65);
//  - else 64 rows: 128 columns from half a tile per CU on (4 groups of 10 rows,
//    input gradient 8192 x 5120: 73 us, with 64 columns 93), or 64 columns,
//    which leave twice as many workgroups to stream (one row, 8192 x 5120: 19 us
//    against 30; 7 groups of 75 rows, 504 columns of depth 5120: 27 against 37,
//    with 128 x 128 tiles 62).
template <int MODE, int AL, int BL>
GroupKernel group_pick(int64_t groups, int64_t rows, int64_t N, int64_t depth, bool f32) {
  auto tiles = [&](int64_t bm, int64_t bn) { return groups * ((rows + bm - 1) / bm) * ((N + bn - 1) / bn); };
  const int64_t cus = cu_count();
  if (rows > 128 && depth > 64 && tiles(256, 256) >= cus * 2 / 3) return group_kernel<MODE, AL, BL, 4, 4, 64, 2>(f32);
  if (rows > 32 && tiles(128, 128) >= (rows > 64 ? cus : 2 * cus)) return group_kernel<MODE, AL, BL, 2, 2, 64, 2>(f32);
  if (tiles(64, 128) >= cus / 2) return group_kernel<MODE, AL, BL, 1, 2, 64, 3>(f32);
  return group_kernel<MODE, AL, BL, 1, 1, 64, 4>(f32);
}

// Rows of an operand start 16 bytes apart; nothing is read through the stride
// of a single row, or of a matrix without elements.
mxtrain_status operand_check(const void *p, int64_t ld, int64_t rows, int64_t cols) {
  if (rows == 0 || cols == 0) return MXTRAIN_OK;
  if (ld < cols || (rows > 1 && ld % 8 != 0)) return MXTRAIN_ERR_STRIDE;
  if (!aligned(p, 16)) return MXTRAIN_ERR_ALIGN;
  if (ld >= mxt::kMaxLd || !extent_ok(rows, cols, ld)) return MXTRAIN_ERR_OVERFLOW;
  return MXTRAIN_OK;
}

}  // namespace
}  // namespace mxt

using namespace mxt;

extern "C" {

mxtrain_status mxtrain_grouped_gemm(const void *a, int64_t lda, const void *b, int64_t ldb, int64_t stride_b,
                                    int transpose_b, const int32_t *group_ends, int64_t G, int64_t M, int64_t N,
                                    int64_t K, void *c, int64_t ldc, int c_dtype, void *stream) {
  if (!type_ok(c_dtype)) return MXTRAIN_ERR_TYPE;
  if (transpose_b != 0 && transpose_b != 1) return MXTRAIN_ERR_VALUE;
  if (G < 0 || G > kMaxGroups || M < 0 || N < 0 || K < 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX)
    return MXTRAIN_ERR_SHAPE;
  if (G == 0 || M == 0 || N == 0) return MXTRAIN_OK;
  if (!group_ends || !c || (K > 0 && (!a || !b))) return MXTRAIN_ERR_NULL;
  const int64_t b_rows = transpose_b ? N : K, b_cols = transpose_b ? K : N;
  mxtrain_status st = operand_check(a, lda, M, K);
  if (st == MXTRAIN_OK) st = operand_check(b, ldb, b_rows, b_cols);
  if (st != MXTRAIN_OK) return st;
  int64_t all;
  if (stride_b < 0 || ldc < N) return MXTRAIN_ERR_STRIDE;
  if (G > 1 && K > 0 && (stride_b % 8 != 0 || stride_b < (b_rows - 1) * ldb + b_cols)) return MXTRAIN_ERR_STRIDE;
  if (!aligned(group_ends, 4) || !aligned(c, (uintptr_t)size_of(c_dtype))) return MXTRAIN_ERR_ALIGN;
  if (!extent_ok(M, N, ldc) || __builtin_mul_overflow(stride_b, G, &all) || all > (INT64_MAX >> 4))
    return MXTRAIN_ERR_OVERFLOW;
  const bool f32 = c_dtype == MXTRAIN_F32;
  const int64_t groups = std::min(G, M), rows = (M + groups - 1) / groups;  // as if evenly spread
  const GroupKernel k = transpose_b ? group_pick<mxt::kGroupM, mxt::kKC, mxt::kKC>(groups, rows, N, K, f32)
                                    : group_pick<mxt::kGroupM, mxt::kKC, mxt::kMC>(groups, rows, N, K, f32);
  // an upper bound of tile rows, each group that has rows (M of them at most)
  // adding at most one partial one: the host never reads the ends
  const int64_t tiles_m = (M + k.bm - 1) / k.bm + groups, tiles_n = (N + k.bn - 1) / k.bn;
  int64_t blocks;
  if (__builtin_mul_overflow(tiles_m, tiles_n, &blocks)) return MXTRAIN_ERR_OVERFLOW;
  mxt::GemmArgs g{};
  g.cus = cu_count();
  if (k.bm == 256) blocks = mxt::work_items_bound(blocks, g.cus);
  g.a = static_cast<const uint16_t *>(a);
  g.b = static_cast<const uint16_t *>(b);
  g.lda = lda;
  g.ldb = ldb;
  g.stride_b = stride_b;
  g.M = M;
  g.N = N;
  g.K = K;
  g.c = c;
  g.ldc = ldc;
  g.ends = group_ends;
  g.G = (int32_t)G;
  g.tiles_m = (int32_t)tiles_m;
  g.tiles_n = (int32_t)tiles_n;
  g.vec_c = vec_c_ok(c, ldc, 0, c_dtype);
  return launch(k.k, blocks, mxt::kThreads, g, stream);
}

mxtrain_status mxtrain_grouped_gemm_k(const void *a, int64_t lda, const void *b, int64_t ldb,
                                      const int32_t *group_ends, int64_t G, int64_t M, int64_t N, int64_t T, void *c,
                                      int64_t ldc, int64_t stride_c, int c_dtype, void *stream) {
  if (!type_ok(c_dtype)) return MXTRAIN_ERR_TYPE;
  if (G < 0 || G > kMaxGroups || M < 0 || N < 0 || T < 0 || M > INT32_MAX || N > INT32_MAX || T > INT32_MAX)
    return MXTRAIN_ERR_SHAPE;
  if (G == 0 || M == 0 || N == 0) return MXTRAIN_OK;
  if (!group_ends || !c || (T > 0 && (!a || !b))) return MXTRAIN_ERR_NULL;
  mxtrain_status st = operand_check(a, lda, T, M);
  if (st == MXTRAIN_OK) st = operand_check(b, ldb, T, N);
  if (st != MXTRAIN_OK) return st;
  int64_t all;
  if (ldc < N || stride_c < 0) return MXTRAIN_ERR_STRIDE;
  if (!aligned(group_ends, 4) || !aligned(c, (uintptr_t)size_of(c_dtype))) return MXTRAIN_ERR_ALIGN;
  if (!extent_ok(M, N, ldc) || __builtin_mul_overflow(stride_c, G, &all) || all > (INT64_MAX >> 4))
    return MXTRAIN_ERR_OVERFLOW;
  if (G > 1 && stride_c < (M - 1) * ldc + N) return MXTRAIN_ERR_STRIDE;
  const GroupKernel k = group_pick<mxt::kGroupK, mxt::kMC, mxt::kMC>(G, M, N, T / G, c_dtype == MXTRAIN_F32);
  const int64_t tiles_m = (M + k.bm - 1) / k.bm, tiles_n = (N + k.bn - 1) / k.bn;
  int64_t blocks;
  if (__builtin_mul_overflow(tiles_m, tiles_n, &blocks) || __builtin_mul_overflow(blocks, G, &blocks))
    return MXTRAIN_ERR_OVERFLOW;
  mxt::GemmArgs g{};
  g.cus = cu_count();
  if (k.bm == 256) blocks = mxt::work_items(blocks, g.cus);
  g.a = static_cast<const uint16_t *>(a);
  g.b = static_cast<const uint16_t *>(b);
  g.lda = lda;
  g.ldb = ldb;
  g.M = M;
  g.N = N;
  g.K = T;
  g.c = c;
  g.ldc = ldc;
  g.stride_c = stride_c;
  g.ends = group_ends;
  g.G = (int32_t)G;
  g.tiles_m = (int32_t)tiles_m;
  g.tiles_n = (int32_t)tiles_n;
  g.vec_c = vec_c_ok(c, ldc, stride_c, c_dtype);
  return launch(k.k, blocks, mxt::kThreads, g, stream);
}

}  // extern "C"
