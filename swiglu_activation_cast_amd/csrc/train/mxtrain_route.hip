// mxtrain_route.hip -- C ABI of the expert sort, dispatch and combine.
// Nothing is allocated, synchronized or read back, and no exception can leave
// an entry point (nothing here throws).
#include "mxtrain_tokens.h"
#include "tr_route.hpp"
#include "tr_sort_run.hpp"

using namespace mxt;

namespace mxt {
namespace {

constexpr int64_t kMaxGrid = INT32_MAX / 1024;

bool pairs_ok(int64_t T, int64_t k) {
  int64_t n;
  return T >= 0 && k >= 0 && T <= INT32_MAX && k <= INT32_MAX && !__builtin_mul_overflow(T, k, &n) && n <= INT32_MAX;
}

// A matrix [rows, H]: not NULL where it has elements, rows long enough, aligned
// to its element, offsets within 64 bits.
mxtrain_status matrix_check(const void *p, int64_t rows, int64_t H, int64_t ld, int dtype) {
  if (rows == 0 || H == 0) return MXTRAIN_OK;
  if (!p) return MXTRAIN_ERR_NULL;
  if (ld < H) return MXTRAIN_ERR_STRIDE;
  if (!aligned(p, (uintptr_t)size_of(dtype))) return MXTRAIN_ERR_ALIGN;
  return extent_ok(rows, H, ld) ? MXTRAIN_OK : MXTRAIN_ERR_OVERFLOW;
}

mxtrain_status sort_check(const void *ids, int64_t ld, int id_type, int64_t T, int64_t k, int64_t first, int64_t G,
                          const void *rank, const void *ends, const void *order, const void *ws, int64_t ws_bytes) {
  if (id_type != MXTRAIN_I32 && id_type != MXTRAIN_I64) return MXTRAIN_ERR_TYPE;
  if (!pairs_ok(T, k) || G < 0 || G > kMaxGroups) return MXTRAIN_ERR_SHAPE;
  if (first > INT64_MAX - G) return MXTRAIN_ERR_VALUE;
  const int64_t n = T * k, need = mxtrain_expert_sort_workspace(n, G);
  if ((n > 0 && (!ids || !rank)) || (G > 0 && !ends) || (need > 0 && !ws)) return MXTRAIN_ERR_NULL;
  if (n > 0 && ld < k) return MXTRAIN_ERR_STRIDE;
  if (!aligned(ids, id_type == MXTRAIN_I64 ? 8 : 4) || !aligned(rank, 4) || !aligned(ends, 4) || !aligned(order, 4) ||
      (need > 0 && !aligned(ws, 4)))
    return MXTRAIN_ERR_ALIGN;
  if (!extent_ok(T, k, ld)) return MXTRAIN_ERR_OVERFLOW;
  return ws_bytes < need ? MXTRAIN_ERR_WORKSPACE : MXTRAIN_OK;
}

SortArgs sort_args(const void *ids, int64_t ld, int id_type, int64_t T, int64_t k, int64_t first, int64_t G,
                   int32_t *rank, int32_t *ends, int32_t *order) {
  SortArgs a{};
  a.ids = ids;
  a.ld = ld;
  a.first = first;
  a.k = divider((uint32_t)std::max<int64_t>(k, 1));
  a.ids_i64 = id_type == MXTRAIN_I64;
  a.n = (u32)(T * k);
  a.n_keys = (u32)G;
  a.rank = rank;
  a.ends = G > 0 ? ends : nullptr;
  a.order = order;
  return a;
}

// Checks that the moves share: `tokens` [T, H] and `rows` [R, H] by T x k ranks.
mxtrain_status route_check(const void *tokens, int64_t ld_t, const void *rows, int64_t ld_r, int dtype,
                           const void *rank, int64_t T, int64_t k, int64_t H, int64_t R) {
  if (!type_ok(dtype)) return MXTRAIN_ERR_TYPE;
  if (!pairs_ok(T, k) || H < 0 || H > INT32_MAX || R < 0 || R > INT32_MAX) return MXTRAIN_ERR_SHAPE;
  if (T > 0 && k > 0 && !rank) return MXTRAIN_ERR_NULL;
  const mxtrain_status st = matrix_check(tokens, T, H, ld_t, dtype);
  if (st != MXTRAIN_OK) return st;
  if (!aligned(rank, 4)) return MXTRAIN_ERR_ALIGN;
  return matrix_check(rows, R, H, ld_r, dtype);
}

RouteArgs route_args(const int32_t *rank, int dtype, int64_t T, int64_t k, int64_t H, int64_t R) {
  RouteArgs a{};
  const int64_t vec = 16 / size_of(dtype), per = (H + vec - 1) / vec;
  a.rank = rank;
  a.T = T;
  a.k = (u32)k;
  a.H = (u32)H;
  a.R = (u32)R;
  a.pieces = {T * per, divider((uint32_t)per)};
  return a;
}

mxtrain_status route_launch(const void *f32, const void *bf16, int dtype, const RouteArgs &a, void *stream) {
  return launch(dtype == MXTRAIN_F32 ? f32 : bf16, std::min((a.pieces.total + 255) / 256, kMaxGrid), 256, a, stream);
}

}  // namespace
}  // namespace mxt

extern "C" {

int64_t mxtrain_expert_sort_workspace(int64_t pairs, int64_t G) {
  if (pairs < 0 || pairs > INT32_MAX || G < 0 || G > kMaxGroups) return 0;
  return sort_plan(pairs, G, false).bytes;
}

mxtrain_status mxtrain_expert_sort(const void *ids, int64_t ld_ids, int id_type, int64_t T, int64_t k, int64_t first,
                                   int64_t G, int32_t *rank, int32_t *ends, int32_t *order, void *workspace,
                                   int64_t workspace_bytes, void *stream) {
  const mxtrain_status st =
      sort_check(ids, ld_ids, id_type, T, k, first, G, rank, ends, order, workspace, workspace_bytes);
  if (st != MXTRAIN_OK) return st;
  if (T * k == 0 && G == 0) return MXTRAIN_OK;
  return sort_run(sort_plan(T * k, G, false), sort_args(ids, ld_ids, id_type, T, k, first, G, rank, ends, order),
                  static_cast<uint8_t *>(workspace), stream);
}

mxtrain_status mxtrain_dispatch_fwd(const void *x, int64_t ld_x, int dtype, const int32_t *rank, int64_t T, int64_t k,
                                    int64_t H, int64_t R, void *xs, int64_t ld_xs, void *stream) {
  const mxtrain_status st = route_check(x, ld_x, xs, ld_xs, dtype, rank, T, k, H, R);
  if (st != MXTRAIN_OK) return st;
  if (T == 0 || k == 0 || H == 0 || R == 0) return MXTRAIN_OK;
  RouteArgs a = route_args(rank, dtype, T, k, H, R);
  a.in = x;
  a.ld_in = ld_x;
  a.out = xs;
  a.ld_out = ld_xs;
  return route_launch((const void *)&k_dispatch<float>, (const void *)&k_dispatch<uint16_t>, dtype, a, stream);
}

mxtrain_status mxtrain_sort_dispatch(const void *x, int64_t ld_x, int dtype, const void *ids, int64_t ld_ids,
                                     int id_type, int64_t T, int64_t k, int64_t first, int64_t G, int64_t H, void *xs,
                                     int64_t ld_xs, int32_t *rank, int32_t *ends, int32_t *order, void *workspace,
                                     int64_t workspace_bytes, void *stream) {
  mxtrain_status st = sort_check(ids, ld_ids, id_type, T, k, first, G, rank, ends, order, workspace, workspace_bytes);
  if (st != MXTRAIN_OK) return st;
  st = route_check(x, ld_x, xs, ld_xs, dtype, rank, T, k, H, T * k);
  if (st != MXTRAIN_OK) return st;
  st = mxtrain_expert_sort(ids, ld_ids, id_type, T, k, first, G, rank, ends, order, workspace, workspace_bytes, stream);
  return st != MXTRAIN_OK ? st : mxtrain_dispatch_fwd(x, ld_x, dtype, rank, T, k, H, T * k, xs, ld_xs, stream);
}

mxtrain_status mxtrain_combine_fwd(const void *ys, int64_t ld_ys, int dtype, const int32_t *rank, const void *weights,
                                   int weight_type, const void *residual, int64_t ld_res, int64_t T, int64_t k,
                                   int64_t H, int64_t R, void *y, int64_t ld_y, void *stream) {
  if (!type_ok(weight_type)) return MXTRAIN_ERR_TYPE;
  mxtrain_status st = route_check(y, ld_y, ys, ld_ys, dtype, rank, T, k, H, R);
  if (st != MXTRAIN_OK) return st;
  if (T > 0 && k > 0 && !weights) return MXTRAIN_ERR_NULL;
  if (!aligned(weights, (uintptr_t)size_of(weight_type))) return MXTRAIN_ERR_ALIGN;
  if (residual && (st = matrix_check(residual, T, H, ld_res, dtype)) != MXTRAIN_OK) return st;
  if (T == 0 || H == 0) return MXTRAIN_OK;
  RouteArgs a = route_args(rank, dtype, T, k, H, R);
  a.in = ys;
  a.ld_in = ld_ys;
  a.other = residual;
  a.ld_other = ld_res;
  a.out = y;
  a.ld_out = ld_y;
  a.weights = weights;
  a.w_f32 = weight_type == MXTRAIN_F32;
  return route_launch((const void *)&k_combine<float>, (const void *)&k_combine<uint16_t>, dtype, a, stream);
}

mxtrain_status mxtrain_dispatch_bwd(const void *dxs, int64_t ld_dxs, int dtype, const int32_t *rank, int64_t T,
                                    int64_t k, int64_t H, int64_t R, void *dx, int64_t ld_dx, void *stream) {
  const mxtrain_status st = route_check(dx, ld_dx, dxs, ld_dxs, dtype, rank, T, k, H, R);
  if (st != MXTRAIN_OK) return st;
  if (T == 0 || H == 0) return MXTRAIN_OK;
  RouteArgs a = route_args(rank, dtype, T, k, H, R);
  a.in = dxs;
  a.ld_in = ld_dxs;
  a.out = dx;
  a.ld_out = ld_dx;
  return route_launch((const void *)&k_combine<float>, (const void *)&k_combine<uint16_t>, dtype, a, stream);
}

mxtrain_status mxtrain_combine_bwd(const void *dy, int64_t ld_dy, const void *ys, int64_t ld_ys, int dtype,
                                   const int32_t *rank, const void *weights, int weight_type, int64_t T, int64_t k,
                                   int64_t H, int64_t R, void *dys, int64_t ld_dys, float *dweights, void *stream) {
  if (!type_ok(weight_type)) return MXTRAIN_ERR_TYPE;
  mxtrain_status st = route_check(dy, ld_dy, ys, ld_ys, dtype, rank, T, k, H, R);
  if (st != MXTRAIN_OK) return st;
  if (T > 0 && k > 0 && (!weights || !dweights)) return MXTRAIN_ERR_NULL;
  if (!aligned(weights, (uintptr_t)size_of(weight_type)) || !aligned(dweights, 4)) return MXTRAIN_ERR_ALIGN;
  if ((st = matrix_check(dys, R, H, ld_dys, dtype)) != MXTRAIN_OK) return st;
  if (T == 0 || k == 0) return MXTRAIN_OK;
  RouteArgs a = route_args(rank, dtype, T, k, std::max<int64_t>(H, 1), H ? R : 0);  // no columns: dweights are zeros
  a.in = ys;
  a.ld_in = ld_ys;
  a.other = dy;
  a.ld_other = ld_dy;
  a.out = dys;
  a.ld_out = ld_dys;
  a.weights = weights;
  a.w_f32 = weight_type == MXTRAIN_F32;
  a.dw = dweights;
  if (H == 0) a.pieces.per.d = 0;
  return launch(dtype == MXTRAIN_F32 ? (const void *)&k_combine_bwd<float> : (const void *)&k_combine_bwd<uint16_t>,
                std::min((T + 3) / 4, kMaxGrid), 256, a, stream);
}

}  // extern "C"
