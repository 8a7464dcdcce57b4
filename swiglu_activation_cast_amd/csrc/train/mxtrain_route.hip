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
      (need > 0 && !aligned(ws, 16)))
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

// Elements of a piece of rows of H: 16 bytes' worth, or single ones.
int64_t route_vec(int dtype, int64_t H) {
  const int64_t vec = 16 / size_of(dtype);
  return H < vec ? 1 : vec;
}

RouteArgs route_args(const int32_t *rank, int dtype, int64_t T, int64_t k, int64_t H, int64_t R) {
  RouteArgs a{};
  const int64_t vec = route_vec(dtype, H), per = (H + vec - 1) / vec;
  a.rank = rank;
  a.T = T;
  a.k = (u32)k;
  a.H = (u32)H;
  a.R = (u32)R;
  a.pieces = {T * per, divider((uint32_t)per)};
  return a;
}

template <class T, int VEC>
const void *dispatch_kernel(bool nt) {
  if constexpr (VEC > 1)
    if (nt) return (const void *)&k_dispatch<T, VEC, true>;
  return (const void *)&k_dispatch<T, VEC, false>;
}

// wtype: the weights', -1: none.
template <class T, int VEC, bool NT>
const void *combine_kernel_nt(int wtype) {
  return wtype < 0 ? (const void *)&k_combine<T, void, VEC, NT>
         : wtype == MXTRAIN_F32 ? (const void *)&k_combine<T, float, VEC, NT>
                                : (const void *)&k_combine<T, uint16_t, VEC, NT>;
}

template <class T, int VEC>
const void *combine_kernel(int wtype, bool nt) {
  if constexpr (VEC > 1)
    if (nt) return combine_kernel_nt<T, VEC, true>(wtype);
  return combine_kernel_nt<T, VEC, false>(wtype);
}

// lanes: of a token, at least its row's pieces where fewer than 64.
template <class T, class W, int VEC>
const void *combine_bwd_lanes(int lanes, bool nt) {
  if (lanes == 16) return (const void *)&k_combine_bwd<T, W, VEC, 16, false>;
  if (lanes == 32) return (const void *)&k_combine_bwd<T, W, VEC, 32, false>;
  if constexpr (VEC > 1)
    if (nt) return (const void *)&k_combine_bwd<T, W, VEC, 64, true>;
  return (const void *)&k_combine_bwd<T, W, VEC, 64, false>;
}

template <class T, int VEC>
const void *combine_bwd_kernel(int wtype, int lanes, bool nt) {
  return wtype == MXTRAIN_F32 ? combine_bwd_lanes<T, float, VEC>(lanes, nt)
                              : combine_bwd_lanes<T, uint16_t, VEC>(lanes, nt);
}

template <class T, int VEC>
const void *sort_dispatch_kernel(int64_t pairs) {
  return pairs <= 256    ? (const void *)&k_sort_dispatch<T, VEC, 1>
         : pairs <= 1024 ? (const void *)&k_sort_dispatch<T, VEC, 4>
                         : (const void *)&k_sort_dispatch<T, VEC, 8>;
}

// fn<T, VEC>(...) for the rows' type and width.
#define ROUTE_PICK(fn, dtype, H, ...)                                                          \
  (dtype == MXTRAIN_F32 ? (route_vec(dtype, H) > 1 ? fn<float, 4>(__VA_ARGS__) : fn<float, 1>(__VA_ARGS__)) \
                        : (route_vec(dtype, H) > 1 ? fn<uint16_t, 8>(__VA_ARGS__) : fn<uint16_t, 1>(__VA_ARGS__)))

mxtrain_status route_launch(const void *kernel, const RouteArgs &a, void *stream) {
  return launch(kernel, std::min((a.pieces.total + 255) / 256, kMaxGrid), 256, a, stream);
}

// Whether combine and its gradients read past the caches: rows of 128 MB or more
// (half the last level's 256 MB).  Combine of 16384 x 8 rows of 2048 bf16: 126 us
// otherwise, 117 so; 4096 x 8 29 and 26; but 2048 x 8 13.5 and 14.0, and odd fp32
// rows of 43 MB 14.0 and 15.7.  Gradients of 16384 x 8 rows 229 and 223, of 4096 x 8
// 62 and 59, of 2048 x 8 26 and 30.
bool route_past_caches(int dtype, int64_t T, int64_t k, int64_t H) {
  return (double)T * (double)k * (double)H * size_of(dtype) >= (double)(1 << 27);
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
  const bool whole_lines = aligned(xs, 64) && ld_xs * size_of(dtype) % 64 == 0;
  return route_launch(ROUTE_PICK(dispatch_kernel, dtype, H, whole_lines), a, stream);
}

mxtrain_status mxtrain_sort_dispatch(const void *x, int64_t ld_x, int dtype, const void *ids, int64_t ld_ids,
                                     int id_type, int64_t T, int64_t k, int64_t first, int64_t G, int64_t H, void *xs,
                                     int64_t ld_xs, int32_t *rank, int32_t *ends, int32_t *order, void *workspace,
                                     int64_t workspace_bytes, void *stream) {
  mxtrain_status st = sort_check(ids, ld_ids, id_type, T, k, first, G, rank, ends, order, workspace, workspace_bytes);
  if (st != MXTRAIN_OK) return st;
  st = route_check(x, ld_x, xs, ld_xs, dtype, rank, T, k, H, T * k);
  if (st != MXTRAIN_OK) return st;
  const SortPlan sp = sort_plan(T * k, G, false);
  if (T * k > 0 && T * k <= kFewPairs && G <= kFewGroups && H > 0) {
    SortDispatchArgs g{};
    g.sort = sort_args(ids, ld_ids, id_type, T, k, first, G, rank, ends, order);
    g.sort.adjacent = ld_ids == k;
    g.sort.bits = sp.bits;
    g.move = route_args(rank, dtype, T, k, H, T * k);
    g.move.in = x;
    g.move.ld_in = ld_x;
    g.move.out = xs;
    g.move.ld_out = ld_xs;
    // half as many workgroups as run at once, since each begins with a sort: 1000 x 2
    // rows of 4096 bf16 9.0 us, 12.1 with 2048; 2000 x 1 of 8192 fp32 25.4 and 25.0
    const int64_t blocks = std::min<int64_t>((g.move.pieces.total + 255) / 256, 1024);
    return launch(ROUTE_PICK(sort_dispatch_kernel, dtype, H, T * k), blocks, 256, g, stream);
  }
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
  return route_launch(ROUTE_PICK(combine_kernel, dtype, H, weight_type, route_past_caches(dtype, T, k, H)), a, stream);
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
  return route_launch(ROUTE_PICK(combine_kernel, dtype, H, -1, route_past_caches(dtype, T, k, H)), a, stream);
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
  a.dw = dweights;
  if (H == 0) a.pieces.per.d = 0;
  // Wavefronts of a token: about four, so that each walks its pieces in equal
  // steps of one; more, up to one a step, where there are few tokens.
  // (16384 x 8 rows of 2048 bf16: one wavefront 243 us, four 226.  1021 x 2 rows of
  // 2049 fp32: sixteen 18 us, four 13.)
  const int64_t per = a.pieces.per.d;
  const int lanes = per <= 16 ? 16 : per <= 32 ? 32 : 64;
  const bool nt = route_past_caches(dtype, T, k, H);
  if (lanes < 64)
    return launch(ROUTE_PICK(combine_bwd_kernel, dtype, H, weight_type, lanes, nt),
                  std::min((T * lanes + 255) / 256, kMaxGrid), 256, a, stream);
  int64_t steps = std::max<int64_t>(1, (per + 128) / 256);
  while (steps > 1 && T * ((per + 64 * steps - 1) / (64 * steps)) < 1024) steps--;
  const int waves = (int)std::min<int64_t>(16, std::max<int64_t>(1, (per + 64 * steps - 1) / (64 * steps)));
  return launch(ROUTE_PICK(combine_bwd_kernel, dtype, H, weight_type, lanes, nt), std::min(T, kMaxGrid), 64 * waves,
                a, stream);
}

}  // extern "C"
