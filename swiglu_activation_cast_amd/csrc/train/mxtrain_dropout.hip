// mxtrain_dropout.hip -- C ABI of dropout.
// Nothing is allocated, synchronized or read back, and no exception can leave
// an entry point (nothing here throws).
#include "mxtrain_tokens.h"
#include "tr_dropout.hpp"
#include "tr_host.hpp"

using namespace mxt;

namespace mxt {
namespace {

mxtrain_status dropout(const void *x, int64_t ld_x, const void *res, int64_t ld_res, int dtype, int64_t M, int64_t N,
                       double p, uint64_t seed, uint64_t offset, const uint64_t *state, void *y, int64_t ld_y,
                       void *stream) {
  if (!type_ok(dtype)) return MXTRAIN_ERR_TYPE;
  if (!(p >= 0.0 && p <= 1.0)) return MXTRAIN_ERR_VALUE;
  if (M < 0 || N < 0 || M > INT32_MAX || N > INT32_MAX) return MXTRAIN_ERR_SHAPE;
  if (M == 0 || N == 0) return MXTRAIN_OK;
  if (!x || !y) return MXTRAIN_ERR_NULL;
  if (ld_x < N || ld_y < N || (res && ld_res < N)) return MXTRAIN_ERR_STRIDE;
  const uintptr_t e = (uintptr_t)size_of(dtype);
  if (!aligned(x, e) || !aligned(y, e) || !aligned(res, e) || !aligned(state, 8)) return MXTRAIN_ERR_ALIGN;
  if (!extent_ok(M, N, ld_x) || !extent_ok(M, N, ld_y) || (res && !extent_ok(M, N, ld_res)))
    return MXTRAIN_ERR_OVERFLOW;
  DropArgs a{};
  a.x = x;
  a.res = res;
  a.y = y;
  a.ld_x = ld_x;
  a.ld_res = ld_res;
  a.ld_y = ld_y;
  a.N = (u32)N;
  a.border = (u32)std::nearbyint(p * 65536.0);
  a.scale = a.border < 65536u ? (float)(65536.0 / (65536.0 - a.border)) : 0.0f;
  a.seed = seed;
  a.offset = offset;
  a.state = state;
  const int64_t per = (N + 7) / 8;
  a.pieces = {M * per, divider((uint32_t)per)};
  const void *kernel = dtype == MXTRAIN_F32 ? (res ? (const void *)&k_dropout<float, true> : (const void *)&k_dropout<float, false>)
                       : res                ? (const void *)&k_dropout<uint16_t, true>
                                            : (const void *)&k_dropout<uint16_t, false>;
  return launch(kernel, std::min<int64_t>((a.pieces.total + 255) / 256, INT32_MAX / 256), 256, a, stream);
}

}  // namespace
}  // namespace mxt

extern "C" {

mxtrain_status mxtrain_dropout_fwd(const void *x, int64_t ld_x, const void *residual, int64_t ld_res, int dtype,
                                   int64_t M, int64_t N, double p, uint64_t seed, uint64_t offset,
                                   const uint64_t *state, void *y, int64_t ld_y, void *stream) {
  return dropout(x, ld_x, residual, ld_res, dtype, M, N, p, seed, offset, state, y, ld_y, stream);
}

mxtrain_status mxtrain_dropout_bwd(const void *dy, int64_t ld_dy, int dtype, int64_t M, int64_t N, double p,
                                   uint64_t seed, uint64_t offset, const uint64_t *state, void *dx, int64_t ld_dx,
                                   void *stream) {
  return dropout(dy, ld_dy, nullptr, 0, dtype, M, N, p, seed, offset, state, dx, ld_dx, stream);
}

}  // extern "C"
