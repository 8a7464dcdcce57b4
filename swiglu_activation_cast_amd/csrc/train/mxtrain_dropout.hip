// mxtrain_dropout.hip -- C ABI of dropout.
// Nothing is allocated, synchronized or read back, and no exception can leave
// an entry point (nothing here throws).
#include "mxtrain_tokens.h"
#include "tr_dropout.hpp"
#include "tr_host.hpp"

using namespace mxt;

namespace mxt {
namespace {

template <class T>
const void *dropout_kernel(bool res, bool nt) {
  return res ? (nt ? (const void *)&k_dropout<T, true, true> : (const void *)&k_dropout<T, true, false>)
             : (nt ? (const void *)&k_dropout<T, false, true> : (const void *)&k_dropout<T, false, false>);
}

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
  const int64_t vec = 16 / size_of(dtype), per = (N + vec - 1) / vec;
  a.pieces = {M * per, divider((uint32_t)per)};
  // 128 MB or more (half the last-level cache) are read past the caches: 16384 x
  // 8192 bf16 with the residual 131 us so, 136 otherwise; 1021 x 2049 fp32 5.4 and 4.9.
  const bool nt = (double)M * (double)N * size_of(dtype) >= (double)(1 << 27);
  const void *kernel = dtype == MXTRAIN_F32 ? dropout_kernel<float>(res, nt) : dropout_kernel<uint16_t>(res, nt);
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
