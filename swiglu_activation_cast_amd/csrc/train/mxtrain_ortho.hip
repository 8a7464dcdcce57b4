// mxtrain_ortho.hip -- C ABI of the orthogonalised updates.
// Nothing is allocated, synchronized or read back, and no exception can leave
// an entry point (nothing here throws).
#include "tr_host.hpp"
#include "tr_ortho_cast.hpp"
#include "tr_ortho_run.hpp"

using namespace mxt;

extern "C" {

int64_t mxtrain_newton_schulz_workspace(int64_t batch, int64_t m, int64_t n, int out_dtype) {
  if (!type_ok(out_dtype) || batch <= 0 || m <= 0 || n <= 0 || batch > kMaxGroups || m >= mxt::kMaxLd ||
      n >= mxt::kMaxLd)
    return 0;
  return std::max<int64_t>(ns_plan(batch, m, n, out_dtype).bytes, 0);
}

mxtrain_status mxtrain_newton_schulz(const void *g, int64_t ld_g, int64_t stride_g, int dtype, int64_t batch,
                                     int64_t m, int64_t n, int steps, const float *coeffs, float eps, void *out,
                                     int64_t ld_out, int64_t stride_out, int out_dtype, void *workspace,
                                     int64_t workspace_bytes, void *stream) {
  if (!type_ok(dtype) || !type_ok(out_dtype)) return MXTRAIN_ERR_TYPE;
  if (!coeffs) return MXTRAIN_ERR_NULL;
  if (steps < 0 || steps > 100 || !(eps >= 0.0f) || std::isinf(eps)) return MXTRAIN_ERR_VALUE;
  for (int i = 0; i < 3; i++)
    if (!std::isfinite(coeffs[i])) return MXTRAIN_ERR_VALUE;
  if (batch < 0 || m < 0 || n < 0 || batch > kMaxGroups || m >= mxt::kMaxLd || n >= mxt::kMaxLd)
    return MXTRAIN_ERR_SHAPE;
  if (batch == 0 || m == 0 || n == 0) return MXTRAIN_OK;
  if (!g || !out || !workspace) return MXTRAIN_ERR_NULL;
  if (ld_g < n || ld_out < n || stride_g < 0 || stride_out < 0) return MXTRAIN_ERR_STRIDE;
  if (!aligned(g, (uintptr_t)size_of(dtype)) || !aligned(out, (uintptr_t)size_of(out_dtype)) || !aligned(workspace, 256))
    return MXTRAIN_ERR_ALIGN;
  int64_t all;
  if (!extent_ok(m, n, ld_g) || !extent_ok(m, n, ld_out) || __builtin_mul_overflow(stride_g, batch, &all) ||
      all > (INT64_MAX >> 4) || __builtin_mul_overflow(stride_out, batch, &all) || all > (INT64_MAX >> 4))
    return MXTRAIN_ERR_OVERFLOW;
  if (batch > 1 && stride_out < (m - 1) * ld_out + n) return MXTRAIN_ERR_STRIDE;
  const NsPlan pl = ns_plan(batch, m, n, out_dtype);
  if (pl.bytes < 0) return MXTRAIN_ERR_OVERFLOW;
  if (workspace_bytes < pl.bytes) return MXTRAIN_ERR_WORKSPACE;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  mxt::NsArgs a{};
  a.g = g;
  a.ld_g = ld_g;
  a.stride_g = stride_g;
  a.rows = m;
  a.cols = n;
  a.batch = batch;
  a.g_f32 = dtype == MXTRAIN_F32;
  const int64_t v = 16 / size_of(dtype);
  a.vec = aligned(g, 16) && ld_g % v == 0 && stride_g % v == 0;
  a.eps = (double)eps;
  a.sums = reinterpret_cast<double *>(ws + pl.sums);
  a.phi = reinterpret_cast<float *>(ws + pl.phi);
  a.x = reinterpret_cast<_Float16 *>(ws + pl.x[0][0]);
  // bf16's eight places fit the high plane: below fp16's normal range, where
  // they do not, the low plane would be zero too
  a.x_lo = pl.split || a.g_f32 ? reinterpret_cast<_Float16 *>(ws + pl.x[0][1]) : nullptr;
  a.ld_x = pl.ld_x;
  a.stride_x = pl.stride_x;
  void *kargs[] = {&a};
  if (hipLaunchKernel((const void *)&mxt::k_ns_norm, dim3(mxt::kNormBlocks, (unsigned)batch), dim3(256), kargs, 0,
                      (hipStream_t)stream) != hipSuccess)
    return MXTRAIN_ERR_LAUNCH;
  const int64_t pieces = (m * (pl.ld_x / 8) + 255) / 256;
  const unsigned grid = (unsigned)std::min<int64_t>(pieces, std::max<int64_t>(1, 2048 / batch));
  if (hipLaunchKernel((const void *)&mxt::k_ns_cast, dim3(grid, (unsigned)batch), dim3(256), kargs, 0,
                      (hipStream_t)stream) != hipSuccess)
    return MXTRAIN_ERR_LAUNCH;
  if (steps == 0) {
    int f32 = out_dtype == MXTRAIN_F32;
    void *pargs[] = {&a, &out, &ld_out, &stride_out, &f32};
    return hipLaunchKernel((const void *)&mxt::k_ns_plain, dim3(grid, (unsigned)batch), dim3(256), pargs, 0,
                           (hipStream_t)stream) == hipSuccess
               ? MXTRAIN_OK
               : MXTRAIN_ERR_LAUNCH;
  }
  return pl.split ? ns_run<true>(pl, a, batch, m, n, steps, coeffs, out, ld_out, stride_out, ws, stream)
                  : ns_run<false>(pl, a, batch, m, n, steps, coeffs, out, ld_out, stride_out, ws, stream);
}

}  // extern "C"
