// mxtrain.hip -- layer norm's C ABI of libmxtrain.so, and the status texts:
// argument checks, the choice of kernel and the launches.
// Nothing is allocated, synchronized or read back, and no exception can leave
// an entry point (nothing here throws).
#include "tr_host.hpp"
#include "tr_norm.hpp"

namespace mxt {
namespace {

// ------------------------------------------------------------- layer norm
// How a row is spread over threads: `tpr` threads (0: a whole workgroup of
// `threads`) holding `elems` elements each; elems == 0: the row does not fit
// registers.
struct RowPlan {
  int tpr, threads, elems;
};

// Short rows share a workgroup of 256 threads (16 or 64 threads a row); a
// longer one has a workgroup of just the wavefronts it needs, with 8 elements a
// thread as long as 1024 threads suffice.  The forward pass over many rows
// prefers 16 elements to more than 512 threads, whose joining costs more than
// it hides (16384 x 8192 bf16: 96 us against 127); the backward pass does not
// (its threads hold five values an element), nor do rows moved by element
// (4096 x 4099: 28 us against 45).
RowPlan row_plan(int64_t M, int64_t N, int vec, bool bwd) {
  const bool many = M >= 1024;
  if (many && N <= 128) return {16, 256, 8};
  if (N <= 512) return {64, 256, 8};
  if (many && N <= 1024) return {64, 256, 16};
  const int cap = many && !bwd && vec > 1 ? 512 : 1024;
  const int64_t chunks = (N + vec - 1) / vec;
  for (int pass = 0; pass < 2; pass++)
    for (int e = 8; e <= 32; e *= 2) {
      if (vec == 1 && e == 32) continue;  // backward: more registers than a thread has; forward: 16 reach as far
      // the kernels' launch bounds
      const int most = bwd ? (e == 8 && vec > 1 ? 1024 : 512) : e <= 16 ? 1024 : 512;
      const int64_t per = e / vec, need = (chunks + per - 1) / per;
      const int64_t t = (need + 63) / 64 * 64;
      if (t <= std::min(pass == 0 ? cap : 1024, most)) return {0, (int)t, e};
    }
  return {0, 1024, 0};
}

// Workgroups of the backward pass, each of which leaves one partial row of
// 2 N sums, of at least four rows each: 512, or 256 where a workgroup has 512
// threads or more (bf16, 16384 rows: of 5120 columns 94 us with 256 workgroups
// and 105 with 512, of 2048 columns 70 and 47).
constexpr int64_t kLnParts = 512;
int64_t ln_parts(int64_t M) { return std::min<int64_t>(kLnParts, (M + 3) / 4); }

// Few enough rows for the column sums to have workgroups of their own in the
// same launch: at most 32 rows to a thread of 512 (1021 x 2049 fp32: 23 us that
// way, 18 with partial rows; 105 x 1818 14 and 18).
bool ln_columns_apart(int64_t M, int64_t N) { return M <= 256 && N <= 8192; }

template <class T, int VEC, int TPR, int E, bool BWD>
const void *ln_pick() {
  if constexpr (BWD) return (const void *)&mxt::k_ln_bwd<T, VEC, TPR, E / VEC>;
  else return (const void *)&mxt::k_ln_fwd<T, VEC, TPR, E / VEC>;
}

template <class T, int VEC, bool BWD>
const void *ln_kernel(const RowPlan &p) {
  if (p.tpr == 16) return ln_pick<T, VEC, 16, 8, BWD>();
  if (p.tpr == 64) return p.elems == 8 ? ln_pick<T, VEC, 64, 8, BWD>() : ln_pick<T, VEC, 64, 16, BWD>();
  if (p.elems == 8) return ln_pick<T, VEC, 0, 8, BWD>();
  // as vectors the backward's 1024 threads of 8 reach as far as its 512 of 16;
  // by element neither pass is planned 32
  if constexpr (VEC == 1) return ln_pick<T, 1, 0, 16, BWD>();
  else if constexpr (BWD) return ln_pick<T, VEC, 0, 32, true>();
  else return p.elems == 16 ? ln_pick<T, VEC, 0, 16, false>() : ln_pick<T, VEC, 0, 32, false>();
}

template <bool BWD>
const void *ln_kernel(const RowPlan &p, int dtype, bool vec) {
  if (p.elems == 0) {
    if constexpr (BWD)
      return dtype == MXTRAIN_F32 ? (const void *)&mxt::k_ln_bwd_long<float> : (const void *)&mxt::k_ln_bwd_long<uint16_t>;
    else
      return dtype == MXTRAIN_F32 ? (const void *)&mxt::k_ln_fwd_long<float> : (const void *)&mxt::k_ln_fwd_long<uint16_t>;
  }
  if (dtype == MXTRAIN_F32) return vec ? ln_kernel<float, 4, BWD>(p) : ln_kernel<float, 1, BWD>(p);
  return vec ? ln_kernel<uint16_t, 8, BWD>(p) : ln_kernel<uint16_t, 1, BWD>(p);
}

// Checks shared by both passes (M > 0, N > 0 from here on).
mxtrain_status ln_check(const void *const *mats, const int64_t *lds, int n, const void *weight, const void *bias,
                        int64_t M, int64_t N, int dtype, int param_dtype) {
  const uintptr_t e = (uintptr_t)size_of(dtype);
  for (int i = 0; i < n; i++)
    if (!mats[i]) return MXTRAIN_ERR_NULL;
  for (int i = 0; i < n; i++)
    if (lds[i] < N) return MXTRAIN_ERR_STRIDE;
  for (int i = 0; i < n; i++)
    if (!aligned(mats[i], e)) return MXTRAIN_ERR_ALIGN;
  if (!aligned(weight, (uintptr_t)size_of(param_dtype)) || !aligned(bias, (uintptr_t)size_of(param_dtype)))
    return MXTRAIN_ERR_ALIGN;
  for (int i = 0; i < n; i++)
    if (!extent_ok(M, N, lds[i])) return MXTRAIN_ERR_OVERFLOW;
  return MXTRAIN_OK;
}

bool ln_vec(const void *const *mats, const int64_t *lds, int n, int64_t N, int dtype) {
  const int v = 16 / size_of(dtype);
  if (N % v != 0) return false;
  for (int i = 0; i < n; i++)
    if (!aligned(mats[i], 16) || lds[i] % v != 0) return false;
  return true;
}

}  // namespace
}  // namespace mxt

using namespace mxt;

extern "C" {

mxtrain_status mxtrain_layer_norm_fwd(const void *x, int64_t ld_x, const void *weight, const void *bias,
                                      int param_dtype, int64_t M, int64_t N, int dtype, float eps, void *y,
                                      int64_t ld_y, float *mean, float *rstd, void *stream) {
  if (!type_ok(dtype) || !type_ok(param_dtype)) return MXTRAIN_ERR_TYPE;
  if (!(eps >= 0.0f) || std::isinf(eps)) return MXTRAIN_ERR_VALUE;
  if (M < 0 || N < 0 || M > INT32_MAX || N > INT32_MAX) return MXTRAIN_ERR_SHAPE;
  if (M == 0) return MXTRAIN_OK;
  if (N == 0) return MXTRAIN_ERR_SHAPE;
  const void *mats[] = {x, y};
  const int64_t lds[] = {ld_x, ld_y};
  const mxtrain_status st = ln_check(mats, lds, 2, weight, bias, M, N, dtype, param_dtype);
  if (st != MXTRAIN_OK) return st;
  if (!aligned(mean, 4) || !aligned(rstd, 4)) return MXTRAIN_ERR_ALIGN;
  const bool vec = ln_vec(mats, lds, 2, N, dtype);
  const RowPlan p = row_plan(M, N, vec ? 16 / size_of(dtype) : 1, false);
  mxt::LnArgs g{};
  g.x = x;
  g.w = weight;
  g.b = bias;
  g.y = y;
  g.ld_x = ld_x;
  g.ld_y = ld_y;
  g.mean = mean;
  g.rstd = rstd;
  g.M = M;
  g.N = (int32_t)N;
  g.w_f32 = param_dtype == MXTRAIN_F32;
  g.p_vec = aligned(weight, 16) && aligned(bias, 16);
  g.eps = eps;
  const int64_t rows = p.tpr ? 256 / p.tpr : 1;
  // About as many workgroups as the CUs hold at once by their registers, each of
  // which then walks rows: 16 or 32 elements a thread leave room for 1024
  // threads to a CU, 8 for 1536 or, moved as vectors, 2048 (16384 x 5120 bf16:
  // 63 us with 1024 threads to a CU, 81 with 1280, more than fit evenly; 16384 x
  // 2048 27 us with 2048, 33 with 1024).  fp32 vectors of 8 elements leave room
  // for 1792 only, and run well with 2048 (16384 x 4096: 90 us, 5.9 TB/s).
  const int per_cu = p.elems > 8 ? 1024 : vec ? 2048 : 1536;
  // (Long rows leave that to the hardware: a workgroup to a row up to the
  // largest launch, then rows are walked too.)
  const int64_t most = p.elems ? cu_count() * std::max<int64_t>(1, per_cu / p.threads) : INT32_MAX / p.threads;
  return launch(ln_kernel<false>(p, dtype, vec), std::min((M + rows - 1) / rows, most), p.threads, g, stream);
}

int64_t mxtrain_layer_norm_bwd_workspace(int64_t M, int64_t N) {
  if (M <= 0 || N <= 0 || M > INT32_MAX || N > INT32_MAX) return 0;
  return ln_columns_apart(M, N) ? 0 : ln_parts(M) * 2 * N * (int64_t)sizeof(float);
}

mxtrain_status mxtrain_layer_norm_bwd(const void *dy, int64_t ld_dy, const void *x, int64_t ld_x, const float *mean,
                                      const float *rstd, const void *weight, int param_dtype, int64_t M, int64_t N,
                                      int dtype, void *dx, int64_t ld_dx, float *dweight, float *dbias,
                                      void *workspace, int64_t workspace_bytes, void *stream) {
  if (!type_ok(dtype) || !type_ok(param_dtype)) return MXTRAIN_ERR_TYPE;
  if (M < 0 || N < 0 || M > INT32_MAX || N > INT32_MAX) return MXTRAIN_ERR_SHAPE;
  if (N == 0) return M == 0 ? MXTRAIN_OK : MXTRAIN_ERR_SHAPE;
  if (!aligned(dweight, 4) || !aligned(dbias, 4)) return MXTRAIN_ERR_ALIGN;
  const bool apart = M > 0 && ln_columns_apart(M, N), sums = (dweight || dbias) && !apart;
  int64_t parts = 0;
  if (M > 0) {
    const void *mats[] = {dy, x, dx};
    const int64_t lds[] = {ld_dy, ld_x, ld_dx};
    if (!mean || !rstd || (sums && !workspace)) return MXTRAIN_ERR_NULL;
    const mxtrain_status st = ln_check(mats, lds, 3, weight, nullptr, M, N, dtype, param_dtype);
    if (st != MXTRAIN_OK) return st;
    if (!aligned(mean, 4) || !aligned(rstd, 4) || (sums && !aligned(workspace, 4))) return MXTRAIN_ERR_ALIGN;
    if (sums && workspace_bytes < mxtrain_layer_norm_bwd_workspace(M, N)) return MXTRAIN_ERR_WORKSPACE;
    const bool vec = ln_vec(mats, lds, 3, N, dtype);
    const RowPlan p = row_plan(M, N, vec ? 16 / size_of(dtype) : 1, true);
    mxt::LnArgs g{};
    g.x = x;
    g.dy = dy;
    g.w = weight;
    g.y = dx;
    g.ld_x = ld_x;
    g.ld_dy = ld_dy;
    g.ld_y = ld_dx;
    g.mean = const_cast<float *>(mean);
    g.rstd = const_cast<float *>(rstd);
    g.part = sums ? static_cast<float *>(workspace) : nullptr;
    g.M = M;
    g.N = (int32_t)N;
    g.w_f32 = param_dtype == MXTRAIN_F32;
    g.p_vec = aligned(weight, 16);
    const int64_t slots = p.tpr ? 256 / p.tpr : 1;
    parts = std::min<int64_t>(ln_parts(M), (M + slots - 1) / slots);
    if (p.threads >= 512) parts = std::min<int64_t>(parts, kLnParts / 2);
    int threads = p.threads;
    int64_t blocks = parts;
    if (apart) {
      // rows by workgroups of 512 threads at least: the columns' take as many
      parts = (M + slots - 1) / slots;
      threads = p.tpr ? p.threads : std::max(p.threads, 512);
      blocks = parts + (dweight || dbias ? (N + 63) / 64 : 0);
      g.dw = dweight;
      g.db = dbias;
    }
    g.row_blocks = parts;
    const unsigned joined = p.tpr && sums ? (unsigned)(slots * 2 * N * (int64_t)sizeof(float)) : 0u;
    const mxtrain_status run = launch(ln_kernel<true>(p, dtype, vec), blocks, threads, g, stream, joined);
    if (run != MXTRAIN_OK) return run;
  }
  if (!sums) return MXTRAIN_OK;
  const float *part = static_cast<const float *>(workspace);
  int n_parts = (int)parts;
  int32_t n = (int32_t)N;
  void *kargs[] = {&part, &n_parts, &n, &dweight, &dbias};
  const int64_t blocks = std::min<int64_t>((2 * N + 31) / 32, INT32_MAX / 1024);
  const hipError_t err = hipLaunchKernel((const void *)&mxt::k_ln_join, dim3((unsigned)blocks), dim3(1024), kargs, 0,
                                         (hipStream_t)stream);
  return err == hipSuccess ? MXTRAIN_OK : MXTRAIN_ERR_LAUNCH;
}

const char *mxtrain_status_str(mxtrain_status status) {
  switch (status) {
    case MXTRAIN_OK: return "ok";
    case MXTRAIN_ERR_NULL: return "a required pointer is NULL";
    case MXTRAIN_ERR_SHAPE: return "a dimension is negative or out of its range";
    case MXTRAIN_ERR_STRIDE: return "a leading dimension is smaller than the row, or not the multiple asked";
    case MXTRAIN_ERR_ALIGN: return "a pointer lacks the alignment asked";
    case MXTRAIN_ERR_TYPE: return "an element type is not one the call takes";
    case MXTRAIN_ERR_OVERFLOW: return "sizes overflow the addressable range or the launch grid";
    case MXTRAIN_ERR_LAUNCH: return "the HIP runtime refused the kernel launch";
    case MXTRAIN_ERR_WORKSPACE: return "the workspace is smaller than the call needs";
    case MXTRAIN_ERR_VALUE: return "a scalar argument is not one the call takes";
  }
  return "unknown status";
}

}  // extern "C"
