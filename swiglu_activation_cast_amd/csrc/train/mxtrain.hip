// mxtrain.hip -- C ABI of libmxtrain.so: argument checks, the choice of kernel
// and the launches.  Nothing is allocated, synchronized or read back, and no
// exception can leave an entry point (nothing here throws).
#include <hip/hip_runtime.h>
#include <algorithm>
#include <cmath>
#include <limits.h>
#include <stdint.h>

#include "mxtrain.h"
#include "tr_gemm.hpp"
#include "tr_norm.hpp"
#include "tr_ortho.hpp"

namespace {

bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Elements of a [rows, cols] matrix with row stride ld, counted from its
// base, fit int64 with room for the element size and a batch on top.
bool extent_ok(int64_t rows, int64_t cols, int64_t ld) {
  int64_t r;
  if (rows == 0 || cols == 0) return true;
  return !__builtin_mul_overflow(rows - 1, ld, &r) && !__builtin_add_overflow(r, cols, &r) && r < (INT64_MAX >> 4);
}

template <class Args>
mxtrain_status launch(const void *kernel, int64_t blocks, int threads, const Args &a, void *stream, unsigned lds = 0) {
  // grid x times block x stays below 2^31
  if (blocks <= 0 || blocks > (int64_t)INT32_MAX / threads) return MXTRAIN_ERR_OVERFLOW;
  Args copy = a;
  void *kargs[] = {&copy};
  const hipError_t err =
      hipLaunchKernel(kernel, dim3((unsigned)blocks), dim3((unsigned)threads), kargs, lds, (hipStream_t)stream);
  return err == hipSuccess ? MXTRAIN_OK : MXTRAIN_ERR_LAUNCH;
}

// Compute units of the current device (it decides tile sizes, no result
// depends on it).
int cu_count() {
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus < 1)
    return 256;
  return cus;
}

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
      if (bwd && vec == 1 && e == 32) continue;  // more registers than a thread has
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
  if (p.elems == 16) return ln_pick<T, VEC, 0, 16, BWD>();
  if constexpr (BWD && VEC == 1) return nullptr;  // not planned
  else return ln_pick<T, VEC, 0, 32, BWD>();
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

bool type_ok(int t) { return t == MXTRAIN_BF16 || t == MXTRAIN_F32; }
int size_of(int t) { return t == MXTRAIN_F32 ? 4 : 2; }

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

// -------------------------------------------------- the experts' products
constexpr int64_t kMaxGroups = 65535;

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
//  - 256 x 256 from two thirds of a tile per CU on;
//  - 128 x 128 where there is one per CU, or two per CU of groups that fill only
//    half of its rows (32 groups of 47 rows, 2048 x 2048: 70 us, with 64 rows
//    72; input gradient 55 against 65);
//  - else 64 rows: 128 columns from half a tile per CU on (4 groups of 10 rows,
//    input gradient 8192 x 5120: 73 us, with 64 columns 93), or 64 columns,
//    which leave twice as many workgroups to stream (one row, 8192 x 5120: 19 us
//    against 30; 7 groups of 75 rows, 504 columns of depth 5120: 27 against 37,
//    with 128 x 128 tiles 62).
template <int MODE, int AL, int BL>
GroupKernel group_pick(int64_t groups, int64_t rows, int64_t N, bool f32) {
  auto tiles = [&](int64_t bm, int64_t bn) { return groups * ((rows + bm - 1) / bm) * ((N + bn - 1) / bn); };
  const int64_t cus = cu_count();
  if (rows > 128 && tiles(256, 256) >= cus * 2 / 3) return group_kernel<MODE, AL, BL, 4, 4, 64, 2>(f32);
  if (rows > 32 && tiles(128, 128) >= (rows > 64 ? cus : 2 * cus)) return group_kernel<MODE, AL, BL, 2, 2, 64, 2>(f32);
  if (tiles(64, 128) >= cus / 2) return group_kernel<MODE, AL, BL, 1, 2, 64, 3>(f32);
  return group_kernel<MODE, AL, BL, 1, 1, 64, 4>(f32);
}

mxtrain_status operand_check(const void *p, int64_t ld, int64_t rows, int64_t cols) {
  if (ld < cols || ld % 8 != 0) return MXTRAIN_ERR_STRIDE;
  if (!aligned(p, 16)) return MXTRAIN_ERR_ALIGN;
  if (ld >= mxt::kMaxLd || !extent_ok(rows, cols, ld)) return MXTRAIN_ERR_OVERFLOW;
  return MXTRAIN_OK;
}

bool vec_c_ok(const void *c, int64_t ldc, int64_t stride_c, int type) {
  const int64_t v = 16 / size_of(type);
  return aligned(c, 16) && ldc % v == 0 && stride_c % v == 0;
}

// ------------------------------------------------------- orthogonalisation
// Workspace: the fp16 planes of X (two, in turn), S and p(S), then the sums
// of squares and phi.  Every part starts at a multiple of 256 bytes.
struct NsPlan {
  bool split, tall;
  int64_t s;             // the shorter side
  int64_t ld_x, stride_x, ld_s, stride_s;
  int64_t x[2][2], sq[2][2];  // byte offsets: [which][plane]; sq: S, p(S)
  int64_t sums, phi, bytes;   // bytes < 0: too large
};

NsPlan ns_plan(int64_t batch, int64_t m, int64_t n, int out_dtype) {
  NsPlan p{};
  p.split = out_dtype == MXTRAIN_F32;
  p.tall = m > n;
  p.s = std::min(m, n);
  p.ld_x = (n + 7) / 8 * 8;
  p.stride_x = m * p.ld_x;
  p.ld_s = (p.s + 7) / 8 * 8;
  p.stride_s = p.s * p.ld_s;
  int64_t at = 0;
  bool ok = true;
  auto take = [&](int64_t elems, int64_t size) {
    const int64_t here = at;
    int64_t b;
    ok = ok && !__builtin_mul_overflow(elems, size * batch, &b) && b < (INT64_MAX >> 8);
    if (ok) at += (b + 255) / 256 * 256;
    return here;
  };
  for (int which = 0; which < 2; which++)
    for (int plane = 0; plane < (p.split ? 2 : 1); plane++) {
      p.x[which][plane] = take(p.stride_x, 2);
      p.sq[which][plane] = take(p.stride_s, 2);
    }
  p.sums = take(mxt::kNormBlocks, 8);
  p.phi = take(1, 4);
  p.bytes = ok ? at : -1;
  return p;
}

template <int STEP, int AL, int BL, bool SPLIT>
mxtrain_status ns_gemm(mxt::NsGemm &p, int64_t batch, void *stream) {
  constexpr bool sym = STEP == mxt::kGram || STEP == mxt::kPoly;
  auto tiles = [&](int64_t b) {
    const int64_t tm = (p.g.M + b - 1) / b, tn = (p.g.N + b - 1) / b;
    return batch * (sym ? tm * (tm + 1) / 2 : tm * tn);
  };
  const int64_t cus = cu_count();
  // Time in units of a round of 256 x 256 tiles, one per CU: a last partial
  // round runs cut down unless the product is symmetric; 128 x 128 tiles run
  // two to a CU.  Five steps with one tile throughout and as chosen here, us:
  //                            256    128     64   chosen
  //   1 x 256 x 512 fp32       423    204    107      107
  //   8 x 2048 x 1024 bf16     629    465    838      424
  //   1 x 2048 x 2048 bf16     676    411    502      423
  //   4 x 2048 x 2048 bf16     842    940   1586      821
  //   1 x 8192 x 1024 bf16    1057    658    431      315
  //   1 x 8192 x 5120 fp32    9242  11154  16711     9180
  auto cost256 = [&] {
    const int64_t t = tiles(256), whole = t / cus, tail = t % cus;
    if (sym) return (double)((t + cus - 1) / cus);
    return whole + (tail == 0 ? 0.0 : tail <= cus / 4 ? 0.35 : tail <= cus / 2 ? 0.6 : 1.0);
  };
  auto cost128 = [&] {
    const int64_t t = tiles(128);
    return t <= cus ? 0.42 : 0.67 * (double)((t + 2 * cus - 1) / (2 * cus));
  };
  auto cost64 = [&] { return 0.2 * (double)((tiles(64) + cus - 1) / cus); };
  const double c256 = cost256(), c128 = cost128(), c64 = cost64();
  const int64_t b = c256 <= c128 && c256 <= c64 ? 256 : c128 <= c64 ? 128 : 64;
  p.g.tiles_m = (int32_t)((p.g.M + b - 1) / b);
  p.g.tiles_n = (int32_t)((p.g.N + b - 1) / b);
  p.g.G = (int32_t)batch;
  p.g.cus = (int32_t)cus;
  int64_t blocks = tiles(b);
  if (b == 256 && !sym) blocks = mxt::work_items(blocks, cus);
  const void *k = b == 256   ? (const void *)&mxt::k_ns_gemm<STEP, AL, BL, 4, 4, SPLIT ? 32 : 64, 2, SPLIT>
                  : b == 128 ? (const void *)&mxt::k_ns_gemm<STEP, AL, BL, 2, 2, SPLIT ? 32 : 64, 2, SPLIT>
                             : (const void *)&mxt::k_ns_gemm<STEP, AL, BL, 1, 1, 64, SPLIT ? 4 : 8, SPLIT>;
  return launch(k, blocks, mxt::kThreads, p, stream);
}

template <bool SPLIT>
mxtrain_status ns_run(const NsPlan &pl, mxt::NsArgs n, int64_t batch, int64_t m, int64_t cols, int steps,
                      const float *co, void *out, int64_t ld_out, int64_t stride_out, uint8_t *ws, void *stream) {
  auto plane = [&](const int64_t *off, int i) { return reinterpret_cast<_Float16 *>(ws + off[i]); };
  auto bits = [](const _Float16 *p) { return reinterpret_cast<const uint16_t *>(p); };
  // p(S) is held times the largest power of two that keeps |a| + 4 |b| + 16 |c|
  // (its bound for singular values up to 2) below fp16's largest number
  const float most = std::max(std::fabs(co[0]) + 4 * std::fabs(co[1]) + 16 * std::fabs(co[2]), 1e-30f);
  const float ps = std::ldexp(1.0f, std::min(14, std::max(-100, std::ilogb(60000.0f / most))));
  mxtrain_status st = MXTRAIN_OK;
  for (int step = 0; step < steps; step++) {
    const int cur = step & 1;
    const bool last = step == steps - 1;
    const _Float16 *x = plane(pl.x[cur], 0), *x_lo = SPLIT ? plane(pl.x[cur], 1) : nullptr;
    _Float16 *s = plane(pl.sq[0], 0), *s_lo = SPLIT ? plane(pl.sq[0], 1) : nullptr;
    _Float16 *q = plane(pl.sq[1], 0), *q_lo = SPLIT ? plane(pl.sq[1], 1) : nullptr;
    mxt::NsGemm gram{}, poly{}, next{};
    gram.g.a = gram.g.b = bits(x);
    gram.a_lo = gram.b_lo = bits(x_lo);
    gram.g.lda = gram.g.ldb = pl.ld_x;
    gram.g.stride_a = gram.g.stride_b = pl.stride_x;
    gram.g.M = gram.g.N = pl.s;
    gram.g.K = pl.tall ? m : cols;
    gram.g.c = s;
    gram.c_lo = s_lo;
    gram.g.ldc = pl.ld_s;
    gram.g.stride_c = pl.stride_s;
    gram.scale = mxt::kSScale / (mxt::kXScale * mxt::kXScale);
    poly.g.a = poly.g.b = bits(s);
    poly.a_lo = poly.b_lo = bits(s_lo);
    poly.s = s;
    poly.s_lo = s_lo;
    poly.g.lda = poly.g.ldb = poly.g.ldc = pl.ld_s;
    poly.g.stride_a = poly.g.stride_b = poly.g.stride_c = pl.stride_s;
    poly.g.M = poly.g.N = poly.g.K = pl.s;
    poly.g.c = q;
    poly.c_lo = q_lo;
    poly.phi = step == 0 ? n.phi : nullptr;
    poly.ca = co[0] * ps;
    poly.cb = co[1] * ps / mxt::kSScale;
    poly.cc = co[2] * ps / (mxt::kSScale * mxt::kSScale);
    const uint16_t *hx = bits(x), *hq = bits(q), *lx = bits(x_lo), *lq = bits(q_lo);
    next.g.a = pl.tall ? hx : hq;
    next.a_lo = pl.tall ? lx : lq;
    next.g.b = pl.tall ? hq : hx;
    next.b_lo = pl.tall ? lq : lx;
    next.g.lda = pl.tall ? pl.ld_x : pl.ld_s;
    next.g.stride_a = pl.tall ? pl.stride_x : pl.stride_s;
    next.g.ldb = pl.tall ? pl.ld_s : pl.ld_x;
    next.g.stride_b = pl.tall ? pl.stride_s : pl.stride_x;
    next.g.M = m;
    next.g.N = cols;
    next.g.K = pl.s;
    next.g.c = last ? out : plane(pl.x[cur ^ 1], 0);
    next.c_lo = last || !SPLIT ? nullptr : plane(pl.x[cur ^ 1], 1);
    next.g.ldc = last ? ld_out : pl.ld_x;
    next.g.stride_c = last ? stride_out : pl.stride_x;
    next.g.vec_c = last && vec_c_ok(out, ld_out, stride_out, SPLIT ? MXTRAIN_F32 : MXTRAIN_BF16);
    next.phi = step == 0 ? n.phi : nullptr;
    next.scale = (last ? 1.0f / mxt::kXScale : 1.0f) / ps;
    using namespace mxt;
    st = pl.tall ? ns_gemm<kGram, kMC, kMC, SPLIT>(gram, batch, stream)
                 : ns_gemm<kGram, kKC, kKC, SPLIT>(gram, batch, stream);
    if (st == MXTRAIN_OK) st = ns_gemm<kPoly, kKC, kKC, SPLIT>(poly, batch, stream);
    if (st == MXTRAIN_OK) {
      if (last)
        st = pl.tall ? ns_gemm<kLast, kKC, kKC, SPLIT>(next, batch, stream)
                     : ns_gemm<kLast, kKC, kMC, SPLIT>(next, batch, stream);
      else
        st = pl.tall ? ns_gemm<kNext, kKC, kKC, SPLIT>(next, batch, stream)
                     : ns_gemm<kNext, kKC, kMC, SPLIT>(next, batch, stream);
    }
    if (st != MXTRAIN_OK) return st;
  }
  return MXTRAIN_OK;
}

}  // namespace

extern "C" {

mxtrain_status mxtrain_layer_norm_fwd(const void *x, int64_t ld_x, const void *weight, const void *bias,
                                      int param_dtype, int64_t M, int64_t N, int dtype, float eps, void *y,
                                      int64_t ld_y, float *mean, float *rstd, void *stream) {
  if (!type_ok(dtype) || !type_ok(param_dtype)) return MXTRAIN_ERR_TYPE;
  if (!(eps >= 0.0f) || std::isinf(eps)) return MXTRAIN_ERR_VALUE;
  if (M < 0 || N < 0 || M > INT32_MAX || N > INT32_MAX - 4096) return MXTRAIN_ERR_SHAPE;
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
  // As many workgroups as the CUs hold at once by their registers, each of
  // which then walks rows: 16 or 32 elements a thread leave room for 1024
  // threads to a CU, 8 for 1536 or, moved as vectors, 2048 (16384 x 5120 bf16:
  // 63 us with 1024 threads to a CU, 81 with 1280, more than fit evenly; 16384 x
  // 2048 27 us with 2048, 33 with 1024).
  const int per_cu = p.elems > 8 ? 1024 : vec ? 2048 : 1536;
  const int64_t most = p.elems ? cu_count() * std::max<int64_t>(1, per_cu / p.threads) : M;
  return launch(ln_kernel<false>(p, dtype, vec), std::min((M + rows - 1) / rows, most), p.threads, g, stream);
}

int64_t mxtrain_layer_norm_bwd_workspace(int64_t M, int64_t N) {
  if (M <= 0 || N <= 0 || M > INT32_MAX || N > INT32_MAX - 4096) return 0;
  return ln_parts(M) * 2 * N * (int64_t)sizeof(float);
}

mxtrain_status mxtrain_layer_norm_bwd(const void *dy, int64_t ld_dy, const void *x, int64_t ld_x, const float *mean,
                                      const float *rstd, const void *weight, int param_dtype, int64_t M, int64_t N,
                                      int dtype, void *dx, int64_t ld_dx, float *dweight, float *dbias,
                                      void *workspace, int64_t workspace_bytes, void *stream) {
  if (!type_ok(dtype) || !type_ok(param_dtype)) return MXTRAIN_ERR_TYPE;
  if (M < 0 || N < 0 || M > INT32_MAX || N > INT32_MAX - 4096) return MXTRAIN_ERR_SHAPE;
  if (N == 0) return M == 0 ? MXTRAIN_OK : MXTRAIN_ERR_SHAPE;
  if (!aligned(dweight, 4) || !aligned(dbias, 4)) return MXTRAIN_ERR_ALIGN;
  const bool sums = dweight || dbias;
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
    const unsigned joined = p.tpr ? (unsigned)(slots * 2 * N * (int64_t)sizeof(float)) : 0u;
    const mxtrain_status run = launch(ln_kernel<true>(p, dtype, vec), parts, p.threads, g, stream, joined);
    if (run != MXTRAIN_OK) return run;
  }
  if (!sums) return MXTRAIN_OK;
  const float *part = static_cast<const float *>(workspace);
  int n_parts = (int)parts;
  int32_t n = (int32_t)N;
  void *kargs[] = {&part, &n_parts, &n, &dweight, &dbias};
  const int64_t blocks = (2 * N + 31) / 32;
  if (blocks > INT32_MAX / 1024) return MXTRAIN_ERR_OVERFLOW;
  const hipError_t err = hipLaunchKernel((const void *)&mxt::k_ln_join, dim3((unsigned)blocks), dim3(1024), kargs, 0,
                                         (hipStream_t)stream);
  return err == hipSuccess ? MXTRAIN_OK : MXTRAIN_ERR_LAUNCH;
}

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
  if (stride_b < 0 || stride_b % 8 != 0 || ldc < N) return MXTRAIN_ERR_STRIDE;
  if (G > 1 && b_rows > 0 && stride_b < (b_rows - 1) * ldb + b_cols) return MXTRAIN_ERR_STRIDE;
  if (!aligned(group_ends, 4) || !aligned(c, (uintptr_t)size_of(c_dtype))) return MXTRAIN_ERR_ALIGN;
  if (!extent_ok(M, N, ldc) || __builtin_mul_overflow(stride_b, G, &all) || all > (INT64_MAX >> 4))
    return MXTRAIN_ERR_OVERFLOW;
  const bool f32 = c_dtype == MXTRAIN_F32;
  const int64_t groups = std::min(G, M), rows = (M + groups - 1) / groups;  // as if evenly spread
  const GroupKernel k = transpose_b ? group_pick<mxt::kGroupM, mxt::kKC, mxt::kKC>(groups, rows, N, f32)
                                    : group_pick<mxt::kGroupM, mxt::kKC, mxt::kMC>(groups, rows, N, f32);
  // an upper bound of tile rows, each group adding at most one partial one:
  // the host never reads the ends
  const int64_t tiles_m = (M + k.bm - 1) / k.bm + G, tiles_n = (N + k.bn - 1) / k.bn;
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
  const GroupKernel k = group_pick<mxt::kGroupK, mxt::kMC, mxt::kMC>(G, M, N, c_dtype == MXTRAIN_F32);
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
  if (batch < 0 || m < 0 || n < 0 || batch > kMaxGroups || m >= mxt::kMaxLd - 8 || n >= mxt::kMaxLd - 8)
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
  a.x_lo = pl.split ? reinterpret_cast<_Float16 *>(ws + pl.x[0][1]) : nullptr;
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
