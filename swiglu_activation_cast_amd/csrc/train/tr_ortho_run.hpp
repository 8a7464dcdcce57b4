// tr_ortho_run.hpp -- the host side of the Newton-Schulz steps: the workspace's
// layout and the launches of a run.  ns_run<false> (bf16 results) and ns_run<true>
// (fp32) are instantiated in a source of their own each, which compile side by
// side.
#pragma once
#include "tr_host.hpp"
#include "tr_ortho.hpp"

namespace mxt {

// ------------------------------------------------------- orthogonalisation
// Workspace: the fp16 planes of X (two of them, high and low, twice, in turn), S and p(S)
// (low planes for fp32 results only), then the sums of squares and phi.  Every part starts at a multiple of 256 bytes.
struct NsPlan {
  bool split, tall;
  int64_t s;             // the shorter side
  int64_t ld_x, stride_x, ld_s, stride_s;
  int64_t x[2][2], sq[2][2];  // byte offsets: [which][plane]; sq: S, p(S)
  int parts;                  // pieces of K that S's products are dealt in (1: whole)
  int64_t part_sums;          // byte offset of their fp32 sums
  int64_t sums, phi, bytes;   // bytes < 0: too large
};

inline NsPlan ns_plan(int64_t batch, int64_t m, int64_t n, int out_dtype) {
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
    for (int plane = 0; plane < 2; plane++) {
      p.x[which][plane] = take(p.stride_x, 2);
      if (plane == 0 || p.split) p.sq[which][plane] = take(p.stride_s, 2);
    }
  // S of at most 16 tiles of 64 x 64 leaves most CUs idle: over 40 stages of K or
  // more it is dealt to as many as 16 workgroups a tile, at least four stages
  // each (five steps of 2 x 6881 x 95 bf16: 161 us, 223 without; fp32 169 and
  // 334; of 8 x 64 x 2048 bf16, 32 stages, either way 94 +- 2).
  const int64_t ts = (p.s + 63) / 64, tiles = ts * (ts + 1) / 2 * batch, stages = (std::max(m, n) + 63) / 64;
  p.parts = tiles <= 16 && stages >= 40 ? (int)std::min<int64_t>({16, 256 / tiles, stages / 4}) : 1;
  p.part_sums = p.parts > 1 ? take(p.stride_s * p.parts, 4) : 0;
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
  //   1 x 256 x 512 fp32       416    203    103      102
  //   8 x 2048 x 1024 bf16     723    600   1053      540
  //   1 x 2048 x 2048 bf16     778    502    616      524
  //   4 x 2048 x 2048 bf16    1044   1192   2073     1042
  //   1 x 8192 x 1024 bf16    1107    708    533      374
  //   1 x 8192 x 5120 fp32    8753  10762  16288     8785
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

// S in parts of K, and their join.
template <int AL, bool SPLIT>
mxtrain_status ns_gram_parts(mxt::NsGemm p, const NsPlan &pl, int64_t batch, uint8_t *ws, void *stream) {
  const int64_t stages = (p.g.K + 63) / 64;
  p.s = static_cast<const _Float16 *>(p.g.c);
  p.s_lo = p.c_lo;
  p.g.c = ws + pl.part_sums;
  p.parts = pl.parts;
  p.part_k = (stages + pl.parts - 1) / pl.parts * 64;
  p.g.tiles_m = p.g.tiles_n = (int32_t)((pl.s + 63) / 64);
  p.g.G = (int32_t)batch;
  p.g.cus = cu_count();
  const int64_t blocks = batch * pl.parts * (int64_t)p.g.tiles_m * (p.g.tiles_m + 1) / 2;
  const mxtrain_status st =
      launch((const void *)&mxt::k_ns_gemm<mxt::kPart, AL, AL, 1, 1, 64, SPLIT ? 4 : 8, SPLIT>, blocks, mxt::kThreads, p, stream);
  if (st != MXTRAIN_OK) return st;
  void *kargs[] = {&p};
  const int64_t grid = std::min<int64_t>((pl.s * pl.s + 255) / 256, std::max<int64_t>(1, 2048 / batch));
  return hipLaunchKernel((const void *)&mxt::k_ns_join<SPLIT>, dim3((unsigned)grid, (unsigned)batch), dim3(256), kargs,
                         0, (hipStream_t)stream) == hipSuccess
             ? MXTRAIN_OK
             : MXTRAIN_ERR_LAUNCH;
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
    const _Float16 *x = plane(pl.x[cur], 0), *x_lo = plane(pl.x[cur], 1);
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
    next.g.b = pl.tall ? hq : hx;
    next.a_lo = pl.tall ? lx : SPLIT ? lq : hq;
    next.b_lo = pl.tall ? (SPLIT ? lq : hq) : lx;
    next.passes = step == 0 && !n.x_lo ? 1 : 2;  // a bf16 G has no low plane
    next.g.lda = pl.tall ? pl.ld_x : pl.ld_s;
    next.g.stride_a = pl.tall ? pl.stride_x : pl.stride_s;
    next.g.ldb = pl.tall ? pl.ld_s : pl.ld_x;
    next.g.stride_b = pl.tall ? pl.stride_s : pl.stride_x;
    next.g.M = m;
    next.g.N = cols;
    next.g.K = pl.s;
    next.g.c = last ? out : plane(pl.x[cur ^ 1], 0);
    next.c_lo = last ? nullptr : plane(pl.x[cur ^ 1], 1);
    next.g.ldc = last ? ld_out : pl.ld_x;
    next.g.stride_c = last ? stride_out : pl.stride_x;
    next.g.vec_c = last && vec_c_ok(out, ld_out, stride_out, SPLIT ? MXTRAIN_F32 : MXTRAIN_BF16);
    next.phi = step == 0 ? n.phi : nullptr;
    next.scale = (last ? 1.0f / mxt::kXScale : 1.0f) / ps;
    using namespace mxt;
    if (pl.parts > 1)
      st = pl.tall ? ns_gram_parts<kMC, SPLIT>(gram, pl, batch, ws, stream)
                   : ns_gram_parts<kKC, SPLIT>(gram, pl, batch, ws, stream);
    else
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

extern template mxtrain_status ns_run<false>(const NsPlan &pl, mxt::NsArgs n, int64_t batch, int64_t m, int64_t cols, int steps,
                      const float *co, void *out, int64_t ld_out, int64_t stride_out, uint8_t *ws, void *stream);
extern template mxtrain_status ns_run<true>(const NsPlan &pl, mxt::NsArgs n, int64_t batch, int64_t m, int64_t cols, int steps,
                      const float *co, void *out, int64_t ld_out, int64_t stride_out, uint8_t *ws, void *stream);

}  // namespace mxt
