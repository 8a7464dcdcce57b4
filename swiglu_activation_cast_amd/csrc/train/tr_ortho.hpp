// tr_ortho.hpp -- orthogonalising weight updates by Newton-Schulz steps.
//
//   X_0 = G / (|G| + eps),  |G| the root of the sum of squares,
//   X <- p(X X^T) X,  p(S) = a I + b S + c S^2       (wide: rows <= columns)
//   X <- X p(X^T X)                                  (tall)
// so that every singular value s goes to a s + b s^3 + c s^5.  S has the
// shorter side; it and p(S) are symmetric, so only the tiles on and below
// their diagonal are computed and the others written as their transposes.
//
// A step is three products: S; S^2 with p's sum in its epilogue (a goes on the
// diagonal, so that the third product needs no extra read of X); and p(S) X.
//
// Number format.  X, S and p(S) are held between the products as fp16 times a
// power of two (their entries are bounded, since the singular values are: X by
// 2^14, S by 2^13, p(S) by a power that keeps its largest possible entry in
// range).  For an fp32 result each is held as two fp16 numbers, high and low
// part, 22 places, and a product is the sum of high x low, low x high and
// high x high (low x low lies below 2^-22): three matrix-core passes, where
// an fp32 product on this card runs at less than a tenth of the 16-bit rate.
//
// For a bf16 result S and p(S) have one part, but X two, of which S is taken
// from the high one and p(S) X from both (K gone through twice).  An error of
// S or p(S) only moves X within its own row space (columns, if tall), by
// fp16's 2^-11 beside bf16's 2^-8; one of X lies anywhere, and outside X's
// space it grows by p(s) / s, 3.4445 a step for the usual quintic: with one part
// of X the result of a 512 x 1024 matrix of rank 4, 32 or 128 is off by 4.3, 2.2
// or 1.1% (Frobenius), with two by 0.2%, full rank or not (an fp32 run rounded
// at its end: 0.17%; all in 64-bit emulation).
//
// The first X is G times a power of two 2^e with (|G| + eps) 2^e in [1/2, 1),
// which is exact for bf16 input; the factor that is left, phi = 1 / ((|G| +
// eps) 2^e) in (1, 2], enters the first step's polynomial and result in fp32.
// |G| is summed in 64 bits, which no fp32 input overflows.
#pragma once
#include "tr_gemm.hpp"

namespace mxt {

typedef _Float16 h4_t __attribute__((ext_vector_type(4)));

constexpr float kXScale = 16384.0f;  // 2^14: singular values up to 2 stay below fp16's 65504
constexpr float kSScale = 8192.0f;   // 2^13
constexpr int kNormBlocks = 512;     // workgroups that share one matrix's sum of squares

struct NsArgs {
  const void *g;
  int64_t ld_g, stride_g;
  int64_t rows, cols, batch;
  int32_t g_f32, vec;
  double eps;
  double *sums;  // [batch][kNormBlocks]
  float *phi;    // [batch]
  _Float16 *x, *x_lo;
  int64_t ld_x, stride_x;
};

// v as two fp16 numbers.  v is made opaque first: fused with the product it
// comes from, the compiler may round that straight to fp16 for one use of the
// high part and by way of fp32 for the other, which near a tie gives two
// different high parts and a low part that fits neither.
__device__ __forceinline__ void split_f16(float v, _Float16 &hi, _Float16 &lo) {
#if __HIP_DEVICE_COMPILE__
  asm volatile("" : "+v"(v));
#endif
  hi = (_Float16)v;
  lo = (_Float16)(v - (float)hi);
}

enum NsStep { kGram = 0, kPoly = 1, kNext = 2, kLast = 3, kPart = 4 };  // kPart: a part of S's sum over K

struct NsGemm {
  GemmArgs g;  // a, b: high planes; c: the result's high plane, or the output
  const uint16_t *a_lo, *b_lo;
  _Float16 *c_lo;
  const _Float16 *s, *s_lo;  // kPoly: S itself
  const float *phi;          // per matrix, or NULL (1)
  float ca, cb, cc;          // kPoly: coefficients times p's scale, b and c over S's scales
  float scale;               // the other steps: of the sums
  int32_t passes;            // one plane, kNext and kLast: 2 where X has a low plane (see Tile)
  int32_t parts;             // kPart: pieces of K, `part_k` of it each (g.c: fp32 sums, g.stride_c apart)
  int64_t part_k;
};

// One step's results at a tile: fp16 planes (high, and low where TWO).
template <int STEP, bool TWO>
struct EmitNs {
  static constexpr bool kF32 = false, kMirror = STEP != kNext;
  static constexpr int kPlanes = TWO ? 2 : 1;
  _Float16 *out[2];             // at the tile
  _Float16 *mir[2];             // at the transposed tile, or NULL
  const _Float16 *s_hi, *s_lo;  // kPoly: S at the tile
  int64_t ld;
  bool diag;                    // kPoly: the tile is on the diagonal
  float f0, f1, f2;

  __device__ __forceinline__ bool mirrored() const { return mir[0] != nullptr; }
  __device__ __forceinline__ void pack(u32 m, u32 n, f32x4_t v, u32x2_t *p) const {
    f32x4_t r;
    if constexpr (STEP == kPoly) {
      // past the matrix (rows and columns that are not stored) S is read at
      // the tile's first element
      const int64_t at = m < rows && n < cols ? (int64_t)m * ld + n : 0;
      const h4_t s = *gptr(reinterpret_cast<const h4_t *>(s_hi + at));
      h4_t sl = {};
      if constexpr (TWO) sl = *gptr(reinterpret_cast<const h4_t *>(s_lo + at));
#pragma unroll
      for (u32 e = 0; e < 4; e++) {
        const float sv = (float)s[e] + (float)sl[e];
        r[e] = fmaf(f2, v[e], f1 * sv) + (diag && m == n + e ? f0 : 0.0f);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; e++) r[e] = v[e] * f0;
    }
    h4_t a, b;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      _Float16 x, y;
      split_f16(r[e], x, y);
      a[e] = x;
      b[e] = y;
    }
    p[0] = __builtin_bit_cast(u32x2_t, a);
    if constexpr (TWO) p[1] = __builtin_bit_cast(u32x2_t, b);
  }
  // Rows are padded to whole chunks of 8, which all fit.
  __device__ __forceinline__ void store(int k, u32 m, u32 n, u32x4_t v) const {
    *gptr(reinterpret_cast<u32x4_t *>(out[k] + (int64_t)m * ld + n)) = v;
  }
  __device__ __forceinline__ void store_mirror(int k, u32 n, u32 m, u32x4_t v) const {
    *gptr(reinterpret_cast<u32x4_t *>(mir[k] + (int64_t)n * ld + m)) = v;
  }
  u32 rows, cols;
};

// The last step's: C in its own type.
template <bool F32>
struct EmitLast : EmitC<F32> {
  float f0;
  __device__ __forceinline__ f32x4_t map(u32, u32, f32x4_t v) const { return f32x4_t{v[0] * f0, v[1] * f0, v[2] * f0, v[3] * f0}; }
  __device__ __forceinline__ void pack(u32 m, u32 n, f32x4_t v, u32x2_t *p) const {
    EmitC<F32>::pack(m, n, map(m, n, v), p);
  }
};

// S from the partial sums of its lower tiles of 64 x 64, in order: a long
// thin matrix has too few tiles of S to fill the card, so K is dealt to several
// workgroups.  A thread takes one element.
template <bool SPLIT>
__global__ __launch_bounds__(256) void k_ns_join(const NsGemm p) {
  const GemmArgs &g = p.g;  // a: unused; c: the sums
  const int64_t batch = blockIdx.y, s = g.M, ld = g.ldc;
  const float *sums = static_cast<const float *>(g.c) + batch * p.parts * g.stride_c;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < s * s; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / s, n = i - m * s;
    const int64_t at = m / 64 >= n / 64 ? m * ld + n : n * ld + m;
    float v = 0.0f;
    for (int k = 0; k < p.parts; k++) v += *gptr(sums + k * g.stride_c + at);
    _Float16 hi, lo;
    split_f16(v * p.scale, hi, lo);
    *gptr(const_cast<_Float16 *>(p.s) + batch * g.stride_c + m * ld + n) = hi;
    if constexpr (SPLIT) *gptr(const_cast<_Float16 *>(p.s_lo) + batch * g.stride_c + m * ld + n) = lo;
  }
}

// Position L in row order of the tiles on and below the diagonal.
__device__ __forceinline__ void lower_tile(u32 L, u32 &tm, u32 &tn) {
  tm = (u32)((sqrtf(8.0f * (float)L + 1.0f) - 1.0f) * 0.5f);
  while (tm * (tm + 1) / 2 > L) tm--;  // the root is within one of the row
  while ((tm + 1) * (tm + 2) / 2 <= L) tm++;
  tn = L - tm * (tm + 1) / 2;
}

template <int STEP, int AL, int BL, int WI, int WJ, int BK, int RING, bool SPLIT>
__global__ __launch_bounds__(kThreads, 1) void k_ns_gemm(const NsGemm p) {
  constexpr int BM = 64 * WI, BN = 64 * WJ;
  constexpr bool SYM = STEP == kGram || STEP == kPoly || STEP == kPart;
  constexpr bool TWICE = !SPLIT && (STEP == kNext || STEP == kLast);  // p(S) times X's planes in turn
  static_assert(!SYM || WI == WJ, "symmetric results take square tiles");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[RING * (BM + BN) * BK * (SPLIT ? 4 : 2)];
  const GemmArgs &g = p.g;
  const u32 tiles = SYM ? (u32)g.tiles_m * (u32)(g.tiles_m + 1) / 2 : (u32)g.tiles_m * (u32)g.tiles_n;
  // whole-matrix products of 256 x 256 tiles end in a cut-down round (the
  // symmetric ones, whose tiles are square, do not)
  constexpr bool kCut = !SYM && WI == 4 && WJ == 4;
  Item it{blockIdx.x, 0, 1};
  const u32 R = tiles * (u32)g.G * (STEP == kPart ? (u32)p.parts : 1u);
  if (kCut && !work_item(blockIdx.x, R, (u32)g.cus, it)) return;
  const u32 whole = kCut ? R - R % (u32)g.cus : R;
  // matrices of fewer tiles than the CUs compute together: whole ones to an XCD
  const u32 L = !SYM && tiles >= 256 ? square_order(it.L, whole) : it.L < whole ? xcd_remap(it.L, whole) : it.L;
  // kPart: matrix `entry` of the partial sums is part entry % parts of matrix batch
  const int64_t entry = L / tiles, batch = STEP == kPart ? entry / p.parts : entry;
  u32 tm, tn;
  if constexpr (SYM) lower_tile(L % tiles, tm, tn);
  else tile_of(L % tiles, (u32)g.tiles_m, (u32)g.tiles_n, tm, tn);
  tm = (u32)__builtin_amdgcn_readfirstlane((int)tm);
  tn = (u32)__builtin_amdgcn_readfirstlane((int)tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN + it.part * (BN / it.parts);
  if (n0 >= g.N) return;  // a part past the last column
  int64_t k0 = 0, k_len = g.K;
  if constexpr (STEP == kPart) {
    k0 = entry % p.parts * p.part_k;
    k_len = max<int64_t>(min<int64_t>(g.K - k0, p.part_k), 0);
    if (k_len == 0) k0 = 0;
  }
  const int64_t a_at = batch * g.stride_a + (AL == kKC ? m0 * g.lda + k0 : m0 + k0 * g.lda);
  const int64_t b_at = batch * g.stride_b + (BL == kKC ? n0 * g.ldb + k0 : n0 + k0 * g.ldb);
  Tile t{g.a + a_at, g.b + b_at, nullptr, nullptr, k_len, (u32)min<int64_t>(BM, g.M - m0),
         (u32)min<int64_t>(BN / it.parts, g.N - n0), 0, p.passes};
  if constexpr (SPLIT || TWICE) {
    t.a_lo = p.a_lo + a_at;
    t.b_lo = p.b_lo + b_at;
  }
  const float phi = p.phi ? *gptr(p.phi + batch) : 1.0f;
  auto run = [&](const auto &e) {
    if constexpr (kCut) {
      if (it.parts == 4) return gemm_tile<kF16, AL, BL, WI, 1, BK, RING, SPLIT, TWICE>(g, t, smem, e);
      if (it.parts == 2) return gemm_tile<kF16, AL, BL, WI, 2, BK, RING, SPLIT, TWICE>(g, t, smem, e);
    }
    gemm_tile<kF16, AL, BL, WI, WJ, BK, RING, SPLIT, TWICE>(g, t, smem, e);
  };
  const int64_t at = entry * g.stride_c + m0 * g.ldc + n0;
  if constexpr (STEP == kPart) {
    run(EmitC<true>{static_cast<float *>(g.c) + at, g.ldc, t.cols, true});
  } else if constexpr (STEP == kLast) {
    EmitLast<SPLIT> e{};
    e.c = SPLIT ? (void *)(static_cast<float *>(g.c) + at) : (void *)(static_cast<uint16_t *>(g.c) + at);
    e.ldc = g.ldc;
    e.cols = t.cols;
    e.vec = g.vec_c != 0;
    e.f0 = p.scale * phi;
    run(e);
  } else {
    constexpr bool TWO = SPLIT || STEP == kNext;
    EmitNs<STEP, TWO> e{};
    e.ld = g.ldc;
    e.rows = t.rows;
    e.cols = t.cols;
    e.out[0] = static_cast<_Float16 *>(g.c) + at;
    if (TWO) e.out[1] = p.c_lo + at;
    if (SYM && tm != tn) {
      const int64_t mir = batch * g.stride_c + n0 * g.ldc + m0;
      e.mir[0] = static_cast<_Float16 *>(g.c) + mir;
      if (TWO) e.mir[1] = p.c_lo + mir;
    }
    if constexpr (STEP == kPoly) {
      e.s_hi = p.s + at;
      if (SPLIT) e.s_lo = p.s_lo + at;
      e.diag = tm == tn;
      e.f0 = p.ca;
      e.f1 = p.cb * phi * phi;
      e.f2 = p.cc * phi * phi * phi * phi;
    } else {
      e.f0 = STEP == kGram ? p.scale : p.scale * phi;
    }
    run(e);
  }
}

}  // namespace mxt
