// tr_norm.hpp -- layer norm, forward and backward (gfx950).
//
// Forward, per row x of N elements:
//   mean = sum x / N,  rstd = 1 / sqrt(sum (x - mean)^2 / N + eps),
//   y = (x - mean) rstd w + b.
// Backward, with xh = (x - mean) rstd and g = dy w:
//   dx = rstd (g - sum g / N - xh sum (g xh) / N),
//   dw = sum over rows of dy xh,  db = sum over rows of dy.
//
// Both are bound by HBM: the forward reads x and writes y, the backward reads
// dy and x and writes dx, each once.  So a row stays in registers between its
// reductions and its output (up to 32 elements a thread), and the backward's
// column sums are kept in registers over all the rows that a workgroup walks,
// written once per workgroup as a partial row and joined by a second kernel in a
// fixed order (no atomics: equal inputs give equal bits).  All arithmetic is
// fp32; outputs are rounded once.
//
// Rows far off centre: the variance is taken from deviations d = x - m to the
// mean m already known, and the second reduction sums d beside d^2.  With
// e = sum d / N, m + e is the mean freed from the first sum's rounding, and
// sum d^2 / N - e^2 the variance about it; y uses d - e, which keeps the
// places that m itself has no room for.  The extra sum rides along in the
// second reduction.  Where the row's mean is smaller than its spread, the
// first sum is as exact as the second (more so for bf16 rows, whose few
// places add up without rounding), and e, then only rounding, is dropped.
#pragma once
#include "tr_common.hpp"

namespace mxt {

struct LnArgs {
  const void *x, *dy, *w, *b;
  void *y;  // y, or dx in the backward pass
  int64_t ld_x, ld_dy, ld_y;
  float *mean, *rstd;  // written by the forward (may be NULL), read by the backward
  float *part;         // backward: partial column sums [row_blocks][2][N], or NULL
  float *dw, *db;      // backward: the column sums, where workgroups of their own take them
  int64_t row_blocks;  // backward: workgroups that walk rows; those after them take columns
  int64_t M;
  int32_t N;
  int32_t w_f32;  // weight and bias are fp32 (else bf16)
  int32_t p_vec;  // and may be read 16 bytes at a time
  float eps;
};

// A thread holds CH chunks of VEC consecutive elements; chunk i starts at
// column (i * TPR + t) * VEC.  VEC is 16 bytes' worth where every row starts
// 16-byte aligned and N is a multiple of it, otherwise 1.
template <class T, int VEC>
__device__ __forceinline__ void store_chunk(T *p, const float *v) {
  if constexpr (VEC == 1) {
    *gptr(p) = from_f32<T>(v[0]);
  } else if constexpr (sizeof(T) == 2) {
    u32x4_t q;
#pragma unroll
    for (int i = 0; i < 4; i++) q[i] = mx::pack_bf16(v[2 * i], v[2 * i + 1]);
    __builtin_nontemporal_store(q, gptr(reinterpret_cast<u32x4_t *>(p)));
  } else {
    f32x4_t q;
#pragma unroll
    for (int i = 0; i < 4; i++) q[i] = v[i];
    __builtin_nontemporal_store(q, gptr(reinterpret_cast<f32x4_t *>(p)));
  }
}

// VEC elements of the weight or bias (bf16 or fp32; `missing` where NULL), 16
// bytes at a time where `vec` says that their base allows it (col is a
// multiple of VEC).
template <int VEC>
__device__ __forceinline__ void load_param(const void *p, bool f32, bool vec, int32_t col, float missing, float *v) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < VEC; i++) v[i] = missing;
  } else if (f32) {
    const float *q = static_cast<const float *>(p) + col;
    if (VEC >= 4 && vec) {
#pragma unroll
      for (int i = 0; i < VEC; i += 4) {
        const f32x4_t u = *gptr(reinterpret_cast<const f32x4_t *>(q + i));
#pragma unroll
        for (int j = 0; j < 4 && i + j < VEC; j++) v[i + j] = u[j];
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i++) v[i] = *gptr(q + i);
    }
  } else {
    const uint16_t *q = static_cast<const uint16_t *>(p) + col;
    if (VEC == 8 && vec) {
      const u32x4_t u = *gptr(reinterpret_cast<const u32x4_t *>(q));
#pragma unroll
      for (int i = 0; i < VEC; i++) v[i] = i % 2 ? mx::hi_f(u[i / 2]) : mx::lo_f(u[i / 2]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i++) v[i] = to_f32(*gptr(q + i));
    }
  }
}

// Sums of a and b over the TPR threads of a row, in every one of them.
// TPR <= 64: lane swaps inside the wavefront.  TPR == 0: the row is the whole
// workgroup (a multiple of 64 threads); `sm` holds two values per wavefront
// and is not reused before another barrier.
template <int TPR>
__device__ __forceinline__ void row_sum2(float &a, float &b, float (*sm)[2]) {
  constexpr int W = TPR == 0 ? 64 : TPR;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) {
    a += __shfl_xor(a, o, 64);
    b += __shfl_xor(b, o, 64);
  }
  if constexpr (TPR == 0) {
    const int w = threadIdx.x >> 6, n = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      sm[w][0] = a;
      sm[w][1] = b;
    }
    __syncthreads();
    a = b = 0.0f;
    for (int i = 0; i < n; i++) {
      a += sm[i][0];
      b += sm[i][1];
    }
  }
}

// The correction e and 1 / sqrt(var + eps) from the second reduction's sums.
__device__ __forceinline__ float ln_rstd(float m, float q, float &e, const LnArgs &g) {
  q /= (float)g.N;
  e = m * m > q ? e / (float)g.N : 0.0f;
  const float var = fmaf(-e, e, q);
  return 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + g.eps);  // a NaN stays one
}

// One chunk as it lies in memory: what a thread holds of the next row.
template <class T, int VEC>
struct Raw {
  static constexpr int kWords = VEC == 1 ? 1 : 4;
  u32 w[kWords];
  __device__ __forceinline__ void load(const T *p, u32 off) {
    if constexpr (VEC == 1) {
      if constexpr (sizeof(T) == 2) w[0] = *gptr(byte_off(p, off));
      else w[0] = __float_as_uint(*gptr(byte_off(p, off)));
    } else {
      const u32x4_t q = *gptr(reinterpret_cast<const u32x4_t *>(byte_off(p, off)));
#pragma unroll
      for (int i = 0; i < 4; i++) w[i] = q[i];
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
    else if constexpr (VEC == 1) return __uint_as_float(w[0] << 16);
    else return j % 2 ? mx::hi_f(w[j / 2]) : mx::lo_f(w[j / 2]);
  }
};

// TPR threads to a row, here and below (0: the whole workgroup).
//
// Workgroup b walks rows b, b + gridDim.x, ... (groups of 256 / TPR rows),
// with the weight and bias in registers and a row's loads issued while the row
// before it is reduced.  16384 x 8192 bf16: 96 us, 5.6 TB/s over x and y (a
// workgroup to every row, the next row's loads waiting for it: 110 us).
template <class T, int VEC, int TPR, int CH>
__global__ __launch_bounds__((TPR != 0 ? 256 : CH * VEC <= 16 ? 1024 : 512)) void k_ln_fwd(const LnArgs g) {
  __shared__ float sm[4][16][2];
  constexpr int kTpr = TPR == 0 ? 1 : TPR;
  constexpr int kSlots = TPR == 0 ? 1 : 256 / kTpr;
  const int tpr = TPR == 0 ? (int)blockDim.x : TPR;
  const int t = TPR == 0 ? (int)threadIdx.x : (int)threadIdx.x % kTpr;
  const int slot = TPR == 0 ? 0 : (int)threadIdx.x / kTpr;
  float w[CH][VEC], b[CH][VEC];
  u32 off[CH];  // byte offset of the chunk in a row; past its end, the row's first chunk
  auto in = [&](int i) { return (i * tpr + t) * VEC < g.N; };
#pragma unroll
  for (int i = 0; i < CH; i++) {
    const int32_t col = in(i) ? (i * tpr + t) * VEC : 0;
    off[i] = (u32)col * (u32)sizeof(T);
    load_param<VEC>(g.w, g.w_f32, g.p_vec, col, 1.0f, w[i]);
    load_param<VEC>(g.b, g.w_f32, g.p_vec, col, 0.0f, b[i]);
  }
  Raw<T, VEC> rx[CH];
  const int64_t step = (int64_t)gridDim.x * kSlots;
  auto fetch = [&](int64_t row) {
    const T *x = static_cast<const T *>(g.x) + row * g.ld_x;
#pragma unroll
    for (int i = 0; i < CH; i++) rx[i].load(x, off[i]);
  };
  int64_t row = (int64_t)blockIdx.x * kSlots + slot;
  if (row < g.M) fetch(row);
  int phase = 0;
  for (; row < g.M; row += step) {
    T *y = static_cast<T *>(g.y) + row * g.ld_y;
    float v[CH][VEC];
    float s = 0.0f, unused = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; i++)
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        v[i][j] = rx[i].get(j);
        s += in(i) ? v[i][j] : 0.0f;
      }
    if (row + step < g.M) fetch(row + step);
    row_sum2<TPR>(s, unused, sm[phase]);  // two buffers a row, the other two next row
    const float m = s / (float)g.N;
    float q = 0.0f, e = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; i++)
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        const float d = in(i) ? v[i][j] - m : 0.0f;
        v[i][j] = d;
        e += d;
        q = fmaf(d, d, q);
      }
    row_sum2<TPR>(q, e, sm[phase + 1]);
    phase ^= 2;
    const float rstd = ln_rstd(m, q, e, g);
#pragma unroll
    for (int i = 0; i < CH; i++) {
#pragma unroll
      for (int j = 0; j < VEC; j++) v[i][j] = fmaf((v[i][j] - e) * rstd, w[i][j], b[i][j]);
      if (in(i)) store_chunk<T, VEC>(byte_off(y, off[i]), v[i]);
    }
    if (t == 0 && g.mean) *gptr(g.mean + row) = m + e;
    if (t == 0 && g.rstd) *gptr(g.rstd + row) = rstd;
  }
}

// Rows longer than the registers of a workgroup hold: the row is read three
// times (sum, squared deviations, output), one element at a time.
template <class T>
__global__ __launch_bounds__(1024) void k_ln_fwd_long(const LnArgs g) {
  __shared__ float sm[2][16][2];
  for (int64_t row = blockIdx.x; row < g.M; row += gridDim.x) {
    const T *x = static_cast<const T *>(g.x) + row * g.ld_x;
    T *y = static_cast<T *>(g.y) + row * g.ld_y;
    float s = 0.0f, q = 0.0f, e = 0.0f, unused = 0.0f;
    for (int64_t c = threadIdx.x; c < g.N; c += 1024) s += to_f32(*gptr(x + c));
    row_sum2<0>(s, unused, sm[0]);
    const float m = s / (float)g.N;
    for (int64_t c = threadIdx.x; c < g.N; c += 1024) {
      const float d = to_f32(*gptr(x + c)) - m;
      e += d;
      q = fmaf(d, d, q);
    }
    row_sum2<0>(q, e, sm[1]);  // its barrier also lies between this row's reads of sm[0] and the next row's writes
    const float rstd = ln_rstd(m, q, e, g);
    for (int64_t c = threadIdx.x; c < g.N; c += 1024) {
      float w, b;
      load_param<1>(g.w, g.w_f32, false, (int32_t)c, 1.0f, &w);
      load_param<1>(g.b, g.w_f32, false, (int32_t)c, 0.0f, &b);
      *gptr(y + c) = from_f32<T>(fmaf((to_f32(*gptr(x + c)) - m - e) * rstd, w, b));
    }
    if (threadIdx.x == 0 && g.mean) *gptr(g.mean + row) = m + e;
    if (threadIdx.x == 0 && g.rstd) *gptr(g.rstd + row) = rstd;
  }
}

// Most threads of a backward workgroup whose threads hold E elements: a thread
// needs five registers an element, one or two more for the row that it holds
// ahead and a few per chunk, of the 128 that 1024 threads leave it or the 256
// that 512 do (with E = 32 only where no row is held ahead).
template <int VEC, int E>
constexpr int kLnBwdThreads = E <= 8 && VEC > 1 ? 1024 : 512;

// The column sums of few rows.  They need no row's reduction, so further
// workgroups of the backward's launch take 64 columns each and read them over all
// rows again (from L2), instead of a second launch over partial rows, which
// costs a small call more than that.
template <class T>
__device__ __forceinline__ void ln_columns(const LnArgs &g, int64_t strip, float (*sm)[64][2]) {
  const int c = threadIdx.x & 63, s = threadIdx.x >> 6, n = blockDim.x >> 6;
  const int64_t col = strip * 64 + c;
  float aw = 0.0f, ab = 0.0f;
  if (col < g.N) {
    const T *x = static_cast<const T *>(g.x) + col, *dy = static_cast<const T *>(g.dy) + col;
#pragma unroll 8
    for (int64_t r = s; r < g.M; r += n) {
      const float d = to_f32(*gptr(dy + r * g.ld_dy));
      const float h = (to_f32(*gptr(x + r * g.ld_x)) - *gptr(g.mean + r)) * *gptr(g.rstd + r);
      aw = fmaf(d, h, aw);
      ab += d;
    }
  }
  sm[s][c][0] = aw;
  sm[s][c][1] = ab;
  __syncthreads();
  if (s == 0 && col < g.N) {
    for (int k = 1; k < n; k++) {
      aw += sm[k][c][0];
      ab += sm[k][c][1];
    }
    if (g.dw) *gptr(g.dw + col) = aw;
    if (g.db) *gptr(g.db + col) = ab;
  }
}

// Backward.  Workgroup b walks rows b, b + gridDim.x, ... (TPR == 0) or the
// same for groups of 256 / TPR rows; every thread keeps its columns' sums of
// dy xh and dy over all of them.  A row's loads are issued before the
// reduction of the row before it, which they would otherwise wait for.  With
// TPR > 0 the row slots of a workgroup are joined in LDS (dynamic: slots * 2 *
// N floats) before the partial row is written.
//
// 16384 x 5120 bf16: 94 us, 5.35 TB/s over dy, x and dx (without the row held
// ahead and with half the wavefronts 155 us).
//
// Workgroups past row_blocks take columns (ln_columns).
//
// Columns past N: a chunk that lies there is read as the row's first one and
// its weight and dy count as zero, so that it adds nothing.
template <class T, int VEC, int TPR, int CH>
__global__ __launch_bounds__((TPR != 0 ? 256 : kLnBwdThreads<VEC, (CH * VEC)>)) void k_ln_bwd(const LnArgs g) {
  __shared__ float sm[2][16][2];
  __shared__ float col_sm[16][64][2];
  extern __shared__ float joined[];
  if ((int64_t)blockIdx.x >= g.row_blocks) {
    ln_columns<T>(g, (int64_t)blockIdx.x - g.row_blocks, col_sm);
    return;
  }
  constexpr int kTpr = TPR == 0 ? 1 : TPR;
  constexpr int kSlots = TPR == 0 ? 1 : 256 / kTpr;
  const int tpr = TPR == 0 ? (int)blockDim.x : TPR;
  const int t = TPR == 0 ? (int)threadIdx.x : (int)threadIdx.x % kTpr;
  const int slot = TPR == 0 ? 0 : (int)threadIdx.x / kTpr;
  const float inv_n = 1.0f / (float)g.N;
  float w[CH][VEC], aw[CH][VEC], ab[CH][VEC];
  u32 off[CH];  // byte offset of the chunk in a row
  auto in = [&](int i) { return (i * tpr + t) * VEC < g.N; };
#pragma unroll
  for (int i = 0; i < CH; i++) {
    const int32_t col = (i * tpr + t) * VEC;
    off[i] = in(i) ? (u32)col * (u32)sizeof(T) : 0u;
    load_param<VEC>(g.w, g.w_f32, g.p_vec, in(i) ? col : 0, 1.0f, w[i]);
#pragma unroll
    for (int j = 0; j < VEC; j++) {
      if (!in(i)) w[i][j] = 0.0f;
      aw[i][j] = ab[i][j] = 0.0f;
    }
  }
  Raw<T, VEC> rx[CH], rd[CH];
  float mean = 0.0f, rstd = 0.0f;
  const int64_t step = g.row_blocks * kSlots;
  auto fetch = [&](int64_t row) {
    const T *x = static_cast<const T *>(g.x) + row * g.ld_x;
    const T *dy = static_cast<const T *>(g.dy) + row * g.ld_dy;
#pragma unroll
    for (int i = 0; i < CH; i++) {
      rx[i].load(x, off[i]);
      rd[i].load(dy, off[i]);
    }
    mean = *gptr(g.mean + row);
    rstd = *gptr(g.rstd + row);
  };
  int64_t row = (int64_t)blockIdx.x * kSlots + slot;
  constexpr bool kAhead = CH * VEC <= 16;
  if (kAhead && row < g.M) fetch(row);
  int phase = 0;
  for (; row < g.M; row += step) {
    if (!kAhead) fetch(row);
    T *dx = static_cast<T *>(g.y) + row * g.ld_y;
    float xh[CH][VEC], d[CH][VEC];
    const float r = rstd;
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; i++)
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        const float h = (rx[i].get(j) - mean) * r, dv = in(i) ? rd[i].get(j) : 0.0f;
        xh[i][j] = h;
        aw[i][j] = fmaf(dv, h, aw[i][j]);
        ab[i][j] += dv;
        const float gd = dv * w[i][j];
        d[i][j] = gd;
        s1 += gd;
        s2 = fmaf(gd, h, s2);
      }
    if (kAhead && row + step < g.M) fetch(row + step);
    row_sum2<TPR>(s1, s2, sm[phase]);  // the other buffer next row: one barrier a row is enough
    phase ^= 1;
    const float c1 = s1 * inv_n, c2 = s2 * inv_n;
#pragma unroll
    for (int i = 0; i < CH; i++) {
#pragma unroll
      for (int j = 0; j < VEC; j++) d[i][j] = (d[i][j] - fmaf(xh[i][j], c2, c1)) * r;
      if (in(i)) store_chunk<T, VEC>(byte_off(dx, off[i]), d[i]);
    }
  }
  if (!g.part) return;
  float *part = g.part + (int64_t)blockIdx.x * 2 * g.N;
  if constexpr (TPR == 0) {
#pragma unroll
    for (int i = 0; i < CH; i++) {
      const int32_t col = (i * tpr + t) * VEC;
      if (in(i)) {
#pragma unroll
        for (int j = 0; j < VEC; j++) {
          *gptr(part + col + j) = aw[i][j];
          *gptr(part + g.N + col + j) = ab[i][j];
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < CH; i++) {
      const int32_t col = (i * tpr + t) * VEC;
      if (in(i)) {
#pragma unroll
        for (int j = 0; j < VEC; j++) {
          joined[(slot * 2) * g.N + col + j] = aw[i][j];
          joined[(slot * 2 + 1) * g.N + col + j] = ab[i][j];
        }
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * g.N; c += 256) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < kSlots; k++) s += joined[k * 2 * g.N + c];
      *gptr(part + c) = s;
    }
  }
}

// Rows longer than the registers hold: two passes over the row, and the
// workgroup's partial sums kept in its own row of `part` (each thread adds to
// its own columns only).
template <class T>
__global__ __launch_bounds__(1024) void k_ln_bwd_long(const LnArgs g) {
  __shared__ float sm[2][16][2];
  float *part = g.part ? g.part + (int64_t)blockIdx.x * 2 * g.N : nullptr;
  const float inv_n = 1.0f / (float)g.N;
  int phase = 0;
  for (int64_t row = blockIdx.x; row < g.M; row += gridDim.x) {
    const T *x = static_cast<const T *>(g.x) + row * g.ld_x;
    const T *dy = static_cast<const T *>(g.dy) + row * g.ld_dy;
    T *dx = static_cast<T *>(g.y) + row * g.ld_y;
    const float mean = *gptr(g.mean + row), rstd = *gptr(g.rstd + row);
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = threadIdx.x; c < g.N; c += 1024) {
      float w;
      load_param<1>(g.w, g.w_f32, false, (int32_t)c, 1.0f, &w);
      const float d = to_f32(*gptr(dy + c)), h = (to_f32(*gptr(x + c)) - mean) * rstd;
      s1 += d * w;
      s2 = fmaf(d * w, h, s2);
      if (part) {
        const bool first = row == (int64_t)blockIdx.x;
        *gptr(part + c) = fmaf(d, h, first ? 0.0f : *gptr(part + c));
        *gptr(part + g.N + c) = d + (first ? 0.0f : *gptr(part + g.N + c));
      }
    }
    row_sum2<0>(s1, s2, sm[phase]);
    phase ^= 1;
    const float c1 = s1 * inv_n, c2 = s2 * inv_n;
    for (int64_t c = threadIdx.x; c < g.N; c += 1024) {
      float w;
      load_param<1>(g.w, g.w_f32, false, (int32_t)c, 1.0f, &w);
      const float d = to_f32(*gptr(dy + c)), h = (to_f32(*gptr(x + c)) - mean) * rstd;
      *gptr(dx + c) = from_f32<T>((d * w - fmaf(h, c2, c1)) * rstd);
    }
  }
}

// dw and db: the sums of `parts` partial rows, in row order within each of 32
// slices and then over the slices.  A workgroup takes 32 columns of the 2 N
// (dw's, then db's) at a time; no rows give zeros.
__global__ __launch_bounds__(1024) void k_ln_join(const float *part, int parts, int32_t N, float *dw, float *db) {
  __shared__ float sm[32][33];
  const int c = threadIdx.x & 31, s = threadIdx.x >> 5;
  const int64_t all = 2 * (int64_t)N;
  for (int64_t first = (int64_t)blockIdx.x * 32; first < all; first += (int64_t)gridDim.x * 32) {
    const int64_t col = first + c;
    float a = 0.0f;
    if (col < all)
#pragma unroll 4
      for (int p = s; p < parts; p += 32) a += *gptr(part + p * all + col);
    sm[s][c] = a;
    __syncthreads();
    if (s == 0 && col < all) {
      float t = 0.0f;
#pragma unroll
      for (int k = 0; k < 32; k++) t += sm[k][c];
      if (col < N) {
        if (dw) *gptr(dw + col) = t;
      } else {
        if (db) *gptr(db + col - N) = t;
      }
    }
    __syncthreads();  // before sm is written again
  }
}

}  // namespace mxt
