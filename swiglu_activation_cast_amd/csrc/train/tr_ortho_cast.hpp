// tr_ortho_cast.hpp -- the way into the Newton-Schulz steps: the norm of G, and
// X_0 in the form that the products read.  Both pass over G once and are bound
// by HBM.
#pragma once
#include "tr_ortho.hpp"

namespace mxt {

// Eight columns from `col` of a row of G; zeros past its end.
__device__ __forceinline__ void ns_load8(const NsArgs &n, int64_t row, int64_t col, int64_t batch, float *v) {
  const int64_t at = batch * n.stride_g + row * n.ld_g + col;
  if (n.vec && col + 8 <= n.cols) {
    if (n.g_f32) {
      const f32x4_t *p = reinterpret_cast<const f32x4_t *>(static_cast<const float *>(n.g) + at);
      const f32x4_t a = *gptr(p), b = *gptr(p + 1);
#pragma unroll
      for (int i = 0; i < 4; i++) v[i] = a[i], v[4 + i] = b[i];
    } else {
      const u32x4_t q = *gptr(reinterpret_cast<const u32x4_t *>(static_cast<const uint16_t *>(n.g) + at));
#pragma unroll
      for (int i = 0; i < 4; i++) v[2 * i] = mx::lo_f(q[i]), v[2 * i + 1] = mx::hi_f(q[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
      v[i] = col + i >= n.cols ? 0.0f
             : n.g_f32         ? *gptr(static_cast<const float *>(n.g) + at + i)
                               : to_f32(*gptr(static_cast<const uint16_t *>(n.g) + at + i));
  }
}

// Chunk i of rows of `cpr` chunks: its row (the short division where it does).
__device__ __forceinline__ int64_t ns_row(int64_t i, int64_t cpr) {
  return ((uint64_t)i >> 32) == 0 ? (int64_t)((u32)i / (u32)cpr) : i / cpr;
}

// Sum over the workgroup's 256 threads, in every thread.
__device__ __forceinline__ double block_sum(double v, double *sm) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = v;
  __syncthreads();
  return (sm[0] + sm[1]) + (sm[2] + sm[3]);
}

// Workgroup (p, batch): the squares of every kNormBlocks-th piece of 256
// eight-column chunks.
__global__ __launch_bounds__(256) void k_ns_norm(const NsArgs n) {
  __shared__ double sm[4];
  const int64_t cpr = (n.cols + 7) / 8, total = n.rows * cpr, batch = blockIdx.y;
  double s = 0.0;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)kNormBlocks * 256) {
    const int64_t row = ns_row(i, cpr);
    float v[8];
    ns_load8(n, row, (i - row * cpr) * 8, batch, v);
#pragma unroll
    for (int j = 0; j < 8; j++) s = fma((double)v[j], (double)v[j], s);
  }
  s = block_sum(s, sm);
  if (threadIdx.x == 0) *gptr(n.sums + batch * kNormBlocks + blockIdx.x) = s;
}

// X_0's fp16 form (both planes where x_lo is given: not for bf16 G and result) and phi.
__global__ __launch_bounds__(256) void k_ns_cast(const NsArgs n) {
  __shared__ double sm[4];
  const int64_t cpr = n.ld_x / 8, total = n.rows * cpr, batch = blockIdx.y;
  double norm = 0.0;
#pragma unroll
  for (int p = 0; p < kNormBlocks; p += 256) norm += *gptr(n.sums + batch * kNormBlocks + p + threadIdx.x);
  norm = sqrt(block_sum(norm, sm)) + n.eps;
  // 2^e with norm 2^e in [1/2, 1); 0 or not finite: no scaling (phi carries it)
  int ex = 0;
  if (norm > 0.0 && norm < 1e300) frexp(norm, &ex);
  if (blockIdx.x == 0 && threadIdx.x == 0) *gptr(n.phi + batch) = (float)(1.0 / ldexp(norm, -ex));
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = ns_row(i, cpr), col = (i - row * cpr) * 8;
    float v[8];
    ns_load8(n, row, col, batch, v);
    typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
    h8_t hi, lo;
#pragma unroll
    for (int j = 0; j < 8; j++) {
      _Float16 a, b;
      split_f16(ldexpf(v[j], 14 - ex), a, b);
      hi[j] = a;
      lo[j] = b;
    }
    const int64_t at = batch * n.stride_x + row * n.ld_x + col;
    *gptr(reinterpret_cast<h8_t *>(n.x + at)) = hi;
    if (n.x_lo) *gptr(reinterpret_cast<h8_t *>(n.x_lo + at)) = lo;
  }
}

// No steps: X_0 itself.
__global__ __launch_bounds__(256) void k_ns_plain(const NsArgs n, void *out, int64_t ld, int64_t stride, int f32) {
  const int64_t cpr = n.ld_x / 8, total = n.rows * cpr, batch = blockIdx.y;
  const float f = *gptr(n.phi + batch) / kXScale;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = ns_row(i, cpr), col = (i - row * cpr) * 8, at = batch * n.stride_x + row * n.ld_x + col;
    for (int j = 0; j < 8 && col + j < n.cols; j++) {
      const float v = ((float)*gptr(n.x + at + j) + (n.x_lo ? (float)*gptr(n.x_lo + at + j) : 0.0f)) * f;
      const int64_t o = batch * stride + row * ld + col + j;
      if (f32) *gptr(static_cast<float *>(out) + o) = v;
      else *gptr(static_cast<uint16_t *>(out) + o) = from_f32<uint16_t>(v);
    }
  }
}

}  // namespace mxt
