// tr_route.hpp -- tokens to their experts and back (gfx950).
//
//   dispatch   xs[rank[t,j]] = x[t]
//   combine    y[t] = residual[t] + sum_j w[t,j] ys[rank[t,j]]
//   its gradients  dys[rank[t,j]] = w[t,j] dy[t],  dw[t,j] = <dy[t], ys[rank[t,j]]>
// (dispatch's gradient is a combine without weights).
//
// All are bound by HBM.  They walk tokens, not sorted rows: a token's row is
// read or written once and its k sorted rows, contiguous pieces of them, once
// each, so that nothing moves twice and no sum needs an order of its own.
#pragma once
#include "tr_sort.hpp"

namespace mxt {

struct RouteArgs {
  const void *in;        // x, ys, or (combine's gradients) ys
  const void *other;     // residual or NULL; dy
  void *out;             // xs, y, dys
  int64_t ld_in, ld_other, ld_out;
  const int32_t *rank;
  const void *weights;   // NULL: ones
  float *dw;
  Pieces pieces;         // of the T rows
  int64_t T;
  u32 k, H, R;
  int32_t w_f32;
};

__device__ __forceinline__ float route_weight(const RouteArgs &a, int64_t pair) {
  if (!a.weights) return 1.0f;
  return a.w_f32 ? *gptr(static_cast<const float *>(a.weights) + pair)
                 : to_f32(*gptr(static_cast<const uint16_t *>(a.weights) + pair));
}

// The row of pair `pair`: at least R where it is dropped.
__device__ __forceinline__ u32 route_row(const RouteArgs &a, int64_t pair) { return (u32)*gptr(a.rank + pair); }

template <class T>
__global__ __launch_bounds__(256) void k_dispatch(const RouteArgs a) {
  constexpr int VEC = 16 / (int)sizeof(T);
  for (int64_t first = (int64_t)blockIdx.x * 256; first < a.pieces.total; first += (int64_t)gridDim.x * 256) {
    if (first + threadIdx.x >= a.pieces.total) continue;
    int64_t t;
    u32 c;
    place_of(a.pieces, first, threadIdx.x, t, c);
    const u32 col = c * VEC;
    const int n = (int)min((u32)VEC, a.H - col);
    Piece<T, VEC> v;
    v.load(static_cast<const T *>(a.in) + t * a.ld_in + col, n);
    for (u32 j = 0; j < a.k; j++) {
      const u32 r = route_row(a, t * a.k + j);
      if (r < a.R) v.store(static_cast<T *>(a.out) + (int64_t)r * a.ld_out + col, n);
    }
  }
}

template <class T>
__global__ __launch_bounds__(256) void k_combine(const RouteArgs a) {
  constexpr int VEC = 16 / (int)sizeof(T);
  for (int64_t first = (int64_t)blockIdx.x * 256; first < a.pieces.total; first += (int64_t)gridDim.x * 256) {
    if (first + threadIdx.x >= a.pieces.total) continue;
    int64_t t;
    u32 c;
    place_of(a.pieces, first, threadIdx.x, t, c);
    const u32 col = c * VEC;
    const int n = (int)min((u32)VEC, a.H - col);
    float acc[VEC] = {};
    for (u32 j = 0; j < a.k; j++) {
      const int64_t pair = t * a.k + j;
      const u32 r = route_row(a, pair);
      if (r >= a.R) continue;
      const float w = route_weight(a, pair);
      Piece<T, VEC> v;
      v.load(static_cast<const T *>(a.in) + (int64_t)r * a.ld_in + col, n);
#pragma unroll
      for (int i = 0; i < VEC; i++) acc[i] = fmaf(w, v.get(i), acc[i]);
    }
    Piece<T, VEC> y;
    if (a.other) {
      y.load(static_cast<const T *>(a.other) + t * a.ld_other + col, n);
#pragma unroll
      for (int i = 0; i < VEC; i++) acc[i] += y.get(i);
    }
    y.set(acc);
    y.store(static_cast<T *>(a.out) + t * a.ld_out + col, n);
  }
}

// Combine's gradients: a wavefront takes a token, its lanes the pieces of the
// row, and up to 8 choices at a time.
template <class T>
__global__ __launch_bounds__(256) void k_combine_bwd(const RouteArgs a) {
  constexpr int VEC = 16 / (int)sizeof(T), K = 8;
  const u32 lane = threadIdx.x & 63, C = a.pieces.per.d;
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < a.T; t += (int64_t)gridDim.x * 4) {
    for (u32 j0 = 0; j0 < a.k; j0 += K) {
      float dot[K] = {};
      for (u32 c = lane; c < C; c += 64) {
        const u32 col = c * VEC;
        const int n = (int)min((u32)VEC, a.H - col);
        Piece<T, VEC> d;
        d.load(static_cast<const T *>(a.other) + t * a.ld_other + col, n);
#pragma unroll
        for (int j = 0; j < K; j++) {
          const int64_t pair = t * a.k + j0 + j;
          const u32 r = j0 + j < a.k ? route_row(a, pair) : ~0u;
          if (r >= a.R) continue;
          const float w = route_weight(a, pair);
          Piece<T, VEC> v;
          v.load(static_cast<const T *>(a.in) + (int64_t)r * a.ld_in + col, n);
          float o[VEC];
#pragma unroll
          for (int i = 0; i < VEC; i++) {
            dot[j] = fmaf(d.get(i), v.get(i), dot[j]);
            o[i] = w * d.get(i);
          }
          v.set(o);
          v.store(static_cast<T *>(a.out) + (int64_t)r * a.ld_out + col, n);
        }
      }
#pragma unroll
      for (int j = 0; j < K; j++) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) dot[j] += __shfl_xor(dot[j], o, 64);
        if (lane == 0 && j0 + j < a.k) *gptr(a.dw + t * a.k + j0 + j) = dot[j];
      }
    }
  }
}

}  // namespace mxt
