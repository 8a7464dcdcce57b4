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
#include <type_traits>

#include "tr_sort.hpp"

namespace mxt {

struct RouteArgs {
  const void *in;        // x, ys, or (combine's gradients) ys
  const void *other;     // residual or NULL; dy
  void *out;             // xs, y, dys
  int64_t ld_in, ld_other, ld_out;
  const int32_t *rank;
  const void *weights;
  float *dw;
  Pieces pieces;         // of the T rows
  int64_t T;
  u32 k, H, R;
};

// Weight of pair `pair`; W void: none, ones.
template <class W>
__device__ __forceinline__ float route_weight(const RouteArgs &a, int64_t pair) {
  if constexpr (std::is_void_v<W>) return 1.0f;
  else return to_f32(*gptr(static_cast<const W *>(a.weights) + pair));
}

// The row of pair `pair`: at least R where it is dropped.
__device__ __forceinline__ u32 route_row(const RouteArgs &a, int64_t pair) { return (u32)*gptr(a.rank + pair); }

// A piece a thread, read once and written k times.  16384 tokens x 8, rows of 2048
// bf16: 103 us, 5.9 TB/s over x and xs (with two pieces a thread 3 us more).
//
// NT: stores past the caches, where rows begin at multiples of 64 bytes (those 103 us
// would be 118; rows of 544, 1056 and 2080 bf16, odd multiples of 64 bytes, take 30, 58
// and 109 us so, 36, 68 and 129 through the caches).  Other rows share such pieces
// of memory with their neighbours, which other workgroups write: rows of 257, 513 and
// 1025 bf16 take 26, 37 and 93 us with the sort through the caches, 39, 59 and 102 past
// them.
template <class T, int VEC, bool NT>
__global__ __launch_bounds__(256) void k_dispatch(const RouteArgs a) {
  for (int64_t first = (int64_t)blockIdx.x * 256; first < a.pieces.total; first += (int64_t)gridDim.x * 256) {
    if (first + threadIdx.x >= a.pieces.total) continue;
    int64_t t;
    u32 c;
    place_of(a.pieces, first, threadIdx.x, t, c);
    const u32 col = piece_col<VEC>(c, a.H);
    Piece<T, VEC> v;
    v.load(static_cast<const T *>(a.in) + t * a.ld_in + col);
    for (u32 j = 0; j < a.k; j++) {
      const u32 r = route_row(a, t * a.k + j);
      if (r < a.R) v.template store<NT>(static_cast<T *>(a.out) + (int64_t)r * a.ld_out + col);
    }
  }
}

// A piece of y a thread; four of its rows in flight together, summed in fp32 in the
// order of j.  16384 tokens x 8, rows of 2048 bf16, with the residual: 113 us, 5.9
// TB/s over ys, residual and y.  W void and no residual: dispatch's gradient.
template <class T, class W, int VEC, bool NT>
__global__ __launch_bounds__(256) void k_combine(const RouteArgs a) {
  constexpr int K = 4;
  for (int64_t first = (int64_t)blockIdx.x * 256; first < a.pieces.total; first += (int64_t)gridDim.x * 256) {
    if (first + threadIdx.x >= a.pieces.total) continue;
    int64_t t;
    u32 c;
    place_of(a.pieces, first, threadIdx.x, t, c);
    const u32 col = piece_col<VEC>(c, a.H);
    float acc[VEC] = {};
    for (u32 j0 = 0; j0 < a.k; j0 += K) {
      u32 r[K];
      float w[K];
      Piece<T, VEC> v[K];
#pragma unroll
      for (int j = 0; j < K; j++) {
        const int64_t pair = t * a.k + min(j0 + j, a.k - 1);
        const u32 row = route_row(a, pair);
        r[j] = j0 + j < a.k ? row : ~0u;
        w[j] = route_weight<W>(a, pair);
      }
#pragma unroll
      for (int j = 0; j < K; j++) {
        v[j].clear();
        if (r[j] < a.R) v[j].template load<NT>(static_cast<const T *>(a.in) + (int64_t)r[j] * a.ld_in + col);
      }
#pragma unroll
      for (int j = 0; j < K; j++)
        if (r[j] < a.R)
#pragma unroll
          for (int i = 0; i < VEC; i++) acc[i] = fmaf(w[j], v[j].get(i), acc[i]);
    }
    Piece<T, VEC> y;
    if (a.other) {
      y.template load<NT>(static_cast<const T *>(a.other) + t * a.ld_other + col);
#pragma unroll
      for (int i = 0; i < VEC; i++) acc[i] += y.get(i);
    }
    y.set(acc);
    y.store(static_cast<T *>(a.out) + t * a.ld_out + col);
  }
}

// Combine's gradients: a workgroup takes a token, its lanes the pieces of the
// row, and up to 8 choices at a time.  Lane j loads choice j's rank and weight, which
// are then uniform values: a dropped pair is a branch.  All eight rows are in flight
// before the first is used.  16384 tokens x 8, rows of 2048 bf16: 221 us, 5.2 TB/s
// over dy, ys and dys (at most as many bytes read as written, where a copy moves
// 4.6); with a wavefront to a token 243 us.
//
// Stores past the caches whatever the rows' alignment: rows of 257, 513, 1024, 1025
// and 2048 bf16 take 35, 72, 107, 132 and 220 us so, 43, 66, 113, 136 and 228 through
// the caches.
//
// L < 64: rows of at most L pieces, 256 / L tokens to a workgroup (16384 tokens x
// 8 rows of 130 bf16: 28 us with a wavefront to a token, 22 with 32 lanes).
template <class T, class W, int VEC, int L, bool NT>
__global__ __launch_bounds__((L == 64 ? 1024 : 256)) void k_combine_bwd(const RouteArgs a) {
  constexpr int K = 8;
  __shared__ float sm[L == 64 ? 16 : 1][K];
  const u32 lane = threadIdx.x % L, wave = threadIdx.x >> 6, waves = blockDim.x >> 6, C = a.pieces.per.d;
  const u32 step = L == 64 ? blockDim.x : L;  // pieces at a time
  constexpr int kTokens = 256 / L;
  const int64_t t0 = L == 64 ? blockIdx.x : (int64_t)blockIdx.x * kTokens + threadIdx.x / L;
  for (int64_t t = t0; t < a.T; t += (int64_t)gridDim.x * (L == 64 ? 1 : kTokens)) {
    for (u32 j0 = 0; j0 < a.k; j0 += K) {
      u32 r[K];
      float w[K], dot[K] = {};
      {
        const int64_t pair = t * a.k + min(j0 + lane, a.k - 1);
        const u32 row = route_row(a, pair);
        const float weight = route_weight<W>(a, pair);
#pragma unroll
        for (int j = 0; j < K; j++) {
          if constexpr (L == 64) {
            r[j] = __builtin_amdgcn_readlane(row, j);
            w[j] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weight), j));
          } else {
            r[j] = __shfl(row, j, L);
            w[j] = __shfl(weight, j, L);
          }
          if (j0 + j >= a.k) r[j] = ~0u;
        }
      }
      for (u32 c = L == 64 ? threadIdx.x : lane; c < C; c += step) {
        const u32 col = piece_col<VEC>(c, a.H);
        Piece<T, VEC> d, v[K];
        d.template load<NT>(static_cast<const T *>(a.other) + t * a.ld_other + col);
#pragma unroll
        for (int j = 0; j < K; j++)
          if (r[j] < a.R) v[j].template load<NT>(static_cast<const T *>(a.in) + (int64_t)r[j] * a.ld_in + col);
        const int shared = (int)(c * VEC - col);  // elements that the piece before counts
#pragma unroll
        for (int j = 0; j < K; j++) {
          if (r[j] >= a.R) continue;
          float o[VEC];
#pragma unroll
          for (int i = 0; i < VEC; i++) o[i] = w[j] * d.get(i);
          Piece<T, VEC> q;
          q.set(o);
          q.store(static_cast<T *>(a.out) + (int64_t)r[j] * a.ld_out + col);
          if (a.H % VEC == 0) {
#pragma unroll
            for (int i = 0; i < VEC; i++) dot[j] = fmaf(d.get(i), v[j].get(i), dot[j]);
          } else {
#pragma unroll
            for (int i = 0; i < VEC; i++)
              dot[j] = i >= shared ? fmaf(d.get(i), v[j].get(i), dot[j]) : dot[j];
          }
        }
      }
#pragma unroll
      for (int j = 0; j < K; j++) {
        if (j0 + j >= a.k) break;
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) dot[j] += __shfl_xor(dot[j], o, 64);
        if (L < 64 || waves == 1) {
          if (lane == 0) *gptr(a.dw + t * a.k + j0 + j) = dot[j];
        } else if (lane == 0) {
          sm[wave][j] = dot[j];
        }
      }
      if (L == 64 && waves > 1) {
        __syncthreads();
        if (threadIdx.x < K && j0 + threadIdx.x < a.k) {
          float sum = 0.0f;
          for (u32 i = 0; i < waves; i++) sum += sm[i][threadIdx.x];
          *gptr(a.dw + t * a.k + j0 + threadIdx.x) = sum;
        }
        __syncthreads();
      }
    }
  }
}

// The sort and the dispatch in one launch, for up to 2048 pairs (ITEMS for each of
// 256 threads) of up to 255 groups: every workgroup ranks all pairs for itself, the
// first writes the result down.  8 x 2 pairs, rows of 5120 bf16: 4.0 us (two
// launches 6.1); 128 x 8 of 2048 5.9 (8.4); 256 x 8 8.0 (9.3); 1000 x 2 of 4096 10.8
// (9.4, and 3 us more of the host's time).
//
// Stores past the caches whatever the rows' alignment: 256 x 8 rows of 513, 1024 and
// 1025 bf16 take 7.9, 7.5 and 8.2 us so, 7.7, 7.7 and 7.9 through the caches, 2000
// rows of 4096 and 4099 12.2 and 12.8, 12.9 and 13.4.
constexpr int kFewPairs = 2048, kFewGroups = 255;

struct SortDispatchArgs {
  SortArgs sort;
  RouteArgs move;
};

template <class T, int VEC, int ITEMS>
__global__ __launch_bounds__(256) void k_sort_dispatch(const SortDispatchArgs g) {
  const SortArgs &s = g.sort;
  const RouteArgs &a = g.move;
  __shared__ SortShared<4> sm;
  __shared__ uint16_t rank[ITEMS * 256];
  const u32 lane = threadIdx.x & 63, w = threadIdx.x >> 6, each = (s.n + 255) / 256;
  u32 item[ITEMS], key[ITEMS], digit[ITEMS], place[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; i++) {
    const u32 p = (w * each + i) * 64 + lane;
    item[i] = (u32)i < each && p < s.n ? p : ~0u;
  }
  sort_keys<ITEMS>(s, item, key);
#pragma unroll
  for (int i = 0; i < ITEMS; i++) digit[i] = item[i] != ~0u ? key[i] : ~0u;
  const u32 total = rank_tile<4, ITEMS>(sm, digit, place, s.bits), base = block_scan<4>(total, sm.wave);
  sm.base[threadIdx.x] = base;
  if (blockIdx.x == 0 && threadIdx.x < s.n_keys) *gptr(s.ends + threadIdx.x) = (int32_t)(base + total);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < ITEMS; i++) {
    if (item[i] == ~0u) continue;
    const u32 to = sm.base[digit[i]] + place[i];
    rank[item[i]] = key[i] < s.n_keys ? (uint16_t)to : (uint16_t)0xffff;
    if (blockIdx.x != 0) continue;
    sort_place(s, item[i], key[i], to);
    sort_rank(s, item[i], key[i], to);
  }
  __syncthreads();
  for (int64_t first = (int64_t)blockIdx.x * 256; first < a.pieces.total; first += (int64_t)gridDim.x * 256) {
    if (first + threadIdx.x >= a.pieces.total) continue;
    int64_t t;
    u32 c;
    place_of(a.pieces, first, threadIdx.x, t, c);
    const u32 col = piece_col<VEC>(c, a.H);
    Piece<T, VEC> v;
    v.load(static_cast<const T *>(a.in) + t * a.ld_in + col);
    for (u32 j = 0; j < a.k; j++) {
      const u32 r = rank[(u32)t * a.k + j];
      if (r != 0xffff) v.store(static_cast<T *>(a.out) + (int64_t)r * a.ld_out + col);
    }
  }
}

}  // namespace mxt
