// tr_embed.hpp -- embedding lookup and its gradient (gfx950).
//
//   y[t] = scale W[id_t - first]            (zeros outside the table)
//   dW[v] = scale sum over t with id_t - first = v of dy[t]
//
// Bound by HBM.  For the gradient the tokens are sorted by word, so that a
// word's rows are summed in a fixed order without atomics.  The sorted tokens
// are cut into chunks of at most 64; a wavefront takes a chunk and 64 pieces of the
// columns, keeps the running sum in registers and writes it where the word
// changes.  A word whose rows lie in several chunks leaves an fp32 part in each,
// and a second kernel joins them in order.  Words without tokens get their zeros
// from further workgroups of the first launch.
#pragma once
#include "tr_sort.hpp"

namespace mxt {

struct EmbedArgs {
  const void *in;  // W, or dy
  void *out;       // y, or dW
  int64_t ld_in, ld_out;
  const void *ids;
  int64_t id_stride, first;
  int32_t ids_i64;
  u32 V, H, T;
  float scale;
  Pieces pieces;  // of y's rows
  // gradient
  const u32 *keys, *order;  // sorted words (V: outside) and their tokens
  float *part;              // [chunks][2][strips * 64 * VEC]
  u32 rows;                 // tokens of a chunk
  u32 chunks, strips;       // and of the columns, 64 pieces each
  u32 sum_blocks;           // workgroups that sum; those after them write zeros
  int32_t accumulate;
};

// Columns that a thread holds: 16 bytes of the narrower type.
template <class T, class U>
constexpr int kEmbedVec = sizeof(T) == 4 && sizeof(U) == 4 ? 4 : 8;

template <class T, class U>
__global__ __launch_bounds__(256) void k_embed(const EmbedArgs a) {
  constexpr int VEC = kEmbedVec<T, U>;
  for (int64_t first = (int64_t)blockIdx.x * 256; first < a.pieces.total; first += (int64_t)gridDim.x * 256) {
    if (first + threadIdx.x >= a.pieces.total) continue;
    int64_t t;
    u32 c;
    place_of(a.pieces, first, threadIdx.x, t, c);
    const u32 col = c * VEC;
    const int n = (int)min((u32)VEC, a.H - col);
    const int64_t at = t * a.id_stride;
    const int64_t id = a.ids_i64 ? *gptr(static_cast<const int64_t *>(a.ids) + at)
                                 : (int64_t)*gptr(static_cast<const int32_t *>(a.ids) + at);
    const uint64_t key = (uint64_t)id - (uint64_t)a.first;
    Piece<T, VEC> w;
    w.clear();
    if (key < a.V) w.load(static_cast<const T *>(a.in) + (int64_t)key * a.ld_in + col, n);
    float v[VEC];
#pragma unroll
    for (int i = 0; i < VEC; i++) v[i] = key < a.V ? w.get(i) * a.scale : 0.0f;
    Piece<U, VEC> y;
    y.set(v);
    y.store(static_cast<U *>(a.out) + t * a.ld_out + col, n);
  }
}

// scale sum (+ what is there) into row `word`.
template <class U, int VEC>
__device__ __forceinline__ void embed_write(const EmbedArgs &a, u32 word, u32 col, int n, const float *sum) {
  U *out = static_cast<U *>(a.out) + (int64_t)word * a.ld_out + col;
  float v[VEC];
  Piece<U, VEC> p;
  if (a.accumulate) {
    p.load(out, n);
#pragma unroll
    for (int i = 0; i < VEC; i++) v[i] = fmaf(a.scale, sum[i], p.get(i));
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i++) v[i] = a.scale * sum[i];
  }
  p.set(v);
  p.store(out, n);
}

template <int VEC>
__device__ __forceinline__ float *embed_part(const EmbedArgs &a, u32 chunk, u32 which, u32 col) {
  return a.part + ((int64_t)chunk * 2 + which) * a.strips * (64 * VEC) + col;
}

// Zeros in the rows of words without tokens, 64 words a workgroup.
template <class U>
__device__ __forceinline__ void embed_zeros(const EmbedArgs &a, u32 block) {
  constexpr int VEC = 16 / (int)sizeof(U);
  const u32 lane = threadIdx.x & 63, v0 = block * 64, v = v0 + lane;
  const u32 upto = keys_up_to(gptr(a.keys), a.T, v);
  const uint64_t named = __ballot(v >= a.V || (upto > 0 && *gptr(a.keys + upto - 1) == v));
  Piece<U, VEC> zero;
  zero.clear();
  for (u32 i = threadIdx.x >> 6; i < 64; i += 4) {
    if (named >> i & 1) continue;
    U *row = static_cast<U *>(a.out) + (int64_t)(v0 + i) * a.ld_out;
    for (u32 col = lane * VEC; col < a.H; col += 64 * VEC) zero.store(row + col, (int)min((u32)VEC, a.H - col));
  }
}

// Part 0 of a chunk belongs to a word that began in an earlier chunk, part 1 to
// one that begins here and goes on in the next.
template <class T, class U>
__global__ __launch_bounds__(256) void k_embed_bwd(const EmbedArgs a) {
  constexpr int VEC = kEmbedVec<T, U>;
  if (blockIdx.x >= a.sum_blocks) {
    embed_zeros<U>(a, blockIdx.x - a.sum_blocks);
    return;
  }
  const u32 lane = threadIdx.x & 63;
  const u32 job = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const u32 chunk = job / a.strips, strip = job - chunk * a.strips;
  if (chunk >= a.chunks) return;
  const u32 lo = chunk * a.rows, count = min(a.rows, a.T - lo);
  const u32 col = (strip * 64 + lane) * VEC;
  const bool in = col < a.H;
  const int n = in ? (int)min((u32)VEC, a.H - col) : 1;
  // lane i holds token i of the chunk, and its word
  const u32 mine = min(lane, count - 1);
  const u32 my_key = *gptr(a.keys + lo + mine), my_token = *gptr(a.order + lo + mine);
  const u32 before = lo ? *gptr(a.keys + lo - 1) : ~0u;
  const u32 after = lo + count < a.T ? *gptr(a.keys + lo + count) : ~0u;
  float sum[VEC] = {};
  bool began = false;  // the running word began in this chunk
  u32 word = __builtin_amdgcn_readlane(my_key, 0);
  began = word != before;
  auto leave = [&](bool goes_on) {
    if (in) {
      if (!began || goes_on) {
        float *to = embed_part<VEC>(a, chunk, began ? 1 : 0, col);
#pragma unroll
        for (int i = 0; i < VEC; i += 4)
          *gptr(reinterpret_cast<f32x4_t *>(to + i)) = f32x4_t{sum[i], sum[i + 1], sum[i + 2], sum[i + 3]};
      } else {
        embed_write<U, VEC>(a, word, col, n, sum);
      }
    }
#pragma unroll
    for (int i = 0; i < VEC; i++) sum[i] = 0.0f;
  };
  for (u32 i = 0; i < count; i++) {
    const u32 key = __builtin_amdgcn_readlane(my_key, i), token = __builtin_amdgcn_readlane(my_token, i);
    if (key != word) {
      if (word < a.V) leave(false);
      word = key;
      began = true;
    }
    if (word >= a.V) break;  // sorted last
    if (in) {
      Piece<T, VEC> d;
      d.load(static_cast<const T *>(a.in) + (int64_t)token * a.ld_in + col, n);
#pragma unroll
      for (int j = 0; j < VEC; j++) sum[j] += d.get(j);
    }
  }
  if (word < a.V) leave(word == after);
}

// Joins the parts of the word that begins in chunk blockIdx.x / strips and goes
// on: part 1 there, then part 0 of the chunks after it as far as the word goes.
template <class T, class U>
__global__ __launch_bounds__(64) void k_embed_join(const EmbedArgs a) {
  constexpr int VEC = kEmbedVec<T, U>;
  const u32 chunk = blockIdx.x / a.strips, strip = blockIdx.x - chunk * a.strips;
  const u32 lo = chunk * a.rows, next = lo + a.rows;
  if (next >= a.T) return;
  const u32 word = *gptr(a.keys + next);
  if (word >= a.V || *gptr(a.keys + next - 1) != word) return;  // nothing goes on
  if (*gptr(a.keys + lo) == word && lo > 0 && *gptr(a.keys + lo - 1) == word) return;  // it began earlier
  const u32 col = (strip * 64 + threadIdx.x) * VEC;
  if (col >= a.H) return;
  float sum[VEC];
  const float *p = embed_part<VEC>(a, chunk, 1, col);
#pragma unroll
  for (int i = 0; i < VEC; i++) sum[i] = *gptr(p + i);
  for (u32 c = chunk + 1; c < a.chunks && *gptr(a.keys + c * a.rows) == word; c++) {
    p = embed_part<VEC>(a, c, 0, col);
#pragma unroll
    for (int i = 0; i < VEC; i++) sum[i] += *gptr(p + i);
  }
  embed_write<U, VEC>(a, word, col, (int)min((u32)VEC, a.H - col), sum);
}

}  // namespace mxt
