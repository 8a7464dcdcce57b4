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
// and a second kernel joins them in a fixed order.  Words without tokens (the sort
// flags those that have some) get their zeros from further workgroups of the first
// launch.
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
  u32 jobs;                 // summing wavefronts: chunks x strips
  const uint8_t *flags;     // [V], 1: the word has tokens
  Pieces zeros;             // of dW's rows, 16 bytes each
  u32 sum_blocks;           // workgroups that sum; those after them write zeros
  int32_t accumulate;
};

// Token t's row of the table; V where it is outside.
__device__ __forceinline__ u32 embed_key(const EmbedArgs &a, int64_t t) {
  const int64_t at = t * a.id_stride;
  const int64_t id = a.ids_i64 ? *gptr(static_cast<const int64_t *>(a.ids) + at)
                               : (int64_t)*gptr(static_cast<const int32_t *>(a.ids) + at);
  const uint64_t key = (uint64_t)id - (uint64_t)a.first;
  return key < a.V ? (u32)key : a.V;
}

// VEC, here and below: columns that a thread holds, 16 bytes of the narrower type,
// or 1 where rows are shorter than that.  N pieces a thread, whose loads of rows are
// in flight together (those of ids are not: embed_key branches on their type, and
// the compiler waits for each before the next): 16640 rows of 5120 bf16 out of 65536
// 50 us, 4.8 TB/s over the distinct rows and y; 16 of 8192 3.2 us.
template <class T, class U, int VEC, int N>
__global__ __launch_bounds__(256) void k_embed(const EmbedArgs a) {
  const int64_t step = (int64_t)gridDim.x * (256 * N);
  for (int64_t first = (int64_t)blockIdx.x * (256 * N); first < a.pieces.total; first += step) {
    int64_t t[N];
    u32 col[N];
    u32 key[N];
    Piece<T, VEC> w[N];
    const int have = (int)min((int64_t)N, (a.pieces.total - first - threadIdx.x + 255) / 256);
#pragma unroll
    for (int u = 0; u < N; u++) {
      if (u >= have) break;
      u32 c;
      place_of(a.pieces, first, u * 256 + threadIdx.x, t[u], c);
      col[u] = piece_col<VEC>(c, a.H);
      key[u] = embed_key(a, t[u]);
    }
#pragma unroll
    for (int u = 0; u < N; u++) {
      w[u].clear();
      if (u < have && key[u] < a.V)
        w[u].load(static_cast<const T *>(a.in) + (int64_t)key[u] * a.ld_in + col[u]);
    }
#pragma unroll
    for (int u = 0; u < N; u++) {
      if (u >= have) break;
      float v[VEC];
#pragma unroll
      for (int i = 0; i < VEC; i++) v[i] = key[u] < a.V ? w[u].get(i) * a.scale : 0.0f;
      Piece<U, VEC> y;
      y.set(v);
      y.store(static_cast<U *>(a.out) + t[u] * a.ld_out + col[u]);
    }
  }
}

// scale sum (+ what is there) into row `word`, at `piece`; elements that the
// piece before has too are added to by that one alone.
template <class U, int VEC>
__device__ __forceinline__ void embed_write(const EmbedArgs &a, u32 word, u32 piece, const float *sum) {
  const u32 col = piece_col<VEC>(piece, a.H);
  U *out = static_cast<U *>(a.out) + (int64_t)word * a.ld_out + col;
  float v[VEC];
  Piece<U, VEC> p;
  if (a.accumulate) {
    p.load(out);
#pragma unroll
    for (int i = 0; i < VEC; i++) v[i] = fmaf(a.scale, sum[i], p.get(i));
    p.set(v);
    if (col == piece * VEC) p.store(out);
    else p.store(out, (int)(piece * VEC - col), VEC);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i++) v[i] = a.scale * sum[i];
    p.set(v);
    p.store(out);
  }
}

// The parts of a chunk, at a piece's own place.
template <int VEC>
__device__ __forceinline__ float *embed_part(const EmbedArgs &a, u32 chunk, u32 which, u32 piece) {
  return a.part + ((int64_t)chunk * 2 + which) * a.strips * (64 * VEC) + piece * VEC;
}

// Zeros in the rows of words without tokens.  One store a thread, workgroup after
// workgroup: 16384 tokens on 65536 words x 5120 fp32 take 250 us so with the sort and
// the join, 58 more where wavefronts walk rows of their own (a front of single stores
// fills 1.3 GB at 6.5-6.8 TB/s, such rows at 5.3) and 107 more with stores through
// the caches.
template <class U, int VEC>
__device__ __forceinline__ void embed_zeros(const EmbedArgs &a) {
  constexpr int Z = VEC == 1 ? 1 : 16 / (int)sizeof(U);
  Piece<U, Z> zero;
  zero.clear();
  const int64_t step = (int64_t)(gridDim.x - a.sum_blocks) * 256;
  for (int64_t first = (int64_t)(blockIdx.x - a.sum_blocks) * 256; first < a.zeros.total; first += step) {
    if (first + threadIdx.x >= a.zeros.total) continue;
    int64_t v;
    u32 c;
    place_of(a.zeros, first, threadIdx.x, v, c);
    if (*gptr(a.flags + v)) continue;
    zero.store(static_cast<U *>(a.out) + v * a.ld_out + piece_col<Z>(c, a.H));
  }
}

// Part 0 of a chunk belongs to a word that began in an earlier chunk, part 1 to
// one that begins here and goes on in the next.
// 16384 tokens on 65536 words x 5120, bf16 into fp32: 230 us, 6.6 TB/s over dy and
// dW, most of it zeros; 65537 on 4099 x 2050 bf16: 65 us, 4.4 TB/s (rows that
// start at odd multiples of 4 bytes; 58 us at 2048 columns).
template <class T, class U, int VEC, bool NT>
__global__ __launch_bounds__(256) void k_embed_bwd(const EmbedArgs a) {
  if (blockIdx.x >= a.sum_blocks) {
    embed_zeros<U, VEC>(a);
    return;
  }
  const u32 lane = threadIdx.x & 63;
  const u32 job = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  if (job >= a.jobs) return;
  const u32 chunk = job / a.strips, strip = job - chunk * a.strips;
  const u32 lo = chunk * a.rows, count = min(a.rows, a.T - lo);
  // lane i holds token i of the chunk, and its word; those outside are sorted last
  const u32 mine = min(lane, count - 1);
  const u32 my_key = *gptr(a.keys + lo + mine), my_token = *gptr(a.order + lo + mine);
  const u32 valid = __popcll(__ballot(lane < count && my_key < a.V));
  if (valid == 0) return;
  const u32 before = lo ? *gptr(a.keys + lo - 1) : ~0u;
  const u32 after = lo + count < a.T ? *gptr(a.keys + lo + count) : ~0u;
  const u32 piece = strip * 64 + lane;
  const bool in = piece * VEC < a.H;
  const T *dy = static_cast<const T *>(a.in) + piece_col<VEC>(in ? piece : 0, a.H);
  float sum[VEC] = {};
  u32 word = __builtin_amdgcn_readlane(my_key, 0);
  bool began = word != before;  // the running word began in this chunk
  auto leave = [&](bool goes_on) {
    if (in) {
      if (!began || goes_on) {
        float *to = embed_part<VEC>(a, chunk, began ? 1 : 0, piece);
        Piece<float, VEC> p;
        p.set(sum);
        p.store(to);
      } else {
        embed_write<U, VEC>(a, word, piece, sum);
      }
    }
#pragma unroll
    for (int i = 0; i < VEC; i++) sum[i] = 0.0f;
  };
  // eight rows in flight; past the last one it is read again and not added
  constexpr int N = 8;
  for (u32 i0 = 0; i0 < valid; i0 += N) {
    Piece<T, VEC> d[N];
#pragma unroll
    for (int u = 0; u < N; u++) {
      const u32 token = __builtin_amdgcn_readlane(my_token, min(i0 + u, valid - 1));
      d[u].template load<NT>(dy + (int64_t)token * a.ld_in);
    }
#pragma unroll
    for (int u = 0; u < N; u++) {
      if (i0 + u >= valid) break;
      const u32 key = __builtin_amdgcn_readlane(my_key, i0 + u);
      if (key != word) {
        leave(false);
        word = key;
        began = true;
      }
#pragma unroll
      for (int j = 0; j < VEC; j++) sum[j] += d[u].get(j);
    }
  }
  leave(word == after);
}

// The gradient for up to 256 tokens in one launch, without a sort: a token's
// workgroup sums the rows of its word, unless an earlier token has that word.  Each
// wavefront looks through 64 tokens and sums what it finds there; the four sums are
// added in order.
// 256 tokens on 32768 words x 512 bf16: 8.5 us (13.8 with the sort), on 219 words x
// 555 4.5 (10.9), all of them one word x 2048 8.3 (10.7).
constexpr u32 kEmbedFew = 256;

// Zeros where no token has the word, 256 pieces (of at most 256 rows) at a time.
template <class U, int VEC>
__device__ __forceinline__ void embed_zeros_few(const EmbedArgs &a) {
  constexpr int Z = VEC == 1 ? 1 : 16 / (int)sizeof(U);
  __shared__ uint8_t named[256];
  Piece<U, Z> zero;
  zero.clear();
  const u32 key = threadIdx.x < a.T ? embed_key(a, threadIdx.x) : a.V;
  const int64_t step = (int64_t)(gridDim.x - a.sum_blocks) * 256;
  for (int64_t first = (int64_t)(blockIdx.x - a.sum_blocks) * 256; first < a.zeros.total; first += step) {
    int64_t v0, v;
    u32 c;
    place_of(a.zeros, first, 0, v0, c);
    named[threadIdx.x] = 0;
    __syncthreads();
    if (key < a.V && key >= v0 && key < v0 + 256) named[key - v0] = 1;
    __syncthreads();
    if (first + threadIdx.x < a.zeros.total) {
      place_of(a.zeros, first, threadIdx.x, v, c);
      if (!named[v - v0]) zero.store(static_cast<U *>(a.out) + v * a.ld_out + piece_col<Z>(c, a.H));
    }
    __syncthreads();  // before the marks are cleared again
  }
}

template <class T, class U, int VEC>
__global__ __launch_bounds__(256) void k_embed_bwd_few(const EmbedArgs a) {
  if (blockIdx.x >= a.sum_blocks) {
    embed_zeros_few<U, VEC>(a);
    return;
  }
  constexpr int N = 8;
  __shared__ float sm[4][64 * VEC];
  __shared__ u32 found[4];  // tokens of the word that a wavefront has; ~0u: it is not this token's to sum
  const u32 lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const u32 t = blockIdx.x / a.strips, strip = blockIdx.x - t * a.strips;
  const u32 word = embed_key(a, t);
  if (word >= a.V) return;
  const u32 i = wave * 64 + lane;
  uint64_t same = __ballot(i < a.T && embed_key(a, min(i, a.T - 1)) == word);
  const u32 mine = __ballot(i < t) & same ? ~0u : __popcll(same);
  if (lane == 0) found[wave] = mine;
  __syncthreads();
  const u32 f0 = found[0], f1 = found[1], f2 = found[2], f3 = found[3];
  if (f0 == ~0u || f1 == ~0u || f2 == ~0u || f3 == ~0u) return;
  const u32 piece = strip * 64 + lane;
  const bool in = piece * VEC < a.H;
  const T *dy = static_cast<const T *>(a.in) + piece_col<VEC>(in ? piece : 0, a.H);
  float sum[VEC] = {};
  while (same) {
    // eight rows in flight, in the order of the tokens; past the last one it is read
    // again and counts as zero
    const u32 count = __popcll(same);
    u32 token = 0;
    Piece<T, VEC> d[N];
#pragma unroll
    for (int u = 0; u < N; u++) {
      token = same ? wave * 64 + __builtin_ctzll(same) : token;
      same &= same - 1;
      d[u].load(dy + (int64_t)__builtin_amdgcn_readfirstlane(token) * a.ld_in);
    }
    // (no branches, behind which the compiler would move the loads)
#pragma unroll
    for (int u = 0; u < N; u++)
#pragma unroll
      for (int j = 0; j < VEC; j++) sum[j] += (u32)u < count ? d[u].get(j) : 0.0f;
  }
  if (mine == f0 + f1 + f2 + f3) {  // all of them are this wavefront's
    if (in) embed_write<U, VEC>(a, word, piece, sum);
    return;
  }
  // (where one wavefront has all, the others leave here)
  if ((f0 != 0) + (f1 != 0) + (f2 != 0) + (f3 != 0) < 2) return;
#pragma unroll
  for (int j = 0; j < VEC; j++) sm[wave][j * 64 + lane] = sum[j];
  __syncthreads();
  if (wave != 0 || !in) return;
#pragma unroll
  for (int j = 0; j < VEC; j++)
    sum[j] = ((sum[j] + sm[1][j * 64 + lane]) + sm[2][j * 64 + lane]) + sm[3][j * 64 + lane];
  embed_write<U, VEC>(a, word, piece, sum);
}

// Joins the parts of the word that begins in chunk blockIdx.x / strips and goes
// on: part 1 there, then part 0 of the chunks after it as far as the word goes.
// The four wavefronts take every fourth part, four or eight at a time, and their
// sums are added in order.
// 65537 tokens on 4099 words (a twentieth of them one word): 8 us.
template <class T, class U, int VEC>
__global__ __launch_bounds__(256) void k_embed_join(const EmbedArgs a) {
  __shared__ float sm[4][64 * VEC];
  const u32 chunk = blockIdx.x / a.strips, strip = blockIdx.x - chunk * a.strips;
  const u32 lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const u32 lo = chunk * a.rows, next = lo + a.rows;
  if (next >= a.T) return;
  // all that decides, in flight together: the word at the border and its
  // neighbours, and the first words of the 64 chunks after it
  const u32 word = *gptr(a.keys + next), last = *gptr(a.keys + next - 1);
  const u32 first = *gptr(a.keys + lo), before = *gptr(a.keys + max(lo, 1u) - 1);
  auto begins = [&](u32 c) { return *gptr(a.keys + (int64_t)min(c, a.chunks - 1) * a.rows); };
  u32 ahead = begins(chunk + 1 + lane);
  if (word >= a.V || last != word) return;                   // nothing goes on
  if (lo > 0 && first == word && before == word) return;     // it began earlier
  // chunks that begin with this word: those after `chunk` up to the first that does not
  u32 parts = 1;
  for (;;) {
    const uint64_t same = __ballot(chunk + parts + lane < a.chunks && ahead == word);
    const u32 n = same == ~0ull ? 64 : __builtin_ctzll(~same);
    parts += n;
    if (n < 64) break;
    ahead = begins(chunk + parts + lane);
  }
  const u32 piece = strip * 64 + lane;
  const bool in = piece * VEC < a.H;
  constexpr int N = VEC == 8 ? 4 : 8;
  float sum[VEC] = {};
  for (u32 i0 = wave; i0 < parts; i0 += 4 * N) {
    Piece<float, VEC> p[N];
#pragma unroll
    for (int u = 0; u < N; u++) {
      const u32 i = min(i0 + 4 * u, parts - 1);
      p[u].load(embed_part<VEC>(a, chunk + i, i == 0 ? 1 : 0, in ? piece : 0));
    }
#pragma unroll
    for (int u = 0; u < N; u++)
      if (i0 + 4 * u < parts)
#pragma unroll
        for (int j = 0; j < VEC; j++) sum[j] += p[u].get(j);
  }
#pragma unroll
  for (int j = 0; j < VEC; j++) sm[wave][j * 64 + lane] = sum[j];
  __syncthreads();
  if (wave != 0 || !in) return;
#pragma unroll
  for (int j = 0; j < VEC; j++)
    sum[j] = ((sum[j] + sm[1][j * 64 + lane]) + sm[2][j * 64 + lane]) + sm[3][j * 64 + lane];
  embed_write<U, VEC>(a, word, piece, sum);
}

}  // namespace mxt
