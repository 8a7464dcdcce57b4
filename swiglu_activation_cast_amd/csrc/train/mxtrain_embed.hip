// mxtrain_embed.hip -- C ABI of the embedding lookup and its gradient.
// Nothing is allocated, synchronized or read back, and no exception can leave
// an entry point (nothing here throws).
#include "mxtrain_tokens.h"
#include "tr_embed.hpp"
#include "tr_sort_run.hpp"

using namespace mxt;

namespace mxt {
namespace {

mxtrain_status embed_check(const void *table, int64_t ld_w, int w_type, const void *ids, int64_t id_stride,
                           int id_type, const void *tokens, int64_t ld_t, int t_type, int64_t T, int64_t first,
                           float scale, int64_t V, int64_t H) {
  if (!type_ok(w_type) || !type_ok(t_type) || (id_type != MXTRAIN_I32 && id_type != MXTRAIN_I64))
    return MXTRAIN_ERR_TYPE;
  if (!std::isfinite(scale)) return MXTRAIN_ERR_VALUE;
  if (T < 0 || V < 0 || H < 0 || T > INT32_MAX || V > INT32_MAX || H > INT32_MAX) return MXTRAIN_ERR_SHAPE;
  if (first > INT64_MAX - V) return MXTRAIN_ERR_VALUE;
  const bool has_t = T > 0 && H > 0, has_w = V > 0 && H > 0;
  if ((T > 0 && !ids) || (has_t && !tokens) || (has_w && !table)) return MXTRAIN_ERR_NULL;
  if ((has_t && ld_t < H) || (has_w && ld_w < H) || (T > 1 && id_stride < 0)) return MXTRAIN_ERR_STRIDE;
  if (!aligned(ids, id_type == MXTRAIN_I64 ? 8 : 4) || !aligned(tokens, (uintptr_t)size_of(t_type)) ||
      !aligned(table, (uintptr_t)size_of(w_type)))
    return MXTRAIN_ERR_ALIGN;
  if ((has_t && !extent_ok(T, H, ld_t)) || (has_w && !extent_ok(V, H, ld_w)) || !extent_ok(T, 1, id_stride))
    return MXTRAIN_ERR_OVERFLOW;
  return MXTRAIN_OK;
}

// Columns that a thread holds.
int64_t embed_vec(int t, int u, int64_t H) {
  const int64_t vec = t == MXTRAIN_F32 && u == MXTRAIN_F32 ? 4 : 8;
  return H < vec ? 1 : vec;
}

// fn<T, U, VEC>(...) for the rows' and the results' types.
#define EMBED_PICK(fn, vec, t_f32, u_f32, ...)                                                             \
  ((vec) == 1 ? (t_f32 ? (u_f32 ? fn<float, float, 1>(__VA_ARGS__) : fn<float, uint16_t, 1>(__VA_ARGS__))  \
                       : (u_f32 ? fn<uint16_t, float, 1>(__VA_ARGS__) : fn<uint16_t, uint16_t, 1>(__VA_ARGS__))) \
              : (t_f32 ? (u_f32 ? fn<float, float, 4>(__VA_ARGS__) : fn<float, uint16_t, 8>(__VA_ARGS__))  \
                       : (u_f32 ? fn<uint16_t, float, 8>(__VA_ARGS__) : fn<uint16_t, uint16_t, 8>(__VA_ARGS__))))

template <class T, class U, int VEC>
const void *lookup_kernel(bool many) {
  return many ? (const void *)&k_embed<T, U, VEC, 2> : (const void *)&k_embed<T, U, VEC, 1>;
}

template <class T, class U, int VEC>
const void *sum_kernel(bool nt) {
  if constexpr (VEC > 1)
    if (nt) return (const void *)&k_embed_bwd<T, U, VEC, true>;
  return (const void *)&k_embed_bwd<T, U, VEC, false>;
}

template <class T, class U, int VEC>
const void *few_kernel() {
  return (const void *)&k_embed_bwd_few<T, U, VEC>;
}

template <class T, class U, int VEC>
const void *join_kernel() {
  return (const void *)&k_embed_join<T, U, VEC>;
}

// Wavefronts that sum: as many workgroups as a launch takes join their parts.
constexpr int64_t kMaxJobs = INT32_MAX / 256;

// Few enough tokens for the gradient without a sort (and every strip of each has
// a workgroup).
bool embed_few(int64_t T, int64_t H, int64_t vec) {
  const int64_t strips = ((H + vec - 1) / vec + 63) / 64;
  return T <= kEmbedFew && T * strips <= kMaxJobs / 2;
}

// How the gradient cuts its work: chunks of 64 tokens, or fewer where that
// leaves less than sixteen wavefronts to a compute unit.
struct EmbedPlan {
  uint32_t rows, chunks, strips;
  int64_t flags, part, bytes;
};

EmbedPlan embed_plan(const SortPlan &sort, int64_t T, int64_t V, int64_t H, int64_t vec) {
  EmbedPlan p{};
  const int64_t strips = ((H + vec - 1) / vec + 63) / 64;
  int64_t rows = 64;
  while (rows > 8 && (T + rows - 1) / rows * strips < 4096) rows /= 2;
  p.rows = (uint32_t)rows;
  p.chunks = (uint32_t)((T + rows - 1) / rows);
  p.strips = (uint32_t)strips;
  p.flags = sort.bytes;
  p.part = p.flags + (V + 15) / 16 * 16;
  p.bytes = p.part + (p.chunks > 1 ? (int64_t)p.chunks * 2 * strips * 64 * vec * 4 : 0);
  return p;
}

}  // namespace
}  // namespace mxt

extern "C" {

mxtrain_status mxtrain_embedding_fwd(const void *weight, int64_t ld_w, int weight_type, int64_t V, int64_t H,
                                     const void *ids, int64_t id_stride, int id_type, int64_t T, int64_t first,
                                     float scale, void *y, int64_t ld_y, int y_type, void *stream) {
  const mxtrain_status st = embed_check(weight, ld_w, weight_type, ids, id_stride, id_type, y, ld_y, y_type, T, first,
                                        scale, V, H);
  if (st != MXTRAIN_OK) return st;
  if (T == 0 || H == 0) return MXTRAIN_OK;
  EmbedArgs a{};
  a.in = weight;
  a.out = y;
  a.ld_in = ld_w;
  a.ld_out = ld_y;
  a.ids = ids;
  a.id_stride = id_stride;
  a.ids_i64 = id_type == MXTRAIN_I64;
  a.first = first;
  a.V = (u32)V;
  a.H = (u32)H;
  a.T = (u32)T;
  a.scale = scale;
  const bool f = weight_type == MXTRAIN_F32, g = y_type == MXTRAIN_F32;
  const int64_t vec = embed_vec(weight_type, y_type, H), per = (H + vec - 1) / vec;
  a.pieces = {T * per, divider((uint32_t)per)};
  // two pieces a thread where that leaves every compute unit eight workgroups:
  // 16640 rows of 5120 bf16 51 us, 60 with one and 50 with four; 65537 of 2050 61
  // with two and 71 with four
  const bool many = a.pieces.total >= 2 * 256 * 2048;
  const void *kernel = EMBED_PICK(lookup_kernel, vec, f, g, many);
  const int64_t step = many ? 512 : 256;
  return launch(kernel, std::min<int64_t>((a.pieces.total + step - 1) / step, INT32_MAX / 256), 256, a, stream);
}

int64_t mxtrain_embedding_bwd_workspace(int64_t T, int64_t V, int64_t H, int dy_type, int dw_type) {
  if (!type_ok(dy_type) || !type_ok(dw_type) || T <= 0 || V <= 0 || H <= 0) return 0;
  if (T > INT32_MAX || V > INT32_MAX || H > INT32_MAX) return 0;
  const int64_t vec = embed_vec(dy_type, dw_type, H);
  if (embed_few(T, H, vec)) return 0;
  const EmbedPlan p = embed_plan(sort_plan(T, V, true), T, V, H, vec);
  return (int64_t)p.chunks * p.strips > kMaxJobs ? 0 : p.bytes;
}

mxtrain_status mxtrain_embedding_bwd(const void *dy, int64_t ld_dy, int dy_type, const void *ids, int64_t id_stride,
                                     int id_type, int64_t T, int64_t first, float scale, int64_t V, int64_t H,
                                     void *dweight, int64_t ld_dw, int dw_type, int accumulate, void *workspace,
                                     int64_t workspace_bytes, void *stream) {
  mxtrain_status st = embed_check(dweight, ld_dw, dw_type, ids, id_stride, id_type, dy, ld_dy, dy_type, T, first, scale,
                                  V, H);
  if (st != MXTRAIN_OK) return st;
  if (accumulate != 0 && accumulate != 1) return MXTRAIN_ERR_VALUE;
  if (V == 0 || H == 0 || (T == 0 && accumulate)) return MXTRAIN_OK;
  const SortPlan sp = sort_plan(T, V, true);
  const int64_t vec = embed_vec(dy_type, dw_type, H), zero_vec = vec == 1 ? 1 : 16 / size_of(dw_type);
  const EmbedPlan ep = embed_plan(sp, T, V, H, vec);
  const bool few = embed_few(T, H, vec);
  const int64_t jobs = (few ? T : (int64_t)ep.chunks) * ep.strips;
  if (jobs > kMaxJobs) return MXTRAIN_ERR_OVERFLOW;
  if (!few && !workspace) return MXTRAIN_ERR_NULL;
  if (!few && !aligned(workspace, 16)) return MXTRAIN_ERR_ALIGN;
  if (!few && workspace_bytes < ep.bytes) return MXTRAIN_ERR_WORKSPACE;
  const int64_t zero_per = (H + zero_vec - 1) / zero_vec, zeros = accumulate ? 0 : V * zero_per;
  const int64_t sum_blocks = few ? jobs : (jobs + 3) / 4;
  const int64_t zero_blocks = std::min<int64_t>((zeros + 255) / 256, INT32_MAX / 512);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  EmbedArgs a{};
  a.in = dy;
  a.out = dweight;
  a.ld_in = ld_dy;
  a.ld_out = ld_dw;
  a.V = (u32)V;
  a.H = (u32)H;
  a.T = (u32)T;
  a.scale = scale;
  a.keys = reinterpret_cast<u32 *>(ws + sp.keys);
  a.order = reinterpret_cast<u32 *>(ws + sp.order);
  a.part = reinterpret_cast<float *>(ws + ep.part);
  a.rows = ep.rows;
  a.chunks = ep.chunks;
  a.strips = ep.strips;
  a.jobs = (u32)jobs;
  a.sum_blocks = (u32)sum_blocks;
  a.zeros = {zeros, divider((uint32_t)zero_per)};
  a.flags = ws + ep.flags;
  a.accumulate = accumulate;
  a.ids = ids;
  a.id_stride = id_stride;
  a.ids_i64 = id_type == MXTRAIN_I64;
  a.first = first;
  const bool f = dy_type == MXTRAIN_F32, g = dw_type == MXTRAIN_F32;
  if (few) return launch(EMBED_PICK(few_kernel, vec, f, g), sum_blocks + zero_blocks, 256, a, stream);
  SortArgs s{};
  s.ids = ids;
  s.ld = id_stride;
  s.first = first;
  s.k = divider(1);
  s.ids_i64 = id_type == MXTRAIN_I64;
  s.n = (u32)T;
  s.n_keys = (u32)V;
  s.flags = accumulate ? nullptr : ws + ep.flags;
  s.order = reinterpret_cast<int32_t *>(ws + sp.order);
  s.key_out = reinterpret_cast<u32 *>(ws + sp.keys);
  if ((st = sort_run(sp, s, ws, stream)) != MXTRAIN_OK) return st;
  // 128 MB or more (half the last-level cache) are read past the caches: 65537 rows
  // of 2048 bf16 on 4099 words 92 us so, 96 otherwise, on 65 words 76 and 82
  const bool nt = (double)T * (double)H * size_of(dy_type) >= (double)(1 << 27);
  st = launch(EMBED_PICK(sum_kernel, vec, f, g, nt), sum_blocks + zero_blocks, 256, a, stream);
  if (st != MXTRAIN_OK || ep.chunks <= 1) return st;
  return launch(EMBED_PICK(join_kernel, vec, f, g), jobs, 256, a, stream);
}

}  // extern "C"
