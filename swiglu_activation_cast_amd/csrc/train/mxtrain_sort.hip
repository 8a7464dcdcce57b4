// mxtrain_sort.hip -- the stable sort's kernels and launches.
#include "tr_sort_run.hpp"

namespace mxt {

// A query's place is the number of keys before it.  A workgroup takes 32 QL queries
// and looks at all keys of their tile, each wavefront at a sixteenth and each half of
// its lanes at half of that.  Queries [0, n) are the items, n + g asks for the keys
// of at most g (one tile only).
// Bound by its loads' way up to about 1000 keys, then by instructions: two compare a
// key with 64 queries, and one LDS read brings four keys for 4 QL of them.  500 keys 4.6
// us, 2000 5.6, 4000 7.0, 8192 10.5; 16384 in tiles 6.9.  (Two queries a lane and quarters of the lanes:
// 0.3 us more for few keys, the same for many.)
template <int QL>
__global__ __launch_bounds__(kSortThreads) void k_sort_rank(const SortArgs a) {
  constexpr u32 kQ = 32 * QL, kMost = kSortTile / 16;
  __shared__ alignas(16) u32 keys[16][kMost + 8];  // (the halves begin in banks of their own)
  __shared__ u32 part[16][kQ];
  const u32 lane = threadIdx.x & 63, w = threadIdx.x >> 6, half = lane >> 5, col = lane & 31;
  const bool one = a.tile == 0;
  const u32 q0 = blockIdx.x * kQ, lo = one ? 0 : q0 / a.tile * a.tile, have = one ? a.n : min(a.tile, a.n - lo);
  // keys of a half (whole fours) and of a wavefront
  const u32 step = (have + 127) / 128 * 4, per = 2 * step, base = lo + w * per;
  u32 p[kSortItems], key[kSortItems], item[QL], mine[QL], count[QL] = {};
#pragma unroll
  for (int i = 0; i < kSortItems; i++) {
    const u32 at = half * step + i * 32 + col;
    p[i] = i * 32u + col < step && w * per + at < have ? base + at : ~0u;
  }
#pragma unroll
  for (int u = 0; u < QL; u++) {
    const u32 q = q0 + u * 32 + col;
    item[u] = q < a.n ? q : ~0u;
  }
  sort_keys<QL>(a, item, mine);
  sort_keys<kSortItems>(a, p, key);
  // one tile: the flags of a range of words are cleared and set by one workgroup
  const u32 f0 = blockIdx.x * a.flag_range, f1 = min(a.n_keys, f0 + a.flag_range);
  if (!one) sort_clear_flags(a);
  else if (a.flags)
    for (u32 v = f0 + threadIdx.x * 16; v < f1; v += kSortThreads * 16)
      *gptr(reinterpret_cast<u32x4_t *>(a.flags + v)) = u32x4_t{};
#pragma unroll
  for (int u = 0; u < QL; u++)
    if (item[u] == ~0u) {
      mine[u] = q0 + u * 32 + col - a.n + 1;
      item[u] = 0;
    }
#pragma unroll
  for (int i = 0; i < kSortItems; i++)
    if (i * 32u + col < step) keys[w][half * (step + 4) + i * 32 + col] = p[i] != ~0u ? key[i] : ~0u;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  // Earlier keys count where they are at most the query's, later ones where they are
  // less; fours that hold the item itself count as later, and the equal ones before
  // it are added.
  const u32 *const some = &keys[w][half * (step + 4)];
  const u32 first = base + half * step;
  auto compare = [&](bool mixed) {
    u32 border[QL];
#pragma unroll
    for (int u = 0; u < QL; u++) border[u] = mine[u] + (base + per <= item[u]);
    for (u32 j = 0; j < step; j += 4) {
      const u32x4_t k = *reinterpret_cast<const u32x4_t *>(some + j);
#pragma unroll
      for (int u = 0; u < QL; u++) {
        if (mixed) border[u] = mine[u] + (first + j + 4 <= item[u]);
#pragma unroll
        for (int e = 0; e < 4; e++) count[u] += k[e] < border[u];
      }
    }
  };
  if (base < q0 + kQ && base + per > q0) {
    compare(true);
#pragma unroll
    for (int u = 0; u < QL; u++) {
      const u32 four = (item[u] & ~3u) - first;
      if (four < step)
#pragma unroll
        for (u32 e = 0; e < 3; e++) count[u] += e < (item[u] & 3) && some[four + e] == mine[u];
    }
  } else {
    compare(false);
  }
#pragma unroll
  for (int u = 0; u < QL; u++) {
    count[u] += __shfl_xor(count[u], 32, 64);
    if (half == 0) part[w][u * 32 + col] = count[u];
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // other wavefronts set what this one cleared
  __syncthreads();
  if (one && a.flags)
#pragma unroll
    for (int i = 0; i < kSortItems; i++)
      if (p[i] != ~0u && key[i] >= f0 && key[i] < f1) *gptr(a.flags + key[i]) = 1;
#pragma unroll
  for (int u = 0; u < QL; u++) {
    if (w != (u32)u || half != 0) continue;
    u32 place = 0;
#pragma unroll
    for (int i = 0; i < 16; i++) place += part[i][u * 32 + col];
    const u32 q = q0 + u * 32 + col;
    if (q >= a.n) {
      if (a.ends && q - a.n < a.n_keys) *gptr(a.ends + (q - a.n)) = (int32_t)place;
    } else if (one) {
      sort_place(a, q, mine[u], place);
      sort_rank(a, q, mine[u], place);
    } else {
      *gptr(a.key_out + lo + place) = mine[u];
      *gptr(a.item_out + lo + place) = q;
    }
  }
}

// Places in the order of all items from tiles that are sorted: a workgroup holds
// all keys and seeks each of its a.per queries in each tile.  Queries [0, n) are the
// items tile by tile, n + g asks for the keys of at most g.  Bound by the way of its
// loads: 16384 keys 5.0 us, 32768 8.2.
__global__ __launch_bounds__(kSortThreads) void k_sort_merge(const SortArgs a) {
  __shared__ alignas(16) u32 keys[kSortMerge];
  __shared__ u32 part[kSortThreads];
  constexpr int kLoads = kSortMerge / kSortThreads / 4;
  u32x4_t k[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; i++) {
    const u32 at = (i * kSortThreads + threadIdx.x) * 4;  // (the workspace has room for whole fours)
    if (at < a.n) k[i] = *gptr(reinterpret_cast<const u32x4_t *>(a.key_in + at));
  }
  const u32 col = threadIdx.x & (a.per - 1), group = threadIdx.x / a.per, groups = kSortThreads / a.per;
  const u32 q = blockIdx.x * a.per + col, tiles = (a.n + a.tile - 1) / a.tile;
  const u32 item = q < a.n ? *gptr(a.item_in + q) : 0;
#pragma unroll
  for (int i = 0; i < kLoads; i++) {
    const u32 at = (i * kSortThreads + threadIdx.x) * 4;
    if (at < a.n) *reinterpret_cast<u32x4_t *>(keys + at) = k[i];
  }
  __syncthreads();
  const u32 own = q < a.n ? q / a.tile : ~0u, key = q < a.n ? keys[q] : q - a.n;
  u32 count = 0;
  for (u32 t = group; t < tiles; t += groups) {
    const u32 lo = t * a.tile, have = min(a.tile, a.n - lo);
    // bounds are after all keys of their value, items after those of earlier tiles
    const u32 border = key + (t < own);
    u32 at = 0;
    for (u32 step = a.tile; step; step >>= 1)
      if (at + step <= have && keys[lo + at + step - 1] < border) at += step;
    count += t == own ? q - lo : at;
  }
  part[threadIdx.x] = count;
  __syncthreads();
  if (threadIdx.x >= a.per) return;
  u32 place = 0;
  for (u32 g = 0; g < groups; g++) place += part[g * a.per + threadIdx.x];
  if (q < a.n) {
    sort_place(a, item, key, place);
    sort_rank(a, item, key, place);
    sort_set_flag(a, key);
  } else if (a.ends && q - a.n < a.n_keys) {
    *gptr(a.ends + (q - a.n)) = (int32_t)place;
  }
}

// Keys and items of the places p[i] (~0u: none) of a pass's source.
template <int ITEMS>
__device__ __forceinline__ void sort_source(const SortArgs &a, const u32 *p, u32 *key, u32 *item) {
  if (a.is_first) {
    sort_keys<ITEMS>(a, p, key);
#pragma unroll
    for (int i = 0; i < ITEMS; i++) item[i] = p[i];
  } else {
#pragma unroll
    for (int i = 0; i < ITEMS; i++)
      if (p[i] != ~0u) {
        key[i] = *gptr(a.key_in + p[i]);
        item[i] = *gptr(a.item_in + p[i]);
      }
  }
}

// counts[b][d]: items of workgroup b's range with digit d.  131072 pairs: 4.8 us,
// the launch and one load's way.
__global__ __launch_bounds__(kSortThreads) void k_sort_count(const SortArgs a) {
  __shared__ u32 count[1 << kSortBits];
  const u32 bins = 1u << a.bits, lo = blockIdx.x * a.per, hi = min(a.n, lo + a.per);
  if (threadIdx.x < bins) count[threadIdx.x] = 0;
  if (a.is_first) sort_clear_flags(a);
  __syncthreads();
  for (u32 p = lo + threadIdx.x; p < hi; p += kSortThreads) {
    u32 key, item;
    sort_source<1>(a, &p, &key, &item);
    atomicAdd(&count[key >> a.shift & (bins - 1)], 1u);
  }
  __syncthreads();
  if (threadIdx.x < bins) *gptr(a.counts + (blockIdx.x << a.bits) + threadIdx.x) = count[threadIdx.x];
}

// Moves workgroup b's range to its places.  Bound by the way of its loads, counts
// and items together, and eight barriers: 131072 pairs by 64 experts in 128
// workgroups 7.4 us (10 with the counts read one at a time).
__global__ __launch_bounds__(kSortThreads) void k_sort_move(const SortArgs a) {
  __shared__ SortShared<16> sm;
  __shared__ u32 sums[2][4 * kSortThreads];  // [groups][bins]
  const u32 lane = threadIdx.x & 63, w = threadIdx.x >> 6, bins = 1u << a.bits, mask = bins - 1;
  const u32 lo = blockIdx.x * a.per, hi = min(a.n, lo + a.per);
  u32 key[kSortItems], item[kSortItems], digit[kSortItems], place[kSortItems];
  // the places of a tile that this thread takes
  auto fetch = [&](u32 tile) {
    const u32 here = min(hi - tile, (u32)kSortTile), each = (here + kSortThreads - 1) / kSortThreads;
#pragma unroll
    for (int i = 0; i < kSortItems; i++) {
      const u32 p = (w * each + i) * 64 + lane;
      digit[i] = (u32)i < each && p < here ? tile + p : ~0u;
    }
    sort_source<kSortItems>(a, digit, key, item);
  };
  fetch(lo);  // in flight while the counts are added up
  if (!a.counts) {
    // Counts of the items from its range on, and before, in up to 16 copies for
    // different lanes, next to each other, so that a frequent digit is not added to by
    // one lane after the other (16384 equal keys 19.5 us with one copy, 8.1 so).
    const u32 copies = min(16u, 4 * kSortThreads / bins), copy = threadIdx.x & (copies - 1);
    for (u32 i = threadIdx.x; i < copies * bins; i += kSortThreads) sums[0][i] = sums[1][i] = 0;
    __syncthreads();
    for (u32 p0 = 0; p0 < a.n; p0 += kSortTile) {
      u32 p[kSortItems], k[kSortItems];
#pragma unroll
      for (int i = 0; i < kSortItems; i++) {
        p[i] = p0 + i * kSortThreads + threadIdx.x;
        p[i] = p[i] < a.n ? p[i] : ~0u;
      }
      sort_keys<kSortItems>(a, p, k);
#pragma unroll
      for (int i = 0; i < kSortItems; i++)
        if (p[i] != ~0u) atomicAdd(&sums[p[i] < lo ? 1 : 0][k[i] * copies + copy], 1u);
    }
    __syncthreads();
    u32 all = 0, before = 0;
    if (threadIdx.x < bins)
      for (u32 i = 0; i < copies; i++) {
        const u32 at = threadIdx.x * copies + ((i + threadIdx.x) & (copies - 1));
        before += sums[1][at];
        all += sums[0][at];
      }
    all += before;
    const u32 base = block_scan<16>(all, sm.wave);
    if (threadIdx.x < bins) sm.base[threadIdx.x] = base + before;
    if (a.ends && blockIdx.x == 0 && threadIdx.x < a.n_keys) *gptr(a.ends + threadIdx.x) = (int32_t)(base + all);
  } else {
    // A thread reads four digits' counts of every `rows`-th workgroup.  Lanes of a
    // wavefront with the same digits are added up there, then the wavefronts, or
    // groups of them that share a row, over LDS.
    const u32 quads = bins / 4, row = threadIdx.x / quads, rows = kSortThreads / quads;
    const u32 d = threadIdx.x % quads * 4, groups = min(16u, rows), group = min(row, w);
    u32x4_t all4 = {}, before4 = {};
#pragma unroll 8
    for (u32 b = row; b < a.blocks; b += rows) {
      const u32x4_t c = *gptr(reinterpret_cast<const u32x4_t *>(a.counts + (b << a.bits) + d));
      all4 += c;
      if (b < blockIdx.x) before4 += c;
    }
    for (u32 o = 32; o >= quads; o >>= 1)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        all4[i] += __shfl_xor(all4[i], o, 64);
        before4[i] += __shfl_xor(before4[i], o, 64);
      }
    if (quads >= 64 || lane < quads)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        sums[0][group * bins + d + i] = all4[i];
        sums[1][group * bins + d + i] = before4[i];
      }
    __syncthreads();
    u32 all = 0, before = 0;
    if (threadIdx.x < bins)
      for (u32 i = 0; i < groups; i++) {
        all += sums[0][i * bins + threadIdx.x];
        before += sums[1][i * bins + threadIdx.x];
      }
    const u32 base = block_scan<16>(all, sm.wave);
    if (threadIdx.x < bins) sm.base[threadIdx.x] = base + before;
    if (a.ends && blockIdx.x == 0 && threadIdx.x < a.n_keys) *gptr(a.ends + threadIdx.x) = (int32_t)(base + all);
  }
  for (u32 tile = lo; tile < hi; tile += kSortTile) {
    if (tile > lo) fetch(tile);
#pragma unroll
    for (int i = 0; i < kSortItems; i++) {
      if (digit[i] == ~0u) continue;
      if (a.is_first) sort_set_flag(a, key[i]);
      digit[i] = key[i] >> a.shift & mask;
    }
    const u32 total = rank_tile<16, kSortItems>(sm, digit, place, a.bits);
    // rank_tile's barriers also lie between sm.base's last write and here
#pragma unroll
    for (int i = 0; i < kSortItems; i++) {
      if (digit[i] == ~0u) continue;
      const u32 to = sm.base[digit[i]] + place[i];
      if (a.is_last) {
        sort_place(a, item[i], key[i], to);
        sort_rank(a, item[i], key[i], to);
      } else {
        *gptr(a.key_out + to) = key[i];
        *gptr(a.item_out + to) = item[i];
      }
    }
    __syncthreads();
    if (threadIdx.x < bins) sm.base[threadIdx.x] += total;
  }
}

// ends[v] from the n sorted keys.
__global__ __launch_bounds__(256) void k_sort_ends(const u32 *keys, u32 n, u32 n_keys, int32_t *ends) {
  for (u32 v = blockIdx.x * 256 + threadIdx.x; v < n_keys; v += gridDim.x * 256)
    *gptr(ends + v) = (int32_t)keys_up_to(gptr(keys), n, v);
}

mxtrain_status sort_run(const SortPlan &p, SortArgs a, uint8_t *ws, void *stream) {
  a.adjacent = a.ld == (int64_t)a.k.d;
  a.bits = p.bits;
  if (p.blocks == 0) {
    const int64_t bounds = a.ends ? a.n_keys : 0, queries = a.n + (p.tile ? 0 : bounds);
    // 128 queries a workgroup where 32 would be more workgroups than run at once
    const bool many = queries > 16384;
    const int64_t of = many ? 128 : 32, blocks = std::max<int64_t>(1, (queries + of - 1) / of);
    SortArgs r = a;
    r.tile = p.tile;
    if (p.tile) {
      r.key_out = reinterpret_cast<u32 *>(ws + p.pair[0]);
      r.item_out = r.key_out + (a.n + 3) / 4 * 4;
      r.ends = nullptr;
    } else {
      r.flag_range = (u32)((((int64_t)a.n_keys + blocks - 1) / blocks + 15) / 16 * 16);
    }
    const mxtrain_status st = launch(many ? (const void *)&k_sort_rank<4> : (const void *)&k_sort_rank<1>, blocks,
                                     kSortThreads, r, stream);
    if (st != MXTRAIN_OK || !p.tile) return st;
    a.tile = p.tile;
    a.key_in = r.key_out;
    a.item_in = r.item_out;
    // a compute unit holds one workgroup: no more of them than there are units
    a.per = 64;
    while (a.per < kSortThreads && (a.n + bounds + a.per - 1) / a.per > 256) a.per *= 2;
    return launch((const void *)&k_sort_merge, (a.n + bounds + a.per - 1) / a.per, kSortThreads, a, stream);
  }
  a.blocks = p.blocks;
  a.per = p.per;
  a.counts = p.recount ? nullptr : reinterpret_cast<u32 *>(ws + p.counts);
  int32_t *const ends = a.ends;
  u32 *const sorted = a.key_out ? a.key_out : p.passes > 1 ? reinterpret_cast<u32 *>(ws + p.keys) : nullptr;
  if (p.passes > 1) a.ends = nullptr;
  for (uint32_t pass = 0; pass < p.passes; pass++) {
    a.is_first = pass == 0;
    a.is_last = pass + 1 == p.passes;
    a.shift = pass * p.bits;
    if (!a.is_first) {
      a.key_in = reinterpret_cast<u32 *>(ws + p.pair[(pass - 1) % 2]);
      a.item_in = a.key_in + a.n;
    }
    a.key_out = a.is_last ? sorted : reinterpret_cast<u32 *>(ws + p.pair[pass % 2]);
    a.item_out = a.is_last ? nullptr : a.key_out + a.n;
    mxtrain_status st = MXTRAIN_OK;
    if (!p.recount) st = launch((const void *)&k_sort_count, p.blocks, kSortThreads, a, stream);
    if (st == MXTRAIN_OK) st = launch((const void *)&k_sort_move, p.blocks, kSortThreads, a, stream);
    if (st != MXTRAIN_OK) return st;
  }
  if (!ends || p.passes == 1) return MXTRAIN_OK;
  const u32 *keys = sorted;
  u32 n = a.n, n_keys = a.n_keys;
  int32_t *out = ends;
  void *kargs[] = {&keys, &n, &n_keys, &out};
  const unsigned grid = (unsigned)std::min<int64_t>((n_keys + 255) / 256, 2048);
  return hipLaunchKernel((const void *)&k_sort_ends, dim3(grid), dim3(256), kargs, 0, (hipStream_t)stream) == hipSuccess
             ? MXTRAIN_OK
             : MXTRAIN_ERR_LAUNCH;
}

}  // namespace mxt
