// mxtrain_sort.hip -- the stable sort's kernels and launches.
#include "tr_sort_run.hpp"

namespace mxt {

// One workgroup sorts everything (n <= kSortTile).  Bound by instructions, six for
// each bit of each item's digit: 8192 keys of 16 bits 18 us, 1000 8.
__global__ __launch_bounds__(kSortThreads) void k_sort_small(const SortArgs a) {
  __shared__ SortShared<16> sm;
  __shared__ u32 keys[kSortTile];
  __shared__ uint16_t items[kSortTile];
  const u32 lane = threadIdx.x & 63, w = threadIdx.x >> 6, mask = (1u << a.bits) - 1;
  // as few items a thread as hold n, so that the wavefronts share them
  const u32 each = (a.n + kSortThreads - 1) / kSortThreads;
  u32 key[kSortItems], item[kSortItems], digit[kSortItems], place[kSortItems];
  u32 total = 0, base = 0;
#pragma unroll
  for (int i = 0; i < kSortItems; i++) {
    const u32 p = (w * each + i) * 64 + lane;
    item[i] = (u32)i < each && p < a.n ? p : ~0u;
  }
  sort_clear_flags(a);
  sort_keys<kSortItems>(a, item, key);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // other wavefronts set what this one cleared
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSortItems; i++)
    if (item[i] != ~0u) sort_set_flag(a, key[i]);
  for (u32 pass = 0; pass < a.passes; pass++) {
    if (pass) {
#pragma unroll
      for (int i = 0; i < kSortItems; i++) {
        const u32 p = (w * each + i) * 64 + lane;
        if (item[i] == ~0u) continue;
        key[i] = keys[p];
        item[i] = items[p];
      }
    }
#pragma unroll
    for (int i = 0; i < kSortItems; i++) digit[i] = item[i] != ~0u ? key[i] >> (pass * a.bits) & mask : ~0u;
    total = rank_tile<16, kSortItems>(sm, digit, place, a.bits);
    base = block_scan<16>(total, sm.wave);
    if (threadIdx.x <= mask) sm.base[threadIdx.x] = base;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSortItems; i++) {
      if (item[i] == ~0u) continue;
      const u32 to = sm.base[digit[i]] + place[i];
      keys[to] = key[i];
      items[to] = (uint16_t)item[i];
      if (pass + 1 == a.passes) sort_rank(a, item[i], key[i], to);
    }
    __syncthreads();
  }
  // from LDS in order: scattered stores take the compute unit a cycle each
  for (u32 p = threadIdx.x; p < a.n; p += kSortThreads) sort_place(a, items[p], keys[p], p);
  if (!a.ends) return;
  if (a.passes == 1) {
    if (threadIdx.x < a.n_keys) *gptr(a.ends + threadIdx.x) = (int32_t)(base + total);
  } else {
    for (u32 v = threadIdx.x; v < a.n_keys; v += kSortThreads) *gptr(a.ends + v) = (int32_t)keys_up_to(keys, a.n, v);
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
  {
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
  a.passes = p.passes;
  if (p.small) return launch((const void *)&k_sort_small, 1, kSortThreads, a, stream);
  a.blocks = p.blocks;
  a.per = p.per;
  a.counts = reinterpret_cast<u32 *>(ws + p.counts);
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
    mxtrain_status st = launch((const void *)&k_sort_count, p.blocks, kSortThreads, a, stream);
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
