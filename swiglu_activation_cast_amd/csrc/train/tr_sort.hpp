// tr_sort.hpp -- stable sort of small integer keys (gfx950): tokens by expert,
// tokens by word.
//
// An item's place is the number of items with a smaller key plus the number of
// earlier ones with the same.  A key is id - first, or n_keys where that is
// not in [0, n_keys): dropped items come last.  No order of execution enters, so
// the result is the one stable order.
//
// Few items are counted by comparing (up to 4096, or 8192 whose keys have more than
// 10 bits): every workgroup compares its items with all.  That is one launch, in which
// no workgroup waits for another.  Up to 32768 items with such long keys are sorted so
// in tiles of 1024, and a second launch seeks each item in the other tiles.
//
// Others are sorted by digits of at most 10 bits, least significant first.  Within a
// wavefront, the lanes with the same digit find each other by one ballot for each
// bit; a lane's place among them is the number of lower lanes, and the lowest adds
// their number to the wavefront's count of that digit.  The wavefronts' counts are
// then summed in order.  Items are dealt to up to 256 workgroups in contiguous
// ranges, and a pass is two launches: each workgroup counts its digits, and then each
// adds up the counts of all workgroups (from L2) to know its first place for every
// digit, and moves its items.  Up to 16384 items of one digit, each counts all of
// them itself, in one launch.
#pragma once
#include "tr_rows.hpp"

namespace mxt {

constexpr int kSortBits = 10;               // most bits of a digit
constexpr int kSortThreads = 1024;          // and, one digit a thread, of most digits
constexpr int kSortItems = 8;               // items a thread in one tile
constexpr int kSortTile = kSortThreads * kSortItems;
constexpr int kSortBlocks = 256;
constexpr int kSortMerge = 32768;           // most items that sorted tiles are merged of, all keys in LDS

struct SortArgs {
  const void *ids;  // the keys' source in the first pass: [n / k, k] with row stride ld
  int64_t ld, first;
  Divider k;
  int32_t ids_i64, adjacent;  // int64 ids; ld == k
  u32 n, n_keys;
  const u32 *key_in, *item_in;  // the source of later passes
  u32 *key_out, *item_out;      // the next pass's source; in the last pass the sorted keys, or NULL
  int32_t *order, *rank, *ends;  // written by the last pass, each may be NULL; ends only where one pass does
  uint8_t *flags;                // [n_keys], 1 where an item has that key; may be NULL
  u32 *counts;                   // [blocks][1 << bits]; NULL: every workgroup counts all items
  u32 shift, bits, blocks, per;  // this pass's digit; workgroups and items of each
  u32 tile, flag_range;          // without digits: items of a tile (0: all); words whose flags a workgroup writes
  int32_t is_first, is_last;
};

// Where item p's id is.
__device__ __forceinline__ int64_t sort_at(const SortArgs &a, u32 p) {
  if (a.adjacent) return p;
  const u32 t = a.k.div(p);
  return (int64_t)t * a.ld + (p - t * a.k.d);
}

// (first + n_keys fits 64 bits, so a difference that wraps is not below n_keys)
__device__ __forceinline__ u32 sort_key(const SortArgs &a, int64_t id) {
  const uint64_t key = (uint64_t)id - (uint64_t)a.first;
  return key < a.n_keys ? (u32)key : a.n_keys;
}

// Keys of the items p[i] of this thread (~0u: none), all loads in flight together.
template <int ITEMS>
__device__ __forceinline__ void sort_keys(const SortArgs &a, const u32 *p, u32 *key) {
  int64_t id[ITEMS];
  if (a.ids_i64) {
#pragma unroll
    for (int i = 0; i < ITEMS; i++)
      if (p[i] != ~0u) id[i] = *gptr(static_cast<const int64_t *>(a.ids) + sort_at(a, p[i]));
  } else {
#pragma unroll
    for (int i = 0; i < ITEMS; i++)
      if (p[i] != ~0u) id[i] = *gptr(static_cast<const int32_t *>(a.ids) + sort_at(a, p[i]));
  }
#pragma unroll
  for (int i = 0; i < ITEMS; i++) key[i] = p[i] != ~0u ? sort_key(a, id[i]) : 0;
}

// LDS of a workgroup of W wavefronts that ranks a tile.
template <int W>
struct SortShared {
  uint16_t count[W][W * 64];  // a tile has at most 8192 items
  u32 base[W * 64];           // first place of each digit
  u32 wave[W];
};

// Exclusive sum of v over the threads of the workgroup (one barrier inside; `sm`
// must not be in use).
template <int W>
__device__ __forceinline__ u32 block_scan(u32 v, u32 *sm) {
  const u32 lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  u32 s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const u32 t = __shfl_up(s, o, 64);
    if (lane >= (u32)o) s += t;
  }
  if (lane == 63) sm[w] = s;
  __syncthreads();
  u32 before = 0;
#pragma unroll
  for (int i = 0; i < W; i++) before += i < (int)w ? sm[i] : 0;
  return before + s - v;
}

// Ranks one tile: digit[i] of this thread's item i (~0u: none), items in the order
// (wavefront, i, lane).  place[i] becomes the number of earlier items of the tile
// with that digit; thread d of those below 1 << bits gets digit d's number of
// items.  Ends with a barrier.
template <int W, int ITEMS>
__device__ __forceinline__ u32 rank_tile(SortShared<W> &sm, const u32 *digit, u32 *place, u32 bits) {
  const u32 lane = threadIdx.x & 63, w = threadIdx.x >> 6, bins = 1u << bits;
  for (u32 d = lane; d < bins; d += 64) sm.count[w][d] = 0;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < ITEMS; i++) {
    const bool have = digit[i] != ~0u;
    const uint64_t any = __ballot(have);
    if (any == 0) break;
    // the lanes with this lane's digit (bits past the last are zero in every lane
    // and change nothing); these are most of a sort's instructions
    u32 same_lo = (u32)any, same_hi = (u32)(any >> 32);
    for (u32 b = 0; b < bits; b += 4)
#pragma unroll
      for (u32 e = 0; e < 4; e++) {
        const u32 one = (u32)__builtin_amdgcn_sbfe((int)digit[i], b + e, 1);  // 0 or ~0
        const uint64_t without = __ballot(one == 0);
        same_lo &= (u32)without ^ one;
        same_hi &= (u32)(without >> 32) ^ one;
      }
    const uint64_t same = (uint64_t)same_hi << 32 | same_lo;
    const u32 lower = __popcll(same & ((1ull << lane) - 1));
    if (have) {
      const u32 before = sm.count[w][digit[i]];
      place[i] = before + lower;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (lower == 0) sm.count[w][digit[i]] = (uint16_t)(before + __popcll(same));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  u32 total = 0;
  if (threadIdx.x < bins) {
    u32 c[W];
#pragma unroll
    for (int i = 0; i < W; i++) c[i] = sm.count[i][threadIdx.x];
#pragma unroll
    for (int i = 0; i < W; i++) {
      sm.count[i][threadIdx.x] = (uint16_t)total;
      total += c[i];
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < ITEMS; i++)
    if (digit[i] != ~0u) place[i] += sm.count[w][digit[i]];
  return total;
}

// The flags are cleared by the first kernel and set by the second (where one kernel
// sorts, it does both).
__device__ __forceinline__ void sort_clear_flags(const SortArgs &a) {
  if (!a.flags) return;  // 16 bytes at a time: they begin and end on multiples of it
  const int64_t step = (int64_t)gridDim.x * kSortThreads * 16;
  for (int64_t i = ((int64_t)blockIdx.x * kSortThreads + threadIdx.x) * 16; i < a.n_keys; i += step)
    *gptr(reinterpret_cast<u32x4_t *>(a.flags + i)) = u32x4_t{};
}

__device__ __forceinline__ void sort_set_flag(const SortArgs &a, u32 key) {
  if (a.flags && key < a.n_keys) *gptr(a.flags + key) = 1;
}

// Writes what the last pass leaves: the item of key `key` at `place` of the order.
__device__ __forceinline__ void sort_place(const SortArgs &a, u32 item, u32 key, u32 place) {
  if (a.order) *gptr(a.order + place) = key < a.n_keys ? (int32_t)item : -1;
  if (a.key_out) *gptr(a.key_out + place) = key;
}

__device__ __forceinline__ void sort_rank(const SortArgs &a, u32 item, u32 key, u32 place) {
  if (a.rank) *gptr(a.rank + item) = key < a.n_keys ? (int32_t)place : -1;
}

// Number of the n ascending keys that are at most `v`.
template <class P>
__device__ __forceinline__ u32 keys_up_to(P keys, u32 n, u32 v) {
  u32 lo = 0, hi = n;
  while (lo < hi) {
    const u32 mid = lo + (hi - lo) / 2;
    if (keys[mid] <= v) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

}  // namespace mxt
