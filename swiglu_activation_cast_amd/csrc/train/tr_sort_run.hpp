// tr_sort_run.hpp -- the sort's plan (host).
#pragma once
#include "tr_host.hpp"
#include "tr_sort.hpp"

namespace mxt {

// How items are sorted, and where the workspace holds what (byte offsets).
// blocks == 0: by comparing, in tiles of `tile` items that are merged, or all at
// once (tile == 0).  Otherwise in passes over digits of equal size by workgroups
// with `per` items each, which count all items themselves (recount) or leave their
// counts for each other.  `keep`: the caller wants sorted keys and order, held in
// the workspace too.
struct SortPlan {
  uint32_t passes, bits, blocks, per, tile;
  bool recount;
  int64_t counts, pair[2], keys, order, bytes;  // pair: keys and items between passes
};

inline SortPlan sort_plan(int64_t n, int64_t n_keys, bool keep) {
  SortPlan p{};
  uint32_t all = 1;
  while (all < 32 && (n_keys >> all) != 0) all++;  // n_keys itself is a key: the dropped items'
  p.passes = (all + kSortBits - 1) / kSortBits;
  p.bits = std::max(2u, (all + p.passes - 1) / p.passes);  // counts are read four digits at a time
  int64_t at = 0;
  auto take = [&](int64_t words) {
    const int64_t here = at;
    at += (words * 4 + 15) / 16 * 16;
    return here;
  };
  if (keep) {
    p.keys = take(n);
    p.order = take(n);
  }
  // Comparing grows with n^2 (and n times the bounds for the ends), but its first
  // launch is the last: the embedding's gradient of 8000 keys of 16 bits, rows of 64,
  // takes 18.6 us so and 27.0 by digits; in tiles 16384 take 22.6 (28.6) and 32768
  // 32.1 (35.2).  One digit takes half as many launches: the sort and move of 2080
  // pairs 8.2 (8.8), but of 4096 9.5 (9.1) and 8192 15.7 (9.7).
  const int64_t queries = n + (keep ? 0 : n_keys);
  if (n <= (p.passes == 1 ? kSortTile / 2 : kSortTile) && n * queries <= 2 * (int64_t)kSortTile * kSortTile) {
    p.bytes = at;
    return p;
  }
  if (p.passes > 1 && n <= kSortMerge) {
    p.tile = kSortThreads;
    p.pair[0] = take(2 * ((n + 3) / 4 * 4));
    p.bytes = at;
    return p;
  }
  // One launch where workgroups of 256 items can count all items each: 8192 pairs by
  // 64 experts and their move 10.0 us, 11.5 in two launches, by 1000 11.4 and 13.3;
  // 16384 11.5 and 11.7.  (The flags need a launch before the one that sets them.)
  p.recount = p.passes == 1 && n <= 2 * kSortTile && !keep;
  if (p.recount) {
    p.per = 256;
  } else {
    // Each workgroup reads all workgroups' counts and moves its share of the items:
    // times that grow with blocks x digits and with n / blocks.  131072 pairs by
    // 1000 experts, rows of 64: 20 us with 43 workgroups, 25 with 128; by 300 17 and 19.
    const double even = 4.0 * std::sqrt((double)n / (double)(1 << p.bits));
    const int64_t most = std::min<int64_t>(kSortBlocks, std::max<int64_t>(16, (int64_t)even));
    const int64_t step = (n + most - 1) / most;
    p.per = (uint32_t)((step + kSortThreads - 1) / kSortThreads * kSortThreads);
  }
  p.blocks = (uint32_t)((n + p.per - 1) / p.per);
  if (!p.recount) p.counts = take((int64_t)p.blocks << p.bits);
  for (int i = 0; i < 2; i++)
    if ((int)p.passes > i + 1) p.pair[i] = take(2 * n);
  // sorted keys, from which several passes find the ends
  if (!keep && p.passes > 1) p.keys = take(n);
  p.bytes = at;
  return p;
}

// Sorts as `a` says (ids, ld, first, k, ids_i64, n, n_keys and the results set
// by the caller).
__attribute__((visibility("hidden"))) mxtrain_status sort_run(const SortPlan &p, SortArgs a, uint8_t *ws,
                                                              void *stream);

}  // namespace mxt
