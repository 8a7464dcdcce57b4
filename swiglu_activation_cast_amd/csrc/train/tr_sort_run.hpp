// tr_sort_run.hpp -- the sort's plan (host).
#pragma once
#include "tr_host.hpp"
#include "tr_sort.hpp"

namespace mxt {

// Passes over digits of equal size, and where the workspace holds what (byte
// offsets).  `keep`: the caller wants sorted keys and order, held in the
// workspace too.
struct SortPlan {
  bool small;
  uint32_t passes, bits, blocks, per;
  int64_t counts, pair[2], keys, order, bytes;  // pair: keys and items between passes
};

inline SortPlan sort_plan(int64_t n, int64_t n_keys, bool keep) {
  SortPlan p{};
  uint32_t all = 1;
  while (all < 32 && (n_keys >> all) != 0) all++;  // n_keys itself is a key: the dropped items'
  p.passes = (all + kSortBits - 1) / kSortBits;
  p.bits = std::max(2u, (all + p.passes - 1) / p.passes);  // counts are read four digits at a time
  // One workgroup's pass over 8192 items takes longer than two launches (12 us
  // against 9), over 4096 less (8); two passes over 8192 about as long as four.
  p.small = n <= (p.passes == 1 ? kSortTile / 2 : kSortTile);
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
  if (!p.small) {
    // Each workgroup reads all workgroups' counts and moves its share of the items:
    // times that grow with blocks x digits and with n / blocks.  131072 pairs by
    // 1000 experts, rows of 64: 20 us with 43 workgroups, 25 with 128; by 300 17 and 19.
    const double even = 4.0 * std::sqrt((double)n / (double)(1 << p.bits));
    const int64_t most = std::min<int64_t>(kSortBlocks, std::max<int64_t>(16, (int64_t)even));
    const int64_t step = (n + most - 1) / most;
    p.per = (uint32_t)((step + kSortThreads - 1) / kSortThreads * kSortThreads);
    p.blocks = (uint32_t)((n + p.per - 1) / p.per);
    p.counts = take((int64_t)p.blocks << p.bits);
    for (int i = 0; i < 2; i++)
      if ((int)p.passes > i + 1) p.pair[i] = take(2 * n);
    // sorted keys, from which several passes find the ends
    if (!keep && p.passes > 1) p.keys = take(n);
  }
  p.bytes = at;
  return p;
}

// Sorts as `a` says (ids, ld, first, k, ids_i64, n, n_keys and the results set
// by the caller).
__attribute__((visibility("hidden"))) mxtrain_status sort_run(const SortPlan &p, SortArgs a, uint8_t *ws,
                                                              void *stream);

}  // namespace mxt
