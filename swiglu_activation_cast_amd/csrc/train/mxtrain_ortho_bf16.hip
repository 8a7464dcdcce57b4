// mxtrain_ortho_bf16.hip -- the Newton-Schulz steps for bf16 results: X in two
// fp16 planes, S and p(S) in one.
#include "tr_ortho_run.hpp"

namespace mxt {
template mxtrain_status ns_run<false>(const NsPlan &pl, mxt::NsArgs n, int64_t batch, int64_t m, int64_t cols, int steps,
                      const float *co, void *out, int64_t ld_out, int64_t stride_out, uint8_t *ws, void *stream);
}  // namespace mxt
