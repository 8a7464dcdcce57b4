// mxtrain_ortho_f32.hip -- the Newton-Schulz steps for fp32 results: two fp16 planes.
#include "tr_ortho_run.hpp"

namespace mxt {
template mxtrain_status ns_run<true>(const NsPlan &pl, mxt::NsArgs n, int64_t batch, int64_t m, int64_t cols, int steps,
                      const float *co, void *out, int64_t ld_out, int64_t stride_out, uint8_t *ws, void *stream);
}  // namespace mxt
