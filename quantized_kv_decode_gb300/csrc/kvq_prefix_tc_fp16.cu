// Tensor-core attention over shared prefixes: fp16 caches.
#include "kvq_extend_tc.cuh"

namespace kvq {
cudaError_t run_prefix_tc_fp16(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream) {
  return ext::run_tc<16, 2, true>(D, nq, p, plan, stream);
}
}  // namespace kvq
