// Tensor-core attention over shared prefixes: nf4 caches.
#include "kvq_extend_tc.cuh"

namespace kvq {
cudaError_t run_prefix_tc_nf4(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream) {
  return ext::run_tc<4, 1, true>(D, nq, p, plan, stream);
}
}  // namespace kvq
