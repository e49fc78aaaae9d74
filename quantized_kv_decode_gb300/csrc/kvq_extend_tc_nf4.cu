// Tensor-core attention of several new tokens: nf4 caches.
#include "kvq_extend_tc.cuh"

namespace kvq {
cudaError_t run_extend_tc_nf4(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream) {
  return ext::run_tc<4, 1>(D, nq, p, plan, stream);
}
}  // namespace kvq
