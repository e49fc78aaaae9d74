// Tensor-core attention of several new tokens: int2 caches.
#include "kvq_extend_tc.cuh"

namespace kvq {
cudaError_t run_extend_tc_int2(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream) {
  return ext::run_tc<2, 0>(D, nq, p, plan, stream);
}
}  // namespace kvq
