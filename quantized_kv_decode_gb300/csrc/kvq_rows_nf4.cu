// Attention of few rows over shared prefixes, codes in registers: nf4 caches.
#include "kvq_rows.cuh"

namespace kvq {
cudaError_t run_rows_nf4(int D, int mt, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream) {
  return rows::run_rows<4, 1>(D, mt, p, plan, stream);
}
}  // namespace kvq
