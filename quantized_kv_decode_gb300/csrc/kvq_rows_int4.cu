// Attention of few rows over shared prefixes, codes in registers: int4 caches.
#include "kvq_rows.cuh"

namespace kvq {
cudaError_t run_rows_int4(int D, int mt, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream) {
  return rows::run_rows<4, 0>(D, mt, p, plan, stream);
}
}  // namespace kvq
