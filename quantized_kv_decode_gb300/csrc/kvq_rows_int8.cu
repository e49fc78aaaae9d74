// Attention of few rows over shared prefixes, codes in registers: int8 caches.
#include "kvq_rows.cuh"

namespace kvq {
cudaError_t run_rows_int8(int D, int mt, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream) {
  return rows::run_rows<8, 0>(D, mt, p, plan, stream);
}
}  // namespace kvq
