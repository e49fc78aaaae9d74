// Host helpers shared by the files that implement the prompt, page-pool and
// shared-prefix calls (kvq_abi_prompt.cu, kvq_abi_prefix.cu).
#pragma once

#include "kvq_host.cuh"
#include "kvq_load.cuh"

namespace kvq {

// [a, a + n) and [b, b + n) share a byte but are not the same array
bool partly_over(const void* a, const void* b, size_t n);
// Rows of a padded batch are counted in 32 bits by the kernels' grids.
bool too_many_rows(int64_t batch, int64_t num_new, int64_t heads);
CacheView view_of(const CacheGeom& g, const kvq_cache* cache);
// Splits of extend attention over max_len positions: `units` CTAs a split,
// `rows` rows of partials.
int32_t choose_extend_splits(int64_t units, int64_t max_len, int64_t rows, int64_t D, bool several, int requested,
                             const ExtendPlan& plan);
kvq_status check_pool(const kvq_page_pool* p);
kvq_status check_pool_arrays(const kvq_page_pool* p);

}  // namespace kvq
