// The page pool: reference counts and block table (include/kvq.h).
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

struct PoolParams {
  kvq_page_pool pool;
  const int32_t* parent;
  const int32_t* keep_lens;
  const int32_t* seq_lens_before;
  const int32_t* new_lens;
  int32_t num_new;
  int32_t* copy_src;
  int32_t* copy_dst;
  int32_t* granted;
  int32_t* num_live;
  int32_t* ws;  // 2 * num_pages int32
  uint32_t* status;
};

// One launch's worth of layers of a page copy: per layer the arrays of a
// cache that hold pages, and each array's bytes per page (multiples of 16).
constexpr int kCopyLayers = 64;
struct PageCopyParams {
  uint8_t* base[kCopyLayers][6];
  uint32_t bytes[6];
  const int32_t* src;
  const int32_t* dst;
  uint32_t* status;
  int32_t num_pages, num_pairs, layers, report;
};

cudaError_t launch_pages_reorder(const PoolParams& p, cudaStream_t stream);
cudaError_t launch_pages_reserve(const PoolParams& p, cudaStream_t stream);
cudaError_t launch_pages_compact(const PoolParams& p, cudaStream_t stream);
cudaError_t launch_pages_copy(const PageCopyParams& p, cudaStream_t stream);

}  // namespace kvq
