// Host helpers shared by the files that implement the C ABI (kvq_abi.cu,
// kvq_abi_prompt.cu).  Not part of the public ABI; the library is built with
// hidden visibility.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

constexpr size_t kAlign = 16;

inline bool aligned(const void* p) { return ((uintptr_t)p % kAlign) == 0; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Validates a cache descriptor; fills `g` (may be null) on success.
kvq_status check_desc(const kvq_cache_desc* d, CacheGeom* g);
kvq_status check_cache(const kvq_cache_desc* d, const kvq_cache* c);
// A failed CUDA call maps to KVQ_ERR_CUDA.
kvq_status from_cuda(cudaError_t e);
int sm_count();
// Positions per split, and the split count (requested > 0: as asked, up to
// one aligned tile per split; 0: chosen from the device's CTA slots).
int32_t split_chunk(int64_t max_len, int32_t splits);
int32_t choose_splits(int64_t units, int64_t max_len, int32_t requested, int ctas_per_sm);

struct Nf4Table {
  float level[16];
  float mid[16];
  bool symmetric;  // level[15 - i] == -level[i]: the tensor-core kernel's sign-magnitude lookup
};
const Nf4Table& nf4_table();

// Debug builds: the extent of every caller array of a call (the sizes
// kvq.h states for debug builds); nothing in a release build.
void dbg_fill(CacheGeom& g, const kvq_cache_desc* desc, const kvq_cache* cache, int32_t batch,
              int32_t num_q_heads, int32_t num_new, const void* q, const void* k_new,
              const void* v_new, const void* lens, const void* out, const void* ws,
              size_t ws_bytes, uint32_t* status);

// Debug builds: sets one array's extent; nothing in a release build.
void dbg_extent(CacheGeom& g, int array, const void* base, size_t bytes);

// The tails of sequences with a shared prefix, one new token each: whether a
// tensor-core decode kernel takes them, and its launch, which leaves partials
// ([batch][num_q_heads][splits]) for the join or (t.one) writes `out`, joined.
struct TailDecode {
  bool takes = false;
  bool one = false;  // the tail kernel: joined with the prefixes and written out
  int wpu = 0;       // its warps a (sequence, KV head)
  int gp = 1, occ = 0;
  int32_t splits = 0;
};
kvq_status tail_decode_plan(const kvq_cache_desc* desc, const CacheGeom& geom, int32_t batch, int32_t num_q_heads,
                            int32_t max_len, int32_t requested, TailDecode* t);
cudaError_t tail_decode(const kvq_cache_desc* desc, const kvq_cache* cache, const CacheGeom& geom, int32_t batch,
                        int32_t num_q_heads, const uint16_t* q, const int32_t* before, const int32_t* new_lens,
                        int32_t max_len, const TailDecode& t, float scale_log2, float* ws_o, float* ws_ml,
                        const void* ws, size_t ws_bytes, uint32_t* status, cudaStream_t stream,
                        const PrefixJoin& join, uint16_t* out);

}  // namespace kvq
