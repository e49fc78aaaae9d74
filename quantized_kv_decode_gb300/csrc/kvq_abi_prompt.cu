// Host side of the prompt and page-pool calls of include/kvq.h: argument
// validation, planning and dispatch.  Nothing here allocates memory or
// synchronizes a stream.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "kvq_host.cuh"
#include "kvq_load.cuh"
#include "kvq_pages.cuh"
#include "kvq_rope.cuh"

using namespace kvq;

namespace {

kvq_status check_rope(const kvq_rope* r) {
  if (!r || r->rotary_dim < 2 || r->rotary_dim > 2 * KVQ_ROPE_MAX_PAIRS || r->rotary_dim % 2)
    return KVQ_ERR_INVALID_ARG;
  if (r->interleaved != 0 && r->interleaved != 1) return KVQ_ERR_INVALID_ARG;
  if (r->amplitude == 0 || r->amplitude >= (1ull << 63)) return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

// [a, a + n) and [b, b + n) share a byte but are not the same array
bool partly_over(const void* a, const void* b, size_t n) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x != y && x < y + n && y < x + n;
}

AppendParams append_params(const CacheGeom& g, const kvq_cache* cache, int32_t batch,
                           int32_t num_new, const uint16_t* k_new, const uint16_t* v_new,
                           const int32_t* before, uint32_t* status) {
  AppendParams a{};
  a.geom = g;
  a.geom.block_table = cache->block_table;
  a.codes[0] = reinterpret_cast<uint8_t*>(cache->k_codes);
  a.codes[1] = reinterpret_cast<uint8_t*>(cache->v_codes);
  a.scale[0] = reinterpret_cast<__half*>(cache->k_scale);
  a.scale[1] = reinterpret_cast<__half*>(cache->v_scale);
  a.zero[0] = reinterpret_cast<__half*>(cache->k_zero);
  a.zero[1] = reinterpret_cast<__half*>(cache->v_zero);
  a.src[0] = reinterpret_cast<const __half*>(k_new);
  a.src[1] = reinterpret_cast<const __half*>(v_new);
  if (g.nf4) memcpy(a.nf4_mid, nf4_table().mid, sizeof(a.nf4_mid));
  a.seq_lens_before = before;
  a.status = status;
  a.batch = batch;
  a.num_new = num_new;
  return a;
}

CacheView view_of(const CacheGeom& g, const kvq_cache* cache) {
  CacheView v{};
  v.geom = g;
  v.geom.block_table = cache->block_table;
  v.codes[0] = reinterpret_cast<const uint8_t*>(cache->k_codes);
  v.codes[1] = reinterpret_cast<const uint8_t*>(cache->v_codes);
  v.scale[0] = reinterpret_cast<const __half*>(cache->k_scale);
  v.scale[1] = reinterpret_cast<const __half*>(cache->v_scale);
  v.zero[0] = reinterpret_cast<const __half*>(cache->k_zero);
  v.zero[1] = reinterpret_cast<const __half*>(cache->v_zero);
  v.window[0] = reinterpret_cast<const __half*>(cache->k_window);
  v.window[1] = reinterpret_cast<const __half*>(cache->v_window);
  if (g.nf4) memcpy(v.nf4_level, nf4_table().level, sizeof(v.nf4_level));
  return v;
}

// Rows of a padded batch are counted in 32 bits by the kernels' grids.
bool too_many_rows(int64_t batch, int64_t num_new, int64_t heads) {
  return batch * num_new > INT32_MAX / 2 || batch * num_new * heads > INT32_MAX / 2;
}

struct ExtendChoice {
  ExtendPlan plan;
  int32_t splits = 0;
};

// Splits spread a call with few row tiles over the device, and even out
// sequences of different lengths.  The automatic choice weighs, in positions
// of a CTA's work: equal sequences, whose CTAs run in whole waves; and (with
// several sequences) lengths spread over the range up to max_seq_len, where
// about 0.6 of the CTAs have keys and the last ones half overlap.  A CTA
// costs kFixed positions beside its own (set-up, filling the pipeline,
// writing out), the partials their bytes written and read, 6800 a ns against
// 13 ns a position with one tile of rows, 20 with two (the fp16 kernel's; the
// quantized ones' are up to a quarter more).  16 sequences of 1390 to 6527
// tokens, 5 new ones, INT4, calls in turn on one cache: 3 splits chosen, 98 us;
// 1 to 12 splits 99, 105, 98, 97, 104, 107, 109, 114, 120, 124, 128, 133.
constexpr int64_t kFixed = 384;
int32_t choose_extend_splits(int64_t units, int64_t max_len, int64_t rows, int64_t D, bool several, int requested,
                             const ExtendPlan& plan) {
  const int64_t L = std::max<int64_t>(max_len, 1);
  if (requested > 0) return choose_splits(units, max_len, requested, 0);
  const int sms = sm_count();
  if (sms <= 0 || plan.occ <= 0) return 0;
  const double slots = (double)sms * plan.occ, ns = plan.kind == 2 ? 20.0 : 13.0;
  const int64_t cap = std::max<int64_t>(1, std::min<int64_t>(ceil_div(L, 256), 64));
  int64_t best = 1;
  double best_cost = 1e300;
  for (int64_t c = 1; c <= cap; ++c) {
    const int64_t chunk = split_chunk(L, (int32_t)c), eff = ceil_div(L, chunk);
    const double waves = (double)std::max<int64_t>(units, 1) * eff / slots, each = (double)(chunk + kFixed);
    const double equal = ceil(waves) * each, spread = std::max(1.0, 0.6 * waves + 0.5) * each;
    const double join = eff > 1 ? (double)rows * D * 8.0 * eff / 6800.0 / ns : 0.0;
    const double cost = (several ? 0.5 * (equal + spread) : equal) + join;
    if (cost < best_cost * 0.999) {
      best_cost = cost;
      best = eff;
    }
  }
  return (int32_t)best;
}

kvq_status choose_extend(const kvq_cache_desc* desc, const CacheGeom& g, int32_t batch,
                         int32_t num_new, int32_t num_q_heads, int32_t max_seq_len,
                         int32_t requested, ExtendChoice* out) {
  const int G = num_q_heads / desc->num_kv_heads;
  const cudaError_t e = extend_plan(g, num_new, G, &out->plan);
  if (e != cudaSuccess) return from_cuda(e);
  const int64_t tiles = ceil_div((int64_t)num_new * G, out->plan.tile_rows);
  const int64_t units = tiles * desc->num_kv_heads * std::max(batch, 1);
  out->splits = choose_extend_splits(units, max_seq_len, (int64_t)batch * num_new * num_q_heads, desc->head_dim,
                                     batch > 1, requested, out->plan);
  if (tiles * out->splits > INT32_MAX) return KVQ_ERR_UNSUPPORTED;
  return out->splits > 0 ? KVQ_OK : KVQ_ERR_CUDA;
}

size_t extend_ws(int64_t rows, int64_t D, int64_t splits) {
  return workspace_bytes(rows, 1, D, splits);
}

kvq_status check_pool(const kvq_page_pool* p) {
  if (!p || p->num_pages <= 0 || p->page_size <= 0 || p->batch < 0 || p->max_blocks_per_seq <= 0)
    return KVQ_ERR_INVALID_ARG;
  if ((int64_t)p->page_size * p->max_blocks_per_seq > INT32_MAX) return KVQ_ERR_INVALID_ARG;
  if (p->num_pages > INT32_MAX / 4) return KVQ_ERR_UNSUPPORTED;
  if (p->batch > KVQ_MAX_POOL_BATCH) return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

kvq_status check_pool_arrays(const kvq_page_pool* p) {
  if (!p->ref_count || (p->batch && !p->block_table)) return KVQ_ERR_INVALID_ARG;
  if (!aligned(p->ref_count) || !aligned(p->block_table)) return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

}  // namespace

extern "C" {

kvq_status kvq_rope_init(const kvq_rope_desc* d, kvq_rope* rope) {
  if (!d || !rope) return KVQ_ERR_INVALID_ARG;
  if (d->rotary_dim < 2 || d->rotary_dim > 2 * KVQ_ROPE_MAX_PAIRS || d->rotary_dim % 2)
    return KVQ_ERR_INVALID_ARG;
  if (d->interleaved != 0 && d->interleaved != 1) return KVQ_ERR_INVALID_ARG;
  if (d->scaling < KVQ_ROPE_NONE || d->scaling > KVQ_ROPE_YARN) return KVQ_ERR_INVALID_ARG;
  if (!(d->base > 1.0) || !isfinite(d->base)) return KVQ_ERR_INVALID_ARG;
  if (!(d->factor >= 1.0) || !isfinite(d->factor)) return KVQ_ERR_INVALID_ARG;
  if (d->scaling == KVQ_ROPE_NONE && d->factor != 1.0) return KVQ_ERR_INVALID_ARG;
  if (!(d->amplitude >= 0.0 && d->amplitude < 4.0)) return KVQ_ERR_INVALID_ARG;
  const bool ranged = d->scaling == KVQ_ROPE_BANDS || d->scaling == KVQ_ROPE_YARN;
  double low = d->low_turns, high = d->high_turns;
  if (!(low >= 0.0) || !(high >= 0.0) || !isfinite(low) || !isfinite(high)) return KVQ_ERR_INVALID_ARG;
  if (low == 0.0) low = 1.0;
  if (high == 0.0) high = d->scaling == KVQ_ROPE_YARN ? 32.0 : 4.0;
  if (ranged && (d->original_context <= 0 || low >= high)) return KVQ_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  const int rd = d->rotary_dim;
  if (d->scaling == KVQ_ROPE_NTK && rd == 2) return KVQ_ERR_INVALID_ARG;  // one pair: no exponent
  double base = d->base, lo = 0.0, span = 1.0;
  if (d->scaling == KVQ_ROPE_NTK) base *= pow(d->factor, (double)rd / (rd - 2));
  if (!isfinite(base)) return KVQ_ERR_INVALID_ARG;
  if (d->scaling == KVQ_ROPE_YARN) {
    // the pair that turns n times in the original context
    auto pair_at = [&](double n) {
      return rd * log(d->original_context / (n * two_pi)) / (2.0 * log(base));
    };
    lo = std::max(floor(pair_at(high)), 0.0);
    const double hi = std::min(ceil(pair_at(low)), rd - 1.0);
    span = std::max(hi - lo, 0.001);
  }
  memset(rope, 0, sizeof(*rope));
  rope->rotary_dim = rd;
  rope->interleaved = d->interleaved;
  double amp = d->amplitude;
  if (amp == 0.0)
    amp = d->scaling == KVQ_ROPE_YARN && d->factor > 1.0 ? 0.1 * log(d->factor) + 1.0 : 1.0;
  if (!(amp < 4.0)) return KVQ_ERR_INVALID_ARG;
  rope->amplitude = (uint64_t)ldexp(amp, 61);
  if (rope->amplitude == 0) return KVQ_ERR_INVALID_ARG;
  for (int i = 0; i < rd / 2; ++i) {
    double w = pow(base, -2.0 * i / rd);
    if (d->scaling == KVQ_ROPE_LINEAR) {
      w /= d->factor;
    } else if (d->scaling == KVQ_ROPE_BANDS) {
      const double n = d->original_context * w / two_pi;
      const double keep = std::min(1.0, std::max(0.0, (n - low) / (high - low)));
      w = w * (keep + (1.0 - keep) / d->factor);
    } else if (d->scaling == KVQ_ROPE_YARN) {
      const double slow = std::min(1.0, std::max(0.0, (i - lo) / span));
      w = w * (1.0 - slow) + w / d->factor * slow;
    }
    rope->turns[i] = (uint64_t)(ldexp(w / two_pi, 64) + 0.5);  // w <= 1: less than a turn
  }
  return KVQ_OK;
}

kvq_status kvq_rope_apply(const kvq_rope* rope, int32_t head_dim, int32_t batch, int32_t num_new,
                          int32_t num_q_heads, const uint16_t* q, uint16_t* q_out,
                          int32_t num_k_heads, const uint16_t* k, uint16_t* k_out,
                          const int32_t* positions, const int32_t* seq_lens_before,
                          const int32_t* new_lens, uint32_t* dev_status, void* stream) {
  kvq_status st = check_rope(rope);
  if (st != KVQ_OK) return st;
  if (head_dim <= 0 || head_dim % 8 || rope->rotary_dim > head_dim) return KVQ_ERR_INVALID_ARG;
  if (head_dim > 2 * KVQ_ROPE_MAX_PAIRS) return KVQ_ERR_UNSUPPORTED;
  if (batch < 0 || num_new < 0 || num_q_heads < 0 || num_k_heads < 0) return KVQ_ERR_INVALID_ARG;
  if (batch == 0 || num_new == 0 || (num_q_heads == 0 && num_k_heads == 0)) return KVQ_OK;
  if (too_many_rows(batch, num_new, std::max(num_q_heads, num_k_heads))) return KVQ_ERR_UNSUPPORTED;
  if (!positions && !seq_lens_before) return KVQ_ERR_INVALID_ARG;
  if (num_q_heads && (!q || !q_out || !aligned(q) || !aligned(q_out))) return KVQ_ERR_INVALID_ARG;
  if (num_k_heads && (!k || !k_out || !aligned(k) || !aligned(k_out))) return KVQ_ERR_INVALID_ARG;
  if (!aligned(positions) || !aligned(seq_lens_before) || !aligned(new_lens)) return KVQ_ERR_INVALID_ARG;
  const size_t row = (size_t)batch * num_new * head_dim * 2;
  if (num_q_heads && partly_over(q, q_out, row * num_q_heads)) return KVQ_ERR_INVALID_ARG;
  if (num_k_heads && partly_over(k, k_out, row * num_k_heads)) return KVQ_ERR_INVALID_ARG;
  RopeParams p{};
  p.rope = *rope;
  p.q = reinterpret_cast<const __half*>(q);
  p.q_out = reinterpret_cast<__half*>(q_out);
  p.k = reinterpret_cast<const __half*>(k);
  p.k_out = reinterpret_cast<__half*>(k_out);
  p.positions = positions;
  p.seq_lens_before = seq_lens_before;
  p.new_lens = new_lens;
  p.status = dev_status;
  p.D = head_dim;
  p.batch = batch;
  p.num_new = num_new;
  p.Hq = num_q_heads;
  p.Hk = num_k_heads;
  return from_cuda(launch_rope(p, reinterpret_cast<cudaStream_t>(stream)));
}

kvq_status kvq_rope_append(const kvq_cache_desc* desc, const kvq_cache* cache, const kvq_rope* rope,
                           int32_t batch, int32_t num_new, const uint16_t* k_new,
                           const uint16_t* v_new, int32_t num_q_heads, const uint16_t* q,
                           uint16_t* q_out, const int32_t* seq_lens_before,
                           const int32_t* new_lens, uint32_t* dev_status, void* stream) {
  CacheGeom g;
  kvq_status st = check_desc(desc, &g);
  if (st != KVQ_OK) return st;
  if ((st = check_cache(desc, cache)) != KVQ_OK) return st;
  if ((st = check_rope(rope)) != KVQ_OK) return st;
  if (rope->rotary_dim > desc->head_dim) return KVQ_ERR_INVALID_ARG;
  if (batch < 0 || num_new < 0 || num_q_heads < 0) return KVQ_ERR_INVALID_ARG;
  if (desc->k_per_channel) return KVQ_ERR_UNSUPPORTED;
  if (batch == 0 || num_new == 0) return KVQ_OK;
  if (too_many_rows(batch, num_new, std::max(num_q_heads, 2 * desc->num_kv_heads)))
    return KVQ_ERR_UNSUPPORTED;
  if (!k_new || !v_new || !seq_lens_before) return KVQ_ERR_INVALID_ARG;
  if (!aligned(k_new) || !aligned(v_new) || !aligned(seq_lens_before) || !aligned(new_lens))
    return KVQ_ERR_INVALID_ARG;
  if (num_q_heads) {
    if (!q || !q_out || !aligned(q) || !aligned(q_out)) return KVQ_ERR_INVALID_ARG;
    if (partly_over(q, q_out, (size_t)batch * num_new * num_q_heads * desc->head_dim * 2))
      return KVQ_ERR_INVALID_ARG;
  }
  RopeAppendParams p{};
  p.a = append_params(g, cache, batch, num_new, k_new, v_new, seq_lens_before, dev_status);
  dbg_fill(p.a.geom, desc, cache, batch, 0, num_new, nullptr, k_new, v_new, seq_lens_before,
           nullptr, nullptr, 0, dev_status);
  p.r.rope = *rope;
  p.r.q = reinterpret_cast<const __half*>(q);
  p.r.q_out = reinterpret_cast<__half*>(q_out);
  p.r.seq_lens_before = seq_lens_before;
  p.r.new_lens = new_lens;
  p.r.status = dev_status;
  p.r.D = desc->head_dim;
  p.r.batch = batch;
  p.r.num_new = num_new;
  p.r.Hq = num_q_heads;
  return from_cuda(launch_rope_append(p, reinterpret_cast<cudaStream_t>(stream)));
}

kvq_status kvq_cache_read(const kvq_cache_desc* desc, const kvq_cache* cache, int32_t batch,
                          int32_t num_rows, const int32_t* seq_lens, const int32_t* start,
                          uint16_t* k_out, uint16_t* v_out, uint32_t* dev_status, void* stream) {
  CacheGeom g;
  kvq_status st = check_desc(desc, &g);
  if (st != KVQ_OK) return st;
  if ((st = check_cache(desc, cache)) != KVQ_OK) return st;
  if (batch < 0 || num_rows < 0) return KVQ_ERR_INVALID_ARG;
  if (batch == 0 || num_rows == 0 || (!k_out && !v_out)) return KVQ_OK;
  if (too_many_rows(batch, num_rows, desc->num_kv_heads))
    return KVQ_ERR_UNSUPPORTED;
  if (!seq_lens || !start) return KVQ_ERR_INVALID_ARG;
  if (!aligned(seq_lens) || !aligned(start) || !aligned(k_out) || !aligned(v_out))
    return KVQ_ERR_INVALID_ARG;
  ReadParams p{};
  p.v = view_of(g, cache);
  dbg_fill(p.v.geom, desc, cache, batch, 0, num_rows, nullptr, k_out, v_out, seq_lens, nullptr,
           nullptr, 0, dev_status);
  p.seq_lens = seq_lens;
  p.start = start;
  p.out[0] = reinterpret_cast<__half*>(k_out);
  p.out[1] = reinterpret_cast<__half*>(v_out);
  p.status = dev_status;
  p.batch = batch;
  p.num_rows = num_rows;
  return from_cuda(launch_read(p, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t kvq_extend_num_splits(const kvq_cache_desc* desc, int32_t batch, int32_t num_new,
                              int32_t num_q_heads, int32_t max_seq_len, int32_t num_splits) {
  CacheGeom g;
  if (check_desc(desc, &g) != KVQ_OK || batch < 0 || num_new < 0 || num_q_heads <= 0 ||
      max_seq_len < 0 || num_splits < 0 || num_q_heads % desc->num_kv_heads ||
      too_many_rows(batch, num_new, num_q_heads))
    return 0;
  ExtendChoice c;
  if (choose_extend(desc, g, batch, num_new, num_q_heads, max_seq_len, num_splits, &c) != KVQ_OK)
    return 0;
  return c.splits;
}

size_t kvq_extend_workspace_size(const kvq_cache_desc* desc, int32_t batch, int32_t num_new,
                                 int32_t num_q_heads, int32_t max_seq_len, int32_t num_splits) {
  const int32_t s = kvq_extend_num_splits(desc, batch, num_new, num_q_heads, max_seq_len, num_splits);
  if (s <= 1) return 0;
  return extend_ws((int64_t)batch * num_new * num_q_heads, desc->head_dim, s);
}

kvq_status kvq_extend_attn(const kvq_cache_desc* desc, const kvq_cache* cache, int32_t batch,
                           int32_t num_new, int32_t num_q_heads, const uint16_t* q,
                           const int32_t* seq_lens_before, const int32_t* new_lens,
                           int32_t max_seq_len, int32_t num_splits, float softmax_scale,
                           uint16_t* out, void* workspace, size_t workspace_size,
                           uint32_t* dev_status, void* stream) {
  CacheGeom g;
  kvq_status st = check_desc(desc, &g);
  if (st != KVQ_OK) return st;
  if ((st = check_cache(desc, cache)) != KVQ_OK) return st;
  if (batch < 0 || num_new < 0 || num_q_heads <= 0 || max_seq_len < 0 || num_splits < 0)
    return KVQ_ERR_INVALID_ARG;
  if (num_q_heads % desc->num_kv_heads) return KVQ_ERR_INVALID_ARG;
  if (!(softmax_scale >= 0.f) || isinf(softmax_scale)) return KVQ_ERR_INVALID_ARG;
  if (batch == 0 || num_new == 0) return KVQ_OK;
  if (batch > KVQ_MAX_BATCH || desc->num_kv_heads > 65535 ||
      too_many_rows(batch, num_new, num_q_heads))
    return KVQ_ERR_UNSUPPORTED;
  if (!q || !out || !seq_lens_before) return KVQ_ERR_INVALID_ARG;
  if (!aligned(q) || !aligned(out) || !aligned(seq_lens_before) || !aligned(new_lens))
    return KVQ_ERR_INVALID_ARG;
  const size_t bytes = (size_t)batch * num_new * num_q_heads * desc->head_dim * 2;
  if (q == out || partly_over(q, out, bytes)) return KVQ_ERR_INVALID_ARG;

  ExtendChoice choice;
  if ((st = choose_extend(desc, g, batch, num_new, num_q_heads, max_seq_len, num_splits, &choice)) != KVQ_OK)
    return st;
  const int64_t rows = (int64_t)batch * num_new * num_q_heads;
  const size_t need = extend_ws(rows, desc->head_dim, choice.splits);
  if (need && (!workspace || workspace_size < need || !aligned(workspace))) return KVQ_ERR_WORKSPACE;

  ExtendParams p{};
  p.v = view_of(g, cache);
  dbg_fill(p.v.geom, desc, cache, batch, num_q_heads * num_new, 0, q, nullptr, nullptr,
           seq_lens_before, out, need ? workspace : nullptr, need ? workspace_size : 0, dev_status);
  p.q = reinterpret_cast<const __half*>(q);
  p.out = reinterpret_cast<__half*>(out);
  p.lens_before = seq_lens_before;
  p.new_lens = new_lens;
  if (need) workspace_carve(workspace, rows, 1, desc->head_dim, choice.splits, &p.ws_o, &p.ws_ml);
  p.status = dev_status;
  p.batch = batch;
  p.num_new = num_new;
  p.Hq = num_q_heads;
  p.G = num_q_heads / desc->num_kv_heads;
  p.splits = choice.splits;
  p.chunk = split_chunk(max_seq_len, choice.splits);
  p.len_limit = (int32_t)std::min<int64_t>(cache_capacity(g), max_seq_len);
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)desc->head_dim);
  p.scale_log2 = scale * 1.4426950408889634f;
  return from_cuda(launch_extend(p, choice.plan, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kvq_pages_workspace_size(const kvq_page_pool* pool) {
  if (check_pool(pool) != KVQ_OK) return 0;
  return (size_t)pool->num_pages * 8;
}

kvq_status kvq_pages_reorder(const kvq_page_pool* pool, const int32_t* parent,
                             const int32_t* keep_lens, uint32_t* dev_status, void* stream) {
  kvq_status st = check_pool(pool);
  if (st != KVQ_OK) return st;
  if (pool->batch == 0) return KVQ_OK;
  if ((st = check_pool_arrays(pool)) != KVQ_OK) return st;
  if (!parent || !aligned(parent) || !aligned(keep_lens)) return KVQ_ERR_INVALID_ARG;
  PoolParams p{};
  p.pool = *pool;
  p.parent = parent;
  p.keep_lens = keep_lens;
  p.status = dev_status;
  return from_cuda(launch_pages_reorder(p, reinterpret_cast<cudaStream_t>(stream)));
}

kvq_status kvq_pages_reserve(const kvq_page_pool* pool, const int32_t* seq_lens_before,
                             const int32_t* new_lens, int32_t num_new, int32_t* copy_src,
                             int32_t* copy_dst, int32_t* granted, void* workspace,
                             size_t workspace_bytes, uint32_t* dev_status, void* stream) {
  kvq_status st = check_pool(pool);
  if (st != KVQ_OK) return st;
  if (num_new < 0) return KVQ_ERR_INVALID_ARG;
  // the blocks that all sequences touch are counted in 32 bits
  const int64_t blocks = std::min<int64_t>(pool->max_blocks_per_seq, (int64_t)num_new / pool->page_size + 2);
  if (blocks * pool->batch > INT32_MAX) return KVQ_ERR_UNSUPPORTED;
  if (pool->batch == 0) return KVQ_OK;
  if ((st = check_pool_arrays(pool)) != KVQ_OK) return st;
  if (!seq_lens_before || !copy_src || !copy_dst) return KVQ_ERR_INVALID_ARG;
  if (!aligned(seq_lens_before) || !aligned(new_lens) || !aligned(copy_src) || !aligned(copy_dst) ||
      !aligned(granted))
    return KVQ_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace) || workspace_bytes < kvq_pages_workspace_size(pool))
    return KVQ_ERR_WORKSPACE;
  PoolParams p{};
  p.pool = *pool;
  p.seq_lens_before = seq_lens_before;
  p.new_lens = new_lens;
  p.num_new = num_new;
  p.copy_src = copy_src;
  p.copy_dst = copy_dst;
  p.granted = granted;
  p.ws = reinterpret_cast<int32_t*>(workspace);
  p.status = dev_status;
  return from_cuda(launch_pages_reserve(p, reinterpret_cast<cudaStream_t>(stream)));
}

kvq_status kvq_pages_compact(const kvq_page_pool* pool, int32_t* move_src, int32_t* move_dst,
                             int32_t* num_live, void* workspace, size_t workspace_bytes,
                             uint32_t* dev_status, void* stream) {
  kvq_status st = check_pool(pool);
  if (st != KVQ_OK) return st;
  if ((st = check_pool_arrays(pool)) != KVQ_OK) return st;
  if (!num_live || (pool->num_pages > 1 && (!move_src || !move_dst))) return KVQ_ERR_INVALID_ARG;
  if (!aligned(move_src) || !aligned(move_dst) || !aligned(num_live)) return KVQ_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace) || workspace_bytes < kvq_pages_workspace_size(pool))
    return KVQ_ERR_WORKSPACE;
  PoolParams p{};
  p.pool = *pool;
  p.copy_src = move_src;
  p.copy_dst = move_dst;
  p.num_live = num_live;
  p.ws = reinterpret_cast<int32_t*>(workspace);
  p.status = dev_status;
  return from_cuda(launch_pages_compact(p, reinterpret_cast<cudaStream_t>(stream)));
}

kvq_status kvq_pages_copy(const kvq_cache_desc* desc, const kvq_cache* caches, int32_t num_layers,
                          const int32_t* copy_src, const int32_t* copy_dst, int32_t num_pairs,
                          uint32_t* dev_status, void* stream) {
  CacheGeom g;
  kvq_status st = check_desc(desc, &g);
  if (st != KVQ_OK) return st;
  if (g.layout != KVQ_PAGED || num_layers < 0 || num_pairs < 0) return KVQ_ERR_INVALID_ARG;
  if (num_layers == 0 || num_pairs == 0) return KVQ_OK;
  if (!caches || !copy_src || !copy_dst || !aligned(copy_src) || !aligned(copy_dst))
    return KVQ_ERR_INVALID_ARG;
  for (int32_t l = 0; l < num_layers; ++l)
    if ((st = check_cache(desc, caches + l)) != KVQ_OK) return st;
  const int64_t rows = (int64_t)g.Hkv * g.slots;
  const int64_t code = rows * g.row_bytes, head = rows * g.ngroups * 2;
  const int64_t khead = g.kch ? (int64_t)g.Hkv * (g.slots / g.g) * g.D * 2 : head;
  const bool zeros = g.bits != 16 && !g.sym && !g.nf4;
  const int64_t bytes[6] = {code, code, khead, zeros ? khead : 0, head, zeros ? head : 0};
  if (std::max(code, khead) > UINT32_MAX) return KVQ_ERR_UNSUPPORTED;
  PageCopyParams p{};
  for (int a = 0; a < 6; ++a) p.bytes[a] = (uint32_t)bytes[a];
  p.src = copy_src;
  p.dst = copy_dst;
  p.status = dev_status;
  p.num_pages = g.num_pages;
  p.num_pairs = num_pairs;
  for (int32_t l0 = 0; l0 < num_layers; l0 += kCopyLayers) {
    p.layers = std::min(kCopyLayers, num_layers - l0);
    p.report = l0 == 0 && dev_status != nullptr;
    for (int32_t l = 0; l < p.layers; ++l) {
      const kvq_cache& c = caches[l0 + l];
      void* const arrays[6] = {c.k_codes, c.v_codes, c.k_scale, c.k_zero, c.v_scale, c.v_zero};
      for (int a = 0; a < 6; ++a) p.base[l][a] = reinterpret_cast<uint8_t*>(arrays[a]);
    }
    const cudaError_t e = launch_pages_copy(p, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return from_cuda(e);
  }
  return KVQ_OK;
}

}  // extern "C"
