// Host side of the shared-prefix calls of include/kvq.h: argument validation,
// planning and dispatch.  Nothing here allocates memory or synchronizes a
// stream.
#include <math.h>

#include <algorithm>

#include "kvq_prompt_host.cuh"

using namespace kvq;

namespace {

// Arrays of a call: bytes, and whether the call writes it.  One that is written
// shares no byte with another.
struct Span {
  const void* at;
  size_t bytes;
  bool out;
};
template <int N>
bool apart(const Span (&spans)[N]) {
  for (int i = 0; i < N; ++i)
    for (int j = 0; j < i; ++j) {
      const Span &a = spans[i], &b = spans[j];
      const uintptr_t x = (uintptr_t)a.at, y = (uintptr_t)b.at;
      if ((a.out || b.out) && a.bytes && b.bytes && x && y && x < y + b.bytes && y < x + a.bytes) return false;
    }
  return true;
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// One pass's partials: sums of rows * splits, then (maximum, sum) pairs.
size_t partial_bytes(int64_t rows, int64_t D, int64_t splits) {
  return up256((size_t)(rows * splits * D) * sizeof(float)) + up256((size_t)(rows * splits) * 2 * sizeof(float));
}
void carve_partials(void* at, int64_t rows, int64_t D, int64_t splits, float** o, float** ml) {
  *o = reinterpret_cast<float*>(at);
  *ml = reinterpret_cast<float*>(reinterpret_cast<char*>(at) + up256((size_t)(rows * splits * D) * sizeof(float)));
}

// How a call runs: the prefix pass, then the tails by a decode kernel or by
// extend attention, then the join.
struct PrefixChoice {
  CacheGeom pg, tg;
  int32_t max_prefix = 0, max_len = 0;  // the call's bounds, at most what the caches hold
  bool prefixes = false;  // there is a prefix pass
  ExtendPlan pre, tail;
  TailDecode decode;
  int32_t prefix_splits = 0, tail_splits = 0;
  size_t prefix_bytes = 0, tail_bytes = 0, word_bytes = 0;  // (a word: start_beside)
  size_t workspace() const { return prefix_bytes + tail_bytes + word_bytes; }
};

// Splits of the prefix pass, and what the call then costs in ns.  A block takes
// kFixed keys' time beside its own; blocks run in whole turns over the device;
// the partials are written and read at 6800 bytes a ns.  The tail kernel
// (tail_warps of them, eight an SM, with tail_keys each) runs beside the pass
// where that leaves room, and behind it where not.  The constants fit head_dim 128
// best.  Of 384 cases (8 to 256 rows over one prefix of 512 to 16384 tokens, tails of
// 64, 8 and 32 KV heads, head_dim 64 and 128; INT4, INT8, NF4, fp16) the choice is
// within 5 % of the best kernel and splits in 78 %, within 15 % in 96 %, and 29 % off
// at worst (NF4 at head_dim 64).  Members are taken to be shared out evenly over the
// prefixes that there is room for: the host does not know better.
int32_t prefix_splits(const ExtendPlan& plan, int64_t units, int64_t max_len, int64_t rows, int64_t D, int requested,
                      int64_t tail_warps, int64_t tail_keys, double* cost) {
  static const double kNs[5] = {40, 16, 20, 25, 30};  // a key, by plan.kind
  static const double kFixed[5] = {200, 550, 650, 128, 180};
  const int64_t L = std::max<int64_t>(max_len, 1);
  const int sms = sm_count(), occ = std::max(plan.occ, 1);
  const int64_t slots = (int64_t)std::max(sms, 1) * occ, cap = std::min<int64_t>(ceil_div(L, 128), 64);
  if (requested > 0) {
    requested = choose_splits(units, L, requested, 0);
  } else if (sms <= 0) {
    return 0;
  }
  // an SM holds eight tail warps
  const double turns = ceil((double)tail_warps / (8.0 * std::max(sms, 1)));
  const double tail = tail_warps ? turns * (2000.0 + 30.0 * tail_keys) : 0.0;
  int32_t best = 0;
  *cost = 1e300;
  for (int64_t s = requested > 0 ? requested : 1; s <= (requested > 0 ? requested : cap);
       s += s < 24 ? 1 : 4) {
    const int64_t chunk = split_chunk(L, (int32_t)s), eff = ceil_div(L, chunk), n = std::max<int64_t>(units, 1) * eff;
    const double pass = ceil((double)n / slots) * (chunk + kFixed[plan.kind]) * kNs[plan.kind];
    // (SMs without a block of the pass: on the others the two would share it)
    const double beside = n >= sms || tail_warps == 0 ? 0.0 : std::min(1.0, (sms - n) * 8.0 / tail_warps);
    const double t = std::max(pass, tail) + (1.0 - beside) * std::min(pass, tail) + rows * D * 8.0 * eff / 6800.0;
    if (t < *cost * 0.999) {
      *cost = t;
      best = (int32_t)eff;
    }
  }
  return best;
}

// The checks of a call's numbers, which need no device.
kvq_status check_sizes(const kvq_cache_desc* pd, const kvq_cache_desc* d, int32_t N, int32_t B, int32_t T, int32_t Hq,
                       int32_t max_prefix, int32_t max_len, int32_t want_prefix, int32_t want_tail, PrefixChoice* c) {
  kvq_status st = check_desc(d, &c->tg);
  if (st != KVQ_OK) return st;
  if (N < 0 || B < 0 || T < 0 || Hq <= 0 || max_prefix < 0 || max_len < 0 || want_prefix < 0 || want_tail < 0)
    return KVQ_ERR_INVALID_ARG;
  if (Hq % d->num_kv_heads) return KVQ_ERR_INVALID_ARG;
  if (N > 0) {
    if ((st = check_desc(pd, &c->pg)) != KVQ_OK) return st;
    if (pd->num_kv_heads != d->num_kv_heads || pd->head_dim != d->head_dim) return KVQ_ERR_INVALID_ARG;
  }
  if (N > KVQ_MAX_PREFIXES || B > KVQ_MAX_BATCH || d->num_kv_heads > 65535 || too_many_rows(B, T, Hq))
    return KVQ_ERR_UNSUPPORTED;
  c->max_len = (int32_t)std::min<int64_t>(cache_capacity(c->tg), max_len);
  if (N > 0) c->max_prefix = (int32_t)std::min<int64_t>(cache_capacity(c->pg), max_prefix);
  return KVQ_OK;
}

// Kernels, splits and workspace of a call whose numbers are right.
kvq_status choose(const kvq_cache_desc* d, int32_t N, int32_t B, int32_t T, int32_t Hq, int32_t want_prefix,
                  int32_t want_tail, PrefixChoice* c) {
  kvq_status st = KVQ_OK;
  const int32_t max_prefix = c->max_prefix, max_len = c->max_len;
  if (B == 0 || T == 0) return KVQ_OK;
  const int G = Hq / d->num_kv_heads;
  const int64_t D = d->head_dim, rows = (int64_t)B * T * Hq, each = (int64_t)T * G;
  if (T == 1 && (st = tail_decode_plan(d, c->tg, B, Hq, max_len, want_tail, &c->decode)) != KVQ_OK) return st;
  c->tail_splits = c->decode.splits;
  if (!c->decode.takes) {
    const cudaError_t e = extend_plan(c->tg, T, G, &c->tail);
    if (e != cudaSuccess) return from_cuda(e);
    const int64_t tiles = ceil_div(each, c->tail.tile_rows);
    c->tail_splits =
        choose_extend_splits(tiles * d->num_kv_heads * B, max_len, rows, D, B > 1, want_tail, c->tail);
    if (tiles * c->tail_splits > INT32_MAX) return KVQ_ERR_UNSUPPORTED;
  }
  if (c->tail_splits <= 0) return KVQ_ERR_CUDA;
  c->tail_bytes = c->decode.one ? 0 : partial_bytes(rows, D, c->tail_splits);
  c->prefixes = max_prefix > 0;
  if (c->prefixes) {
    const int32_t used = std::min(N, B);
    const int64_t per_prefix = ceil_div(B * each, used);
    double best = 1e300;
    for (int few = 0; few <= extend_prefix_few(c->pg, per_prefix); ++few) {
      ExtendPlan plan;
      const cudaError_t e = extend_prefix_plan(c->pg, per_prefix, few, &plan);
      if (e != cudaSuccess) return from_cuda(e);
      // (members are taken to be shared out evenly; the grid has room for any way)
      const int64_t units = used * ceil_div(per_prefix, plan.tile_rows) * d->num_kv_heads;
      const int64_t tail_warps = c->decode.one ? (int64_t)B * d->num_kv_heads * c->decode.wpu : 0;
      double cost = 0;
      const int32_t splits = prefix_splits(plan, units, max_prefix, rows, D, want_prefix, tail_warps,
                                           c->decode.one ? max_len / c->decode.wpu : 0, &cost);
      if (splits > 0 && cost < best) {
        best = cost;
        c->pre = plan;
        c->prefix_splits = splits;
      }
    }
    if (c->prefix_splits <= 0) return KVQ_ERR_CUDA;
    if (prefix_tiles_bound(B, N, each, c->pre.tile_rows) * c->prefix_splits > INT32_MAX) return KVQ_ERR_UNSUPPORTED;
    c->prefix_bytes = partial_bytes(rows, D, c->prefix_splits);
    // tails that start beside the pass: all but those of the decode kernels with splits
    if (c->decode.one || !c->decode.takes) c->word_bytes = up256(sizeof(unsigned long long));
  }
  return KVQ_OK;
}

}  // namespace

extern "C" {

size_t kvq_prefix_plan_size(int32_t batch, int32_t num_prefixes) {
  if (batch < 0 || num_prefixes < 0 || batch > KVQ_MAX_BATCH || num_prefixes > KVQ_MAX_PREFIXES) return 0;
  return plan_words(batch, num_prefixes) * sizeof(int32_t);
}

kvq_status kvq_prefix_plan(int32_t batch, int32_t num_prefixes, const int32_t* prefix_of, const int32_t* prefix_lens,
                           void* plan, size_t plan_bytes, uint32_t* dev_status, void* stream) {
  if (batch < 0 || num_prefixes < 0) return KVQ_ERR_INVALID_ARG;
  if (batch > KVQ_MAX_BATCH || num_prefixes > KVQ_MAX_PREFIXES) return KVQ_ERR_UNSUPPORTED;
  if ((batch && !prefix_of) || (num_prefixes && !prefix_lens) || !aligned(prefix_of) || !aligned(prefix_lens))
    return KVQ_ERR_INVALID_ARG;
  if (!plan || !aligned(plan) || plan_bytes < kvq_prefix_plan_size(batch, num_prefixes)) return KVQ_ERR_WORKSPACE;
  const Span spans[] = {{plan, kvq_prefix_plan_size(batch, num_prefixes), true},
                        {prefix_of, (size_t)batch * 4, false},
                        {prefix_lens, (size_t)num_prefixes * 4, false}};
  if (!apart(spans)) return KVQ_ERR_INVALID_ARG;
  PrefixPlanParams p{};
  p.of = prefix_of;
  p.len = prefix_lens;
  p.plan = reinterpret_cast<int32_t*>(plan);
  p.status = dev_status;
  p.B = batch;
  p.N = num_prefixes;
  return from_cuda(launch_prefix_plan(p, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kvq_prefix_find_workspace_size(const kvq_page_pool* pool) {
  if (check_pool(pool) != KVQ_OK) return 0;
  return (size_t)pool->batch * 24 + 16;
}

kvq_status kvq_prefix_find(const kvq_page_pool* pool, const int32_t* seq_lens_before, int32_t min_tokens,
                           int32_t max_prefixes, int32_t* prefix_of, int32_t* prefix_lens, int32_t* prefix_table,
                           int32_t* tail_table, int32_t* tail_lens, int32_t* num_prefixes, void* workspace,
                           size_t workspace_bytes, uint32_t* dev_status, void* stream) {
  kvq_status st = check_pool(pool);
  if (st != KVQ_OK) return st;
  if (min_tokens < 0 || max_prefixes < 1) return KVQ_ERR_INVALID_ARG;
  if (max_prefixes > KVQ_MAX_PREFIXES) return KVQ_ERR_UNSUPPORTED;
  // a group's savings and run are compared as one 64-bit number
  const double M = pool->max_blocks_per_seq;
  if (pool->batch * M * (M + 1) >= 0x1p62) return KVQ_ERR_UNSUPPORTED;
  if ((st = check_pool_arrays(pool)) != KVQ_OK) return st;
  if (!prefix_lens || !prefix_table || !aligned(prefix_lens) || !aligned(prefix_table)) return KVQ_ERR_INVALID_ARG;
  if (pool->batch && (!seq_lens_before || !prefix_of || !tail_table || !tail_lens)) return KVQ_ERR_INVALID_ARG;
  if (!aligned(seq_lens_before) || !aligned(prefix_of) || !aligned(tail_table) || !aligned(tail_lens) ||
      !aligned(num_prefixes))
    return KVQ_ERR_INVALID_ARG;
  const size_t need = kvq_prefix_find_workspace_size(pool);
  if (!workspace || !aligned(workspace) || workspace_bytes < need) return KVQ_ERR_WORKSPACE;
  const size_t row = (size_t)pool->max_blocks_per_seq * 4, each = (size_t)pool->batch * 4, most = max_prefixes;
  const Span spans[] = {{pool->block_table, pool->batch * row, false},
                        {seq_lens_before, each, false},
                        {prefix_of, each, true},
                        {prefix_lens, most * 4, true},
                        {prefix_table, most * row, true},
                        {tail_table, pool->batch * row, true},
                        {tail_lens, each, true},
                        {num_prefixes, 4, true},
                        {workspace, need, true}};
  if (!apart(spans)) return KVQ_ERR_INVALID_ARG;
  PrefixFindParams p{};
  p.pool = *pool;
  p.lens = seq_lens_before;
  p.of = prefix_of;
  p.len = prefix_lens;
  p.prefix_table = prefix_table;
  p.tail_table = tail_table;
  p.tail_lens = tail_lens;
  p.num = num_prefixes;
  p.best = reinterpret_cast<unsigned long long*>(workspace);
  p.status = dev_status;
  p.most = max_prefixes;
  p.depth = (int32_t)std::max<int64_t>(1, ceil_div(min_tokens, pool->page_size));
  return from_cuda(launch_prefix_find(p, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kvq_prefix_attn_workspace_size(const kvq_cache_desc* prefix_desc, const kvq_cache_desc* desc,
                                      int32_t num_prefixes, int32_t batch, int32_t num_new, int32_t num_q_heads,
                                      int32_t max_prefix_len, int32_t max_seq_len, int32_t prefix_splits,
                                      int32_t tail_splits) {
  PrefixChoice c;
  if (check_sizes(prefix_desc, desc, num_prefixes, batch, num_new, num_q_heads, max_prefix_len, max_seq_len,
                  prefix_splits, tail_splits, &c) != KVQ_OK ||
      choose(desc, num_prefixes, batch, num_new, num_q_heads, prefix_splits, tail_splits, &c) != KVQ_OK)
    return 0;
  return c.workspace();
}

kvq_status kvq_prefix_attn(const kvq_cache_desc* prefix_desc, const kvq_cache* prefix_cache, int32_t num_prefixes,
                           const kvq_cache_desc* desc, const kvq_cache* cache, int32_t batch, int32_t num_new,
                           int32_t num_q_heads, const uint16_t* q, const int32_t* seq_lens_before,
                           const int32_t* new_lens, const void* plan, size_t plan_bytes, int32_t max_prefix_len,
                           int32_t max_seq_len, int32_t prefix_splits, int32_t tail_splits, float softmax_scale,
                           uint16_t* out, void* workspace, size_t workspace_size, uint32_t* dev_status, void* stream) {
  PrefixChoice c;
  kvq_status st = check_sizes(prefix_desc, desc, num_prefixes, batch, num_new, num_q_heads, max_prefix_len,
                              max_seq_len, prefix_splits, tail_splits, &c);
  if (st != KVQ_OK) return st;
  if (!(softmax_scale >= 0.f) || isinf(softmax_scale)) return KVQ_ERR_INVALID_ARG;
  if ((st = check_cache(desc, cache)) != KVQ_OK) return st;
  if (num_prefixes > 0 && (st = check_cache(prefix_desc, prefix_cache)) != KVQ_OK) return st;
  if (batch == 0 || num_new == 0) return KVQ_OK;
  if (!q || !out || !seq_lens_before || !plan) return KVQ_ERR_INVALID_ARG;
  if (!aligned(q) || !aligned(out) || !aligned(seq_lens_before) || !aligned(new_lens) || !aligned(plan))
    return KVQ_ERR_INVALID_ARG;
  if (plan_bytes < kvq_prefix_plan_size(batch, num_prefixes)) return KVQ_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)batch * num_new * num_q_heads;
  const size_t bytes = (size_t)rows * desc->head_dim * 2, each = (size_t)batch * 4;
  Span spans[] = {{q, bytes, false},
                  {seq_lens_before, each, false},
                  {new_lens, each, false},
                  {plan, kvq_prefix_plan_size(batch, num_prefixes), false},
                  {out, bytes, true},
                  {workspace, 0, true}};
  if (!apart(spans)) return KVQ_ERR_INVALID_ARG;
  if ((st = choose(desc, num_prefixes, batch, num_new, num_q_heads, prefix_splits, tail_splits, &c)) != KVQ_OK)
    return st;
  const size_t need = c.workspace();
  if (need && (!workspace || workspace_size < need || !aligned(workspace))) return KVQ_ERR_WORKSPACE;
  spans[5].bytes = need;
  if (!apart(spans)) return KVQ_ERR_INVALID_ARG;

  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t D = desc->head_dim;
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)desc->head_dim);
  const float scale_log2 = scale * 1.4426950408889634f;
  float *po = nullptr, *pml = nullptr, *to = nullptr, *tml = nullptr;
  if (c.prefixes) carve_partials(workspace, rows, D, c.prefix_splits, &po, &pml);
  if (c.tail_bytes) carve_partials(reinterpret_cast<char*>(workspace) + c.prefix_bytes, rows, D, c.tail_splits, &to, &tml);

  unsigned long long* const started =
      c.word_bytes ? reinterpret_cast<unsigned long long*>(reinterpret_cast<char*>(workspace) + c.prefix_bytes + c.tail_bytes)
                   : nullptr;

  ExtendParams p{};  // what both passes of extend attention share
  p.started = started;
  p.partials = 1;
  p.q = reinterpret_cast<const __half*>(q);
  p.status = dev_status;
  p.num_new = num_new;
  p.Hq = num_q_heads;
  p.G = num_q_heads / desc->num_kv_heads;
  p.scale_log2 = scale_log2;
  const PrefixPlan pl = plan_of(plan, batch, num_prefixes);
  cudaError_t e = cudaSuccess;
  int32_t prefix_limit = 0;
  if (c.prefixes) {
    ExtendParams x = p;
    x.v = view_of(c.pg, prefix_cache);
    dbg_fill(x.v.geom, prefix_desc, prefix_cache, num_prefixes, 0, 0, nullptr, nullptr, nullptr, nullptr, nullptr,
             workspace, workspace_size, dev_status);
    dbg_extent(x.v.geom, KVQ_ARRAY_Q, q, bytes);
    x.ws_o = po;
    x.ws_ml = pml;
    x.batch = num_prefixes;
    x.splits = c.prefix_splits;
    x.chunk = split_chunk(c.max_prefix, c.prefix_splits);
    x.len_limit = prefix_limit = c.max_prefix;
    x.new_lens = new_lens;
    x.plan = pl;
    if ((e = launch_extend_prefix(x, c.pre, s)) != cudaSuccess) return from_cuda(e);
  }
  const int32_t splits = std::max(c.prefix_splits, 1), chunk = split_chunk(c.max_prefix, splits);  // of the prefixes
  if (c.decode.takes) {
    PrefixJoin j{};
    j.o = po;
    j.ml = pml;
    j.of = pl.of;
    j.len = pl.len;
    j.N = num_prefixes;
    j.splits = splits;
    j.chunk = chunk;
    j.limit = prefix_limit;
    j.lift = c.pre.lift;
    j.started = started;
    e = tail_decode(desc, cache, c.tg, batch, num_q_heads, q, seq_lens_before, new_lens, c.max_len, c.decode,
                    scale_log2, to, tml, workspace, workspace_size, dev_status, s, j, out);
    if (c.decode.one) return from_cuda(e);
  } else {
    ExtendParams x = p;
    x.v = view_of(c.tg, cache);
    dbg_fill(x.v.geom, desc, cache, batch, num_q_heads * num_new, 0, q, nullptr, nullptr, seq_lens_before, nullptr,
             workspace, workspace_size, dev_status);
    x.ws_o = to;
    x.ws_ml = tml;
    x.lens_before = seq_lens_before;
    x.new_lens = new_lens;
    x.batch = batch;
    x.splits = c.tail_splits;
    x.chunk = split_chunk(c.max_len, c.tail_splits);
    x.len_limit = c.max_len;
    e = launch_extend_partials(x, c.tail, s);
  }
  if (e != cudaSuccess) return from_cuda(e);

  PrefixJoinParams j{};
  j.geom = c.tg;
  dbg_fill(j.geom, desc, cache, batch, num_q_heads * num_new, 0, nullptr, nullptr, nullptr, seq_lens_before, out,
           workspace, workspace_size, dev_status);
  j.plan = pl;
  j.part[0] = {po, pml, splits, chunk, c.pre.lift};
  j.part[1] = {to, tml, c.tail_splits, split_chunk(c.max_len, c.tail_splits), c.decode.takes ? 0.f : c.tail.lift};
  j.out = reinterpret_cast<__half*>(out);
  j.tail_before = seq_lens_before;
  j.new_lens = new_lens;
  j.T = num_new;
  j.Hq = num_q_heads;
  j.D = desc->head_dim;
  j.prefix_limit = prefix_limit;
  j.tail_limit = c.max_len;
  j.status = dev_status;
  return from_cuda(launch_prefix_join(j, s));
}

}  // extern "C"
