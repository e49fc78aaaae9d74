// Prefixes that several sequences share: the plan of a batch (which sequences
// are on which prefix), what a page pool's table says about it, and the join of
// attention over a prefix with attention over a sequence's own tail.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

// The plan: int32 words in one caller's buffer, made by kvq_prefix_plan.
//   of [B]       prefix of each sequence, -1: none (every entry in [-1, N))
//   order [B]    the sequences, those of prefix 0 first, ascending within one
//   first [N+1]  where each prefix's sequences begin in order
//   len [N]      tokens of each prefix, >= 0
// Kernels that read it check its entries against B and N all the same.
struct PrefixPlan {
  const int32_t* of;
  const int32_t* order;
  const int32_t* first;
  const int32_t* len;
  int32_t B, N;
};
inline __host__ __device__ long long plan_pad(long long n) { return (n + 3) & ~3ll; }
inline size_t plan_words(long long B, long long N) {
  return (size_t)(2 * plan_pad(B) + plan_pad(N + 1) + plan_pad(N));
}
inline PrefixPlan plan_of(const void* words, int32_t B, int32_t N) {
  PrefixPlan p;
  p.of = reinterpret_cast<const int32_t*>(words);
  p.order = p.of + plan_pad(B);
  p.first = p.order + plan_pad(B);
  p.len = p.first + plan_pad(N + 1);
  p.B = B;
  p.N = N;
  return p;
}

// Tokens of prefix n that count: 0 for one that its cache or the call's bound
// does not hold (the join flags it).
__device__ __forceinline__ int prefix_len(const PrefixPlan& p, int n, int limit) {
  const int len = __ldg(p.len + n);
  return len > limit ? 0 : max(len, 0);
}

// The sequence at place i of `order`.
__device__ __forceinline__ int plan_member(const PrefixPlan& p, int i) {
  const int b = __ldg(p.order + min(max(i, 0), p.B - 1));
  return min(max(b, 0), p.B - 1);
}

// Tile `flat` of the tiles of `rows` rows that all prefixes' members make, one
// prefix after another (a member is `each` rows): its prefix n (-1: no such
// tile), its place among that prefix's tiles, and the prefix's members.  Every
// lane of a warp calls it; 32 prefixes a turn, up to the last that has members.
struct PrefixTile {
  int n, tile, first, count;
};
__device__ __forceinline__ PrefixTile prefix_tile(const PrefixPlan& p, long long flat, int each, int rows) {
  const int lane = threadIdx.x & 31;
  const int all = __ldg(p.first + p.N);  // members of all prefixes
  for (int base = 0; base < p.N; base += 32) {
    const int n = base + lane;
    int f0 = 0, count = 0;
    if (n < p.N) {
      f0 = min(max(__ldg(p.first + n), 0), p.B);
      count = min(max(__ldg(p.first + n + 1), f0), p.B) - f0;
    }
    const bool last = __any_sync(0xffffffffu, f0 + count >= all);
    if (n < p.N && __ldg(p.len + n) <= 0) count = 0;
    const int tiles = (int)(((long long)count * each + rows - 1) / rows);
    int upto = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const int total = __shfl_sync(0xffffffffu, upto, 31);
    if (flat < total) {
      const int hit = __ffs(__ballot_sync(0xffffffffu, flat < upto)) - 1;
      PrefixTile t;
      t.n = base + hit;
      t.tile = (int)flat - __shfl_sync(0xffffffffu, upto - tiles, hit);
      t.first = __shfl_sync(0xffffffffu, f0, hit);
      t.count = __shfl_sync(0xffffffffu, count, hit);
      return t;
    }
    if (last) break;
    flat -= total;
  }
  return PrefixTile{-1, 0, 0, 0};
}
// The tokens of a prefix's members, as rows of `G` heads: row r of the prefix
// (this lane's) is head r % G of token *tok, counted b T + t over the padded
// batch (rows behind the last: some token of the first member).  Returns the
// rows there are.  Of a padded batch only live tokens make rows, found by a
// scan over the members, 32 a turn (24 sequences of 1 to 200 tokens: 442 us with
// a row for each of the 200, half of them dead, 224 without, when this came); one new token a
// sequence takes its place in any case.  Every lane of a warp calls it.
__device__ __forceinline__ int prefix_rows(const PrefixPlan& p, const PrefixTile& pt, const int32_t* new_lens, int T,
                                           int G, long long r, int* tok) {
  const int lane = threadIdx.x & 31;
  if (!new_lens || T == 1) {
    const int live = pt.count * T * G;
    const int x = (int)(r < live ? r : 0) / G, m = x / T;
    *tok = plan_member(p, pt.first + m) * T + (x - m * T);
    return live;
  }
  const int want = (int)(r / G);
  int base = 0;
  *tok = plan_member(p, pt.first) * T;
  for (int i0 = 0; i0 < pt.count; i0 += 32) {
    const bool in = i0 + lane < pt.count;
    const int b = plan_member(p, pt.first + (in ? i0 + lane : 0));
    const int n = in ? max(new_rows_of(new_lens, b, T), 0) : 0;
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const int total = __shfl_sync(0xffffffffu, upto, 31), x = want - base;
    int k = 0;  // the first lane with upto > x
#pragma unroll
    for (int o = 16; o; o >>= 1) k += __shfl_sync(0xffffffffu, upto, k + o - 1) <= x ? o : 0;
    const int bk = __shfl_sync(0xffffffffu, b, k), before = __shfl_sync(0xffffffffu, upto - n, k);
    if (x >= 0 && x < total) *tok = bk * T + (x - before);
    base += total;
  }
  return base * G;
}
// At most so many tiles.
inline long long prefix_tiles_bound(long long B, long long N, long long each, long long rows) {
  return B * each / rows + (B < N ? B : N);
}

struct PrefixPlanParams {
  const int32_t* of;
  const int32_t* len;
  int32_t* plan;
  uint32_t* status;
  int32_t B, N;
};
cudaError_t launch_prefix_plan(const PrefixPlanParams& p, cudaStream_t stream);

struct PrefixFindParams {
  kvq_page_pool pool;
  const int32_t* lens;
  int32_t* of;
  int32_t* len;           // [most]
  int32_t* prefix_table;  // [most][max_blocks]
  int32_t* tail_table;    // [batch][max_blocks]
  int32_t* tail_lens;
  int32_t* num;           // may be null
  unsigned long long* best;  // workspace (see the kernels)
  uint32_t* status;
  int32_t most, depth;    // depth: blocks a prefix has at least
};
cudaError_t launch_prefix_find(const PrefixFindParams& p, cudaStream_t stream);

// The join of a row's partials over its prefix and over its tail.  A partial is
// (m, l, o): reference maximum in log2 units, sum and weighted sum of 2^(s - m),
// both times 2^lift.
struct PrefixPartials {
  const float* o;   // [row][splits][D]
  const float* ml;  // [row][splits][2]
  int32_t splits, chunk;
  float lift;
};
struct PrefixJoinParams {
  CacheGeom geom;  // (debug extents: out, workspace)
  PrefixPlan plan;
  PrefixPartials part[2];  // prefix, tail
  __half* out;             // [B][T][Hq][D]
  const int32_t* tail_before;
  const int32_t* new_lens;
  int32_t T, Hq, D;
  int32_t prefix_limit, tail_limit;
  uint32_t* status;
};
cudaError_t launch_prefix_join(const PrefixJoinParams& p, cudaStream_t stream);

}  // namespace kvq
