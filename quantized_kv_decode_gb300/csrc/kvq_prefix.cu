// Shared prefixes: the plan of a batch, the prefixes that a page pool's table
// holds, and the join of prefix and tail attention.
#include <algorithm>

#include "kvq_decode_fast.cuh"
#include "kvq_prefix.cuh"
#include "kvq_rope.cuh"

namespace kvq {
namespace {

__device__ __forceinline__ void flag(uint32_t* status, uint32_t f) {
  if (f && status) atomicOr(status, f);
}
__device__ __forceinline__ unsigned lanes_below() { return (1u << (threadIdx.x & 31)) - 1u; }

// ---- the plan ----------------------------------------------------------
//
// A warp per prefix (and one more for the sequences without): it counts the
// sequences of the prefixes before its own, then writes its own in ascending
// order.  Integer sums and one writer an entry, so the plan is determined by
// the inputs.  Bound by latency: two passes over B entries from the L2 cache (4.9
// us by itself for 4 to 256 sequences).
constexpr int kPlanWarps = 8;
__device__ __forceinline__ int prefix_of(const PrefixPlanParams& p, int b, uint32_t& flags) {
  const int n = __ldg(p.of + b);
  if (n >= -1 && n < p.N) return n;
  flags |= KVQ_FLAG_BLOCK_TABLE;
  return -1;
}
__global__ void __launch_bounds__(kPlanWarps * 32) prefix_plan_kernel(const __grid_constant__ PrefixPlanParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int n = blockIdx.x * kPlanWarps + (threadIdx.x >> 5);  // N: the sequences without a prefix
  if (n > p.N) return;
  int32_t* const of = p.plan;
  int32_t* const order = of + plan_pad(p.B);
  int32_t* const first = order + plan_pad(p.B);
  int32_t* const len = first + plan_pad(p.N + 1);
  uint32_t flags = 0;
  int before = 0;
#pragma unroll 4
  for (int b = lane; b < p.B; b += 32) {
    const int x = prefix_of(p, b, flags);
    before += x >= 0 && x < n;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0) {
    first[n] = before;
    if (n < p.N) {
      int l = __ldg(p.len + n);
      if (l < 0) flags |= KVQ_FLAG_SEQ_LEN, l = 0;
      len[n] = l;
    }
  }
  if (n == p.N && lane < 3) {  // the words between the arrays: every word of a plan is its inputs'
    if (p.B + lane < plan_pad(p.B)) of[p.B + lane] = order[p.B + lane] = 0;
    if (p.N + 1 + lane < plan_pad(p.N + 1)) first[p.N + 1 + lane] = 0;
    if (p.N + lane < plan_pad(p.N)) len[p.N + lane] = 0;
  }
  const int mine = n < p.N ? n : -1;
#pragma unroll 4
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    uint32_t unused = 0;
    const bool hit = b < p.B && prefix_of(p, b, unused) == mine;
    const unsigned m = __ballot_sync(0xffffffffu, hit);
    if (hit) {
      order[before + __popc(m & lanes_below())] = b;
      of[b] = mine;
    }
    before += __popc(m);
  }
  flag(p.status, flags);
}

// ---- prefixes in a page pool's table -------------------------------------
//
// Three kernels: leaders and runs (a warp a sequence), savings and the numbers
// of the groups (a warp a sequence, the last block numbers them), tables (a warp
// a row).  Bound by memory latency: keys and (leader, run) pairs are brought to
// shared memory by the block, rows are read and written 256 entries at a time.
// 2048 sequences of up to 1012 blocks: 27 us, of which 17, 9 and 8 by themselves
// (43 when rows went 128 at a time and every warp looked through the pairs and the
// groups' savings in global memory); 8 sequences 6.2.  The rows' first entries
// fetched before the leaders are known: 17.7 -> 26 us of the first kernel.
// Integer sums and maxima only: the result does not depend on the order.
constexpr int kFindWarps = 16;
constexpr int kFindHeld = 4096;  // keys or pairs held in shared memory at a time
constexpr int kRowLoads = 8;     // loads in flight a lane
constexpr int kRanks = 4;        // sequences a thread numbers at a time

__device__ __forceinline__ bool is_page(const kvq_page_pool& pl, int e) { return e >= 0 && e < pl.num_pages; }

// Whole blocks of sequence b (0 for a length that cannot be), flagged.
__device__ __forceinline__ int whole_blocks(const PrefixFindParams& p, int b, uint32_t& flags) {
  const kvq_page_pool& pl = p.pool;
  const int L = __ldg(p.lens + b);
  if (L < 0 || (long long)L > (long long)pl.page_size * pl.max_blocks_per_seq) {
    flags |= KVQ_FLAG_SEQ_LEN;
    return 0;
  }
  return L / pl.page_size;
}
// What candidates share: the page in block depth - 1; -1: no candidate.
__device__ __forceinline__ int key_of(const PrefixFindParams& p, int b) {
  uint32_t unused = 0;
  if (whole_blocks(p, b, unused) < p.depth) return -1;
  const int e = __ldg(p.pool.block_table + (long long)b * p.pool.max_blocks_per_seq + p.depth - 1);
  return is_page(p.pool, e) ? e : -1;
}

struct FindSpace {
  unsigned long long* best;  // [B] of a leader: (blocks saved) (M + 1) + run
  int2* pair;                // [B] leader (-1: member of no group), run
  int32_t* rank;             // [B] of a leader whose group has a prefix
  int32_t* lead;             // [B] the leaders by rank
  int32_t* done;             // blocks of the second kernel that are through; prefixes
};
__device__ __forceinline__ FindSpace space_of(const PrefixFindParams& p) {
  FindSpace s;
  const int B = p.pool.batch;
  s.best = p.best;
  s.pair = reinterpret_cast<int2*>(p.best + B);
  s.rank = reinterpret_cast<int32_t*>(s.pair + B);
  s.lead = s.rank + B;
  s.done = s.lead + B;
  return s;
}

// A warp per sequence: its leader (lowest sequence with the same key) and how
// many leading blocks it shares with it.
__global__ void __launch_bounds__(kFindWarps * 32) find_leaders_kernel(const __grid_constant__ PrefixFindParams p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ int keys[kFindHeld];
  const kvq_page_pool& pl = p.pool;
  const int B = pl.batch, M = pl.max_blocks_per_seq;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x * kFindWarps + (threadIdx.x >> 5);
  const int last = min(B, (int)(blockIdx.x + 1) * kFindWarps);  // no leader lies behind its members
  int own = -1, lead = b;
  if (b < B) own = key_of(p, b);
  bool found = false;
  for (int base = 0; base < last; base += kFindHeld) {
    const int n = min(kFindHeld, last - base);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) keys[i] = key_of(p, base + i);
    __syncthreads();
    for (int i = 0; own >= 0 && !found && i < n; i += 32) {
      const unsigned m = __ballot_sync(0xffffffffu, i + lane < n && keys[i + lane] == own);
      if (m) {
        lead = base + i + __ffs(m) - 1;  // (at the latest the sequence itself)
        found = true;
      }
    }
  }
  const FindSpace s = space_of(p);
  if (blockIdx.x == 0 && threadIdx.x == 0) s.done[0] = 0;
  if (b >= B) return;
  uint32_t flags = 0, unused = 0;
  const int whole = whole_blocks(p, b, flags);
  int run = 0;
  if (own >= 0) {
    const int most = min(whole, whole_blocks(p, lead, unused));
    const int32_t* x = pl.block_table + (long long)b * M;
    const int32_t* y = pl.block_table + (long long)lead * M;
    run = most;
    for (int j0 = 0; j0 < most && run == most; j0 += 32 * kRowLoads) {
      int e[kRowLoads], f[kRowLoads];
#pragma unroll
      for (int u = 0; u < kRowLoads; ++u) {
        const int j = j0 + 32 * u + lane;
        e[u] = j < most ? __ldg(x + j) : 0;
        f[u] = j < most ? __ldg(y + j) : 0;
      }
#pragma unroll
      for (int u = kRowLoads - 1; u >= 0; --u) {
        const int j = j0 + 32 * u + lane;
        const unsigned m = __ballot_sync(0xffffffffu, j < most && (e[u] != f[u] || !is_page(pl, e[u])));
        if (m) run = j0 + 32 * u + __ffs(m) - 1;
      }
    }
  }
  if (lane == 0) {
    s.pair[b] = make_int2(run >= p.depth ? lead : -1, run);
    s.best[b] = 0;
    flag(p.status, flags);
  }
}

// A warp per sequence: what its run would save as the group's prefix.  The last
// block through numbers the groups that have one.
__global__ void __launch_bounds__(kFindWarps * 32) find_savings_kernel(const __grid_constant__ PrefixFindParams p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ __align__(16) int2 pairs[kFindHeld];
  __shared__ int sums[kFindWarps + 1], is_last;
  const int B = p.pool.batch;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x * kFindWarps + warp;
  const FindSpace s = space_of(p);
  const int2 own = b < B ? s.pair[b] : make_int2(-1, 0);
  int with = 0;  // members with at least this run
  for (int base = 0; base < B; base += kFindHeld) {
    const int n = min(kFindHeld, B - base);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) pairs[i] = s.pair[base + i];
    __syncthreads();
    if (own.x >= 0) {  // (two pairs a load)
      const int4* const two = reinterpret_cast<const int4*>(pairs);
#pragma unroll 4
      for (int i = lane; i < n / 2; i += 32) {
        const int4 v = two[i];
        with += (v.x == own.x && v.y >= own.y) + (v.z == own.x && v.w >= own.y);
      }
      if ((n & 1) && lane == 0) with += pairs[n - 1].x == own.x && pairs[n - 1].y >= own.y;
    }
  }
  with = __reduce_add_sync(0xffffffffu, with);
  if (lane == 0 && own.x >= 0 && with > 1)
    atomicMax(s.best + own.x, (unsigned long long)(with - 1) * own.y * (unsigned)(p.pool.max_blocks_per_seq + 1u) + own.y);
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) is_last = atomicAdd(s.done, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  int groups = 0;
  for (int base = 0; base < B; base += kFindWarps * 32 * kRanks) {
    // a warp takes 32 kRanks neighbours, so that one look at the warps' sums does
    bool has[kRanks];
    const int i0 = base + warp * (32 * kRanks) + lane;
#pragma unroll
    for (int u = 0; u < kRanks; ++u) has[u] = i0 + 32 * u < B && __ldcg(s.best + i0 + 32 * u) != 0;
    int mine = 0;
#pragma unroll
    for (int u = 0; u < kRanks; ++u) mine += __popc(__ballot_sync(0xffffffffu, has[u]));
    if (lane == 0) sums[warp] = mine;
    __syncthreads();
    int r = groups, all = 0;
#pragma unroll
    for (int w = 0; w < kFindWarps; ++w) {
      r += w < warp ? sums[w] : 0;
      all += sums[w];
    }
#pragma unroll
    for (int u = 0; u < kRanks; ++u) {
      const unsigned m = __ballot_sync(0xffffffffu, has[u]);
      if (has[u]) {
        s.rank[i0 + 32 * u] = r + __popc(m & lanes_below());
        s.lead[r + __popc(m & lanes_below())] = i0 + 32 * u;
      }
      r += __popc(m);
    }
    groups += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    s.done[1] = groups;
    if (p.num) *p.num = groups;
  }
}

// Copies n entries of a table row, -1 behind, by one warp.
__device__ __forceinline__ void copy_row(const int32_t* from, int n, int32_t* to, int M, int lane) {
  for (int j0 = 0; j0 < M; j0 += 32 * kRowLoads) {
    int e[kRowLoads];
#pragma unroll
    for (int u = 0; u < kRowLoads; ++u) {
      const int j = j0 + 32 * u + lane;
      e[u] = j < n ? __ldg(from + j) : -1;
    }
#pragma unroll
    for (int u = 0; u < kRowLoads; ++u) {
      const int j = j0 + 32 * u + lane;
      if (j < M) to[j] = e[u];
    }
  }
}

// A warp per sequence (its prefix and its tail's row) and per prefix (its row).
__global__ void __launch_bounds__(kFindWarps * 32) find_tables_kernel(const __grid_constant__ PrefixFindParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const kvq_page_pool& pl = p.pool;
  const int B = pl.batch, M = pl.max_blocks_per_seq;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * kFindWarps + (threadIdx.x >> 5);
  const FindSpace s = space_of(p);
  const unsigned base = (unsigned)M + 1u;
  if (w < B) {
    const int b = (int)w;
    const int2 own = s.pair[b];
    const int prefix = own.x < 0 ? 0 : (int)(s.best[own.x] % base);
    int n = -1;
    if (prefix > 0 && own.y >= prefix) {
      const int r = s.rank[own.x];
      if (r < p.most) n = r;
    }
    const int shift = n >= 0 ? prefix : 0;
    if (lane == 0) {
      p.of[b] = n;
      p.tail_lens[b] = __ldg(p.lens + b) - shift * pl.page_size;
    }
    copy_row(pl.block_table + (long long)b * M + shift, M - shift, p.tail_table + (long long)b * M, M, lane);
  } else if (w < (long long)B + p.most) {
    const int n = (int)(w - B);
    const int lead = B > 0 && n < s.done[1] ? s.lead[n] : -1;
    const int prefix = lead < 0 ? 0 : (int)(s.best[lead] % base);
    if (lane == 0) {
      p.len[n] = prefix * pl.page_size;
      if (B == 0 && n == 0 && p.num) *p.num = 0;
    }
    copy_row(pl.block_table + (long long)max(lead, 0) * M, prefix, p.prefix_table + (long long)n * M, M, lane);
  }
}

// ---- the join -----------------------------------------------------------
//
// out = sum_i 2^(m_i - lift_i - X) o_i / sum_i 2^(m_i - lift_i - X) l_i over the
// partials of a row, X their largest m - lift.  A block takes a token, or some of
// its heads where tokens are few: D / 4 threads a row, four channels each.  What a
// token needs (its sequence, lengths, how many partials) is worked out once for all
// its heads: with a block for eight rows wherever they lie, each thread dividing for
// itself, 4800 tokens (half of them live) of 32 heads of 128 took 57 us by itself
// and cold, 37 so, 29 with the pairs of unsplit passes joined without a loop.  Bound
// by instructions and latency (53 % of the issue slots at 3.2 TB/s).
constexpr int kJoinBlocks = 1216;  // eight an SM

// The heads of token `tok` that are this block's: partials 0 .. use - 1 are the
// prefix's, those up to total the tail's; U of them in flight (two are all there
// are where neither pass is split: 195 -> 188 us of the call with those tokens).
template <int U>
__device__ __forceinline__ void join_rows(const PrefixJoinParams& p, unsigned tok, int use, int total) {
  const CacheGeom& c = p.geom;
  const int per = p.D / 4, step = 256 / per;  // 16, 32 or 64 threads a row
  const int d = threadIdx.x % per * 4;
  for (int h = blockIdx.y * step + threadIdx.x / per; h < p.Hq; h += gridDim.y * step) {
    const long long row = (long long)tok * p.Hq + h;
    const long long at0 = row * p.part[0].splits, at1 = row * p.part[1].splits - use;
    float M = -INFINITY, den = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < total; s0 += U) {
      float2 v[U];
      float4 x[U];
      float Mn = M;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = s0 + u;
        const bool pre = i < use;
        const long long at = (pre ? at0 : at1) + i;
        const float* const ml = (pre ? p.part[0].ml : p.part[1].ml) + 2 * at;
        const float* const o = (pre ? p.part[0].o : p.part[1].o) + at * p.D + d;
        v[u] = make_float2(-INFINITY, 0.f);
        x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < total && KVQ_IN(c, KVQ_ARRAY_WORKSPACE, ml, 8) && KVQ_IN(c, KVQ_ARRAY_WORKSPACE, o, 16)) {
          v[u] = *reinterpret_cast<const float2*>(ml);
          v[u].x -= pre ? p.part[0].lift : p.part[1].lift;
          x[u] = *reinterpret_cast<const float4*>(o);
        }
        Mn = fmaxf(Mn, v[u].x);
      }
      const float base = Mn == -INFINITY ? 0.f : Mn, a = fast::ex2(M - base);
      num = make_float4(num.x * a, num.y * a, num.z * a, num.w * a);
      den *= a;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (v[u].x == -INFINITY && !(v[u].y != 0.f)) continue;  // nothing seen there
        const float f = fast::ex2(v[u].x - base);
        num.x = fmaf(f, x[u].x, num.x);
        num.y = fmaf(f, x[u].y, num.y);
        num.z = fmaf(f, x[u].z, num.z);
        num.w = fmaf(f, x[u].w, num.w);
        den = fmaf(f, v[u].y, den);
      }
      M = Mn;
    }
    const float inv = den != 0.f ? 1.f / den : 0.f;
    uint2* to = reinterpret_cast<uint2*>(p.out + row * p.D + d);
    if (KVQ_IN(c, KVQ_ARRAY_OUT, to, 8))
      *to = make_uint2(fast::pack_h2(num.x * inv, num.y * inv), fast::pack_h2(num.z * inv, num.w * inv));
  }
}
__global__ void __launch_bounds__(256) prefix_join_kernel(const __grid_constant__ PrefixJoinParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const CacheGeom& c = p.geom;
  // prefixes that do not fit, whether a sequence is on them or not
  if (blockIdx.y == 0)
    for (long long n = (long long)blockIdx.x * 256 + threadIdx.x; n < p.plan.N; n += (long long)gridDim.x * 256)
      if (__ldg(p.plan.len + n) > p.prefix_limit) flag(p.status, KVQ_FLAG_SEQ_LEN);
  const unsigned tok = blockIdx.x;
  const int b = (int)(tok / (unsigned)p.T), t = (int)(tok - (unsigned)b * p.T);
  const int n_new = new_rows_of(p.new_lens, b, p.T);
  if (t >= n_new) return;
  const int before = checked_len(c, p.tail_before, b, -1);
  const bool fits = before >= 0 && (long long)before + n_new <= p.tail_limit;
  int use = 0, total = fits ? (before + n_new + p.part[1].chunk - 1) / p.part[1].chunk : 0;  // of the prefix, of both
  const int n = __ldg(p.plan.of + b);
  if (fits && n >= 0 && n < p.plan.N)
    use = (prefix_len(p.plan, n, p.prefix_limit) + p.part[0].chunk - 1) / p.part[0].chunk;
  total += use;
  if (total <= 2) join_rows<2>(p, tok, use, total);
  else join_rows<4>(p, tok, use, total);
}

}  // namespace

cudaError_t launch_prefix_plan(const PrefixPlanParams& p, cudaStream_t stream) {
  const long long warps = (long long)p.N + 1;
  return launch_pdl(prefix_plan_kernel, dim3((unsigned)((warps + kPlanWarps - 1) / kPlanWarps)), dim3(kPlanWarps * 32),
                    0, stream, p);
}

cudaError_t launch_prefix_find(const PrefixFindParams& p, cudaStream_t stream) {
  const auto grid = [](long long warps) { return dim3((unsigned)((warps + kFindWarps - 1) / kFindWarps)); };
  const int B = p.pool.batch;
  cudaError_t e = cudaSuccess;
  if (B > 0) e = launch_pdl(find_leaders_kernel, grid(B), dim3(kFindWarps * 32), 0, stream, p);
  if (e == cudaSuccess && B > 0) e = launch_pdl(find_savings_kernel, grid(B), dim3(kFindWarps * 32), 0, stream, p);
  if (e == cudaSuccess)
    e = launch_pdl(find_tables_kernel, grid((long long)B + p.most), dim3(kFindWarps * 32), 0, stream, p);
  return e;
}

cudaError_t launch_prefix_join(const PrefixJoinParams& p, cudaStream_t stream) {
  const long long tokens = (long long)p.plan.B * p.T;
  const int step = 256 / (p.D / 4), most = (p.Hq + step - 1) / step;
  const long long slices = std::min<long long>(std::min(most, 65535), (kJoinBlocks + tokens - 1) / tokens);
  return launch_pdl(prefix_join_kernel, dim3((unsigned)tokens, (unsigned)slices), dim3(256), 0, stream, p);
}

}  // namespace kvq
