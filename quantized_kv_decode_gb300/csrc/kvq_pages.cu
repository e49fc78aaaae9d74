// Page pool kernels: reorder (fork, trim, permute, free), reserve, compact,
// and the copy of pages in the layers' caches.
//
// What bounds them.  reorder, reserve and compact: the latency of a few
// dependent passes over the table and counts (256 sequences of 190 blocks: 5 us
// and, for the first two blocks of each, 11 us; reserve and compact are one
// CTA, so that their prefix sums need no second launch).  copy:
// memory, the rate of a plain copy (16 layers of a compaction, 646 us).
//
// Reference counts change by integer atomics only, whose sums do not depend
// on the order, and pages are handed out by prefix sums over the page index,
// so every result is determined by the inputs.
#include "kvq_pages.cuh"

namespace kvq {
namespace {

constexpr int kOne = 1024;  // threads of the single-CTA kernels

__device__ __forceinline__ void flag(uint32_t* status, uint32_t f) {
  if (f && status) atomicOr(status, f);
}

// Exclusive prefix sum of x over the CTA's threads (kOne of them), and the
// total.  `scratch`: 33 ints of shared memory, free again on return.
__device__ __forceinline__ int block_scan(int x, int* scratch, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const int w = lane < kOne / 32 ? scratch[lane] : 0;
    int s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    scratch[lane] = s - w;
    if (lane == 31) scratch[32] = s;
  }
  __syncthreads();
  const int r = scratch[warp] + inc - x;
  *total = scratch[32];
  __syncthreads();
  return r;
}

// Which of pages i .. i + 3 (i a multiple of 4) exist and have count 0, and
// count > 0, as bits.
__device__ __forceinline__ void states4(const kvq_page_pool& pl, int i, int* free4, int* live4) {
  int c[4] = {-1, -1, -1, -1};
  if (i + 4 <= pl.num_pages) {
    const int4 v = *reinterpret_cast<const int4*>(pl.ref_count + i);
    c[0] = v.x, c[1] = v.y, c[2] = v.z, c[3] = v.w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < pl.num_pages) c[e] = pl.ref_count[i + e];
  }
  *free4 = (c[0] == 0) | (c[1] == 0) << 1 | (c[2] == 0) << 2 | (c[3] == 0) << 3;
  *live4 = (c[0] > 0) | (c[1] > 0) << 1 | (c[2] > 0) << 2 | (c[3] > 0) << 3;
}

// ---- reorder ----------------------------------------------------------

// One CTA per group of `cols` table columns: the columns of every row are
// read to shared memory, then written through parent[], so the table changes
// in place.  Counts: -1 for every old entry, +1 for every new one.
__global__ void __launch_bounds__(1024) reorder_kernel(const __grid_constant__ PoolParams p, int cols) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ int32_t old[];  // [batch][cols]
  const kvq_page_pool& pl = p.pool;
  const int M = pl.max_blocks_per_seq;
  const int c0 = blockIdx.x * cols;
  uint32_t flags = 0;
  for (int i = threadIdx.x; i < pl.batch * cols; i += blockDim.x) {
    const int b = i / cols, c = c0 + i % cols;
    int e = -1;
    if (c < M) {
      e = pl.block_table[(long long)b * M + c];
      if (e >= pl.num_pages) flags |= KVQ_FLAG_BLOCK_TABLE;
      if (e < 0 || e >= pl.num_pages) e = -1;
    }
    old[i] = e;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < pl.batch * cols; i += blockDim.x) {
    const int b = i / cols, k = i % cols, c = c0 + k;
    if (c >= M) continue;
    int par = __ldg(p.parent + b);
    if (par < -1 || par >= pl.batch) {
      flags |= KVQ_FLAG_BLOCK_TABLE;
      par = -1;
    }
    int blocks = M;
    if (p.keep_lens) {
      const int keep = __ldg(p.keep_lens + b);
      if (keep < 0 || (long long)keep > (long long)M * pl.page_size) {
        if (par >= 0) flags |= KVQ_FLAG_SEQ_LEN;
        blocks = 0;
      } else {
        blocks = (int)(((long long)keep + pl.page_size - 1) / pl.page_size);
      }
    }
    const int e = (par >= 0 && c < blocks) ? old[par * cols + k] : -1;
    const int was = old[i];
    pl.block_table[(long long)b * M + c] = e;
    if (e != was) {
      if (e >= 0) atomicAdd(pl.ref_count + e, 1);
      if (was >= 0) atomicSub(pl.ref_count + was, 1);
    }
  }
  flag(p.status, flags);
}

// ---- reserve ----------------------------------------------------------

// What sequence b asks for: the touched blocks [first, last), and whether
// the first holds tokens from before (partial).
struct Ask {
  int first, last, n;
  bool partial;
  uint32_t flags;
};
__device__ __forceinline__ Ask ask_of(const PoolParams& p, int b) {
  const kvq_page_pool& pl = p.pool;
  Ask a{0, 0, 0, false, 0u};
  const int before = __ldg(p.seq_lens_before + b);
  const int n = p.new_lens ? __ldg(p.new_lens + b) : p.num_new;
  if (n == 0 && before >= 0) return a;
  if (n < 0 || n > p.num_new || before < 0 ||
      (long long)before + n > (long long)pl.max_blocks_per_seq * pl.page_size) {
    a.flags = KVQ_FLAG_SEQ_LEN;
    return a;
  }
  a.n = n;
  a.first = before / pl.page_size;
  a.last = (int)(((long long)before + n + pl.page_size - 1) / pl.page_size);
  a.partial = before % pl.page_size != 0;
  return a;
}

__device__ __forceinline__ int entry(const PoolParams& p, int b, int j) {
  const int e = p.pool.block_table[(long long)b * p.pool.max_blocks_per_seq + j];
  return (e < 0 || e >= p.pool.num_pages) ? -1 : e;
}

// One CTA.  Shared: mine[b] = the mapped partial page of b (-1: none), later
// whether it is replaced; at[b] = exclusive prefix of the pages needed.
__global__ void __launch_bounds__(kOne) reserve_kernel(const __grid_constant__ PoolParams p, int lps) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ int32_t sh[];
  __shared__ int scratch[33];
  const kvq_page_pool& pl = p.pool;
  // a group of lps lanes (4 .. 32) per sequence: as many as it touches blocks
  const int B = pl.batch, groups = kOne / lps, group = threadIdx.x / lps, gl = threadIdx.x % lps;
  const int shift = threadIdx.x & 31 & ~(lps - 1);  // the group's first lane
  const unsigned all = lps == 32 ? 0xffffffffu : (1u << lps) - 1u;
  const long long M = pl.max_blocks_per_seq;
  int32_t* mine = sh;
  int32_t* at = sh + B;
  uint32_t flags = 0;

  for (int b = threadIdx.x; b < B; b += kOne) {
    const Ask a = ask_of(p, b);
    flags |= a.flags;
    mine[b] = (a.n && a.partial) ? entry(p, b, a.first) : -1;
  }
  __syncthreads();
  // A shared partial page is replaced for all its askers but the last, who
  // keeps it when every holder asks: how many ask for a page, and the last of
  // them, are counted in ws (16384 forks of one page, all asking: 250 us;
  // 2580 when each looked through the rows before it).
  for (int b = threadIdx.x; b < B; b += kOne) {
    const int e = mine[b];
    at[b] = e >= 0 ? pl.ref_count[e] : 0;
    if (at[b] > 1) p.ws[e] = 0, p.ws[pl.num_pages + e] = -1;
  }
  __syncthreads();
  for (int b = threadIdx.x; b < B; b += kOne)
    if (at[b] > 1) {
      atomicAdd(p.ws + mine[b], 1);
      atomicMax(p.ws + pl.num_pages + mine[b], b);
    }
  __syncthreads();
  for (int b = threadIdx.x; b < B; b += kOne) {
    const int e = mine[b], refs = at[b];
    int replaced = 0;
    if (refs > 1) {
      const int asking = p.ws[e];
      replaced = asking < refs || p.ws[pl.num_pages + e] != b;
      if (asking > refs) {  // (a count that is too low: rank k of the askers leaves refs - k)
        int k = 0;
        for (int i = 0; i < b; ++i) k += mine[i] == e;
        replaced = refs - k > 1;
      }
    }
    at[b] = replaced;
  }
  __syncthreads();
  for (int b = threadIdx.x; b < B; b += kOne) mine[b] = at[b];
  __syncthreads();
  // pages needed per sequence
  for (int b0 = 0; b0 < B; b0 += groups) {
    const int b = b0 + group;
    int need = 0;
    if (b < B) {
      const Ask a = ask_of(p, b);
      for (int j = a.first + gl; j < a.last; j += lps) {
        const int e = entry(p, b, j);
        const bool part = j == a.first && a.partial;
        need += e < 0 ? 1 : (part ? mine[b] : pl.ref_count[e] > 1);
      }
    }
    for (int o = lps >> 1; o; o >>= 1) need += __shfl_xor_sync(0xffffffffu, need, o);
    if (gl == 0 && b < B) at[b] = need;
  }
  __syncthreads();
  int total = 0;
  for (int b0 = 0; b0 < B; b0 += kOne) {
    const int b = b0 + threadIdx.x;
    int sum;
    const int ex = block_scan(b < B ? at[b] : 0, scratch, &sum);
    if (b < B) at[b] = total + ex;
    total += sum;
  }
  // the lowest free pages, in order
  int found = 0;
  for (int i0 = 0; i0 < pl.num_pages && found < total; i0 += 4 * kOne) {
    const int i = i0 + 4 * threadIdx.x;
    int free4 = 0, live4 = 0, sum;
    if (i < pl.num_pages) states4(pl, i, &free4, &live4);
    int at_free = found + block_scan(__popc(free4), scratch, &sum);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if ((free4 >> e & 1) && at_free < total) p.ws[at_free] = i + e, ++at_free;
    found += sum;
  }
  __syncthreads();
  const bool ok = found >= total;
  if (!ok && threadIdx.x == 0) flags |= KVQ_FLAG_POOL_EMPTY;
  for (int b0 = 0; b0 < B; b0 += groups) {
    const int b = b0 + group;
    Ask a{0, 0, 0, false, 0u};
    if (b < B) a = ask_of(p, b);
    int src = -1, dst = -1, next = b < B ? at[b] : 0;
    // (as many rounds as the warp's longest group: the ballot needs all lanes)
    for (int j0 = a.first; __any_sync(0xffffffffu, ok && j0 < a.last); j0 += lps) {
      const int j = j0 + gl;
      const bool mine_j = ok && j < a.last;
      const int e = mine_j ? entry(p, b, j) : 0;
      const bool part = j == a.first && a.partial;
      const bool take = mine_j && (e < 0 || (part ? mine[b] != 0 : pl.ref_count[e] > 1));
      const unsigned who = (__ballot_sync(0xffffffffu, take) >> shift) & all;
      if (take) {
        const int rank = next + __popc(who & ((1u << gl) - 1));
        const int page = p.ws[rank];
        pl.block_table[(long long)b * M + j] = page;
        pl.ref_count[page] = 1;
        p.ws[pl.num_pages + rank] = e;
        if (e >= 0 && part) {
          src = e;
          dst = page;
        }
      }
      next += __popc(who);
    }
    if (gl == 0 && b < B) {  // the partial block is the first one: lane 0 of the first round
      p.copy_src[b] = src;
      p.copy_dst[b] = dst;
      if (p.granted) p.granted[b] = ok ? a.n : 0;
    }
  }
  // the replaced pages' holders are counted off last, so that every decision
  // above went by the counts before the call
  __syncthreads();
  if (ok)
    for (int k = threadIdx.x; k < total; k += kOne) {
      const int e = p.ws[pl.num_pages + k];
      if (e >= 0) atomicSub(pl.ref_count + e, 1);
    }
  flag(p.status, flags);
}

// ---- compact ----------------------------------------------------------

// One CTA.  ws[page]: for a live page at or behind n, its rank among them.
__global__ void __launch_bounds__(kOne) compact_kernel(const __grid_constant__ PoolParams p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ int scratch[33];
  const kvq_page_pool& pl = p.pool;
  const int N = pl.num_pages, half = N / 2;
  int n = 0;
  {
    int mine = 0, sum;
    for (int i = 4 * threadIdx.x; i < N; i += 4 * kOne) {
      int free4, live4;
      states4(pl, i, &free4, &live4);
      mine += __popc(live4);
    }
    block_scan(mine, scratch, &sum);
    n = sum;
  }
  int movers = 0, holes = 0;
  for (int i0 = 0; i0 < N; i0 += 4 * kOne) {
    const int i = i0 + 4 * threadIdx.x;
    int free4 = 0, live4 = 0, sum;
    if (i < N) states4(pl, i, &free4, &live4);
    const int exist = i >= N ? 0 : i + 4 <= N ? 15 : (1 << (N - i)) - 1;
    const int before = n <= i ? 0 : n >= i + 4 ? 15 : (1 << (n - i)) - 1;  // of them, in front of the border
    const int mover = live4 & ~before, hole = exist & before & ~live4;
    const int ex = block_scan(__popc(mover) | (__popc(hole) << 16), scratch, &sum);
    int km = movers + (ex & 0xffff), kh = holes + (ex >> 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (mover >> e & 1) {
        p.copy_src[km] = i + e;
        p.ws[i + e] = km++;
      }
      if (hole >> e & 1) p.copy_dst[kh++] = i + e;
    }
    movers += sum & 0xffff;
    holes += sum >> 16;
  }
  for (int k = movers + threadIdx.x; k < half; k += kOne) p.copy_src[k] = p.copy_dst[k] = -1;
  if (threadIdx.x == 0) *p.num_live = n;
  __syncthreads();
  uint32_t flags = 0;
  const long long entries = (long long)pl.batch * pl.max_blocks_per_seq;
  for (long long i = threadIdx.x; i < entries; i += kOne) {
    const int e = pl.block_table[i];
    if (e < 0) continue;
    if (e >= N || pl.ref_count[e] <= 0) {
      pl.block_table[i] = -1;
      flags |= KVQ_FLAG_BLOCK_TABLE;
    } else if (e >= n) {
      pl.block_table[i] = p.copy_dst[p.ws[e]];
    }
  }
  __syncthreads();
  for (int k = threadIdx.x; k < movers; k += kOne) {
    const int s = p.copy_src[k], d = p.copy_dst[k];
    pl.ref_count[d] = pl.ref_count[s];
    pl.ref_count[s] = 0;
  }
  flag(p.status, flags);
}

// ---- copy -------------------------------------------------------------

// Grid: x = pairs, y = layers.
constexpr int kCopyThreads = 128, kCopyLoads = 8;
constexpr int kListInline = 2048;  // pairs up to which the copying CTAs check the list
__device__ __forceinline__ bool copied(const PageCopyParams& p, int s, int d) {
  return s >= 0 && d >= 0 && s < p.num_pages && d < p.num_pages;
}
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ PageCopyParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int i = blockIdx.x, layer = blockIdx.y;
  const int s = __ldg(p.src + i), d = __ldg(p.dst + i);
  if (s < 0 || d < 0) return;
  const bool report = p.report && layer == 0;
  if (s >= p.num_pages || d >= p.num_pages) {
    if (report && threadIdx.x == 0) flag(p.status, KVQ_FLAG_BLOCK_TABLE);
    return;
  }
  // the arrays' pieces of 16 bytes in one row, eight loads of a thread in flight
  uint32_t ends[6], total = 0;
#pragma unroll
  for (int a = 0; a < 6; ++a) ends[a] = total += p.bytes[a] / 16;
  for (uint32_t k0 = threadIdx.x; k0 < total; k0 += kCopyThreads * kCopyLoads) {
    uint4 v[kCopyLoads];
    uint4* to[kCopyLoads];
#pragma unroll
    for (int u = 0; u < kCopyLoads; ++u) {
      const uint32_t k = k0 + u * kCopyThreads;
      to[u] = nullptr;
      if (k >= total) continue;
      uint8_t* base = p.base[layer][0];
      uint32_t bytes = p.bytes[0], first = 0;
#pragma unroll
      for (int a = 1; a < 6; ++a)
        if (k >= ends[a - 1]) base = p.base[layer][a], bytes = p.bytes[a], first = ends[a - 1];
      v[u] = *(reinterpret_cast<const uint4*>(base + (size_t)s * bytes) + (k - first));
      to[u] = reinterpret_cast<uint4*>(base + (size_t)d * bytes) + (k - first);
    }
#pragma unroll
    for (int u = 0; u < kCopyLoads; ++u)
      if (to[u]) *to[u] = v[u];
  }
  if (report && p.num_pairs <= kListInline) {
    uint32_t flags = d == s ? KVQ_FLAG_PAGE_LIST : 0u;
    for (int j = threadIdx.x; j < p.num_pairs; j += blockDim.x) {
      if (j == i) continue;
      const int sj = __ldg(p.src + j), dj = __ldg(p.dst + j);
      if (copied(p, sj, dj) && (sj == d || dj == d)) flags = KVQ_FLAG_PAGE_LIST;
    }
    flag(p.status, flags);
  }
}

// The same check of a long list: a CTA per kListPages pages marks the targets
// among them in a bitmap, then looks the sources up.  Sixteen pairs a thread
// in flight: 500 000 pairs 90 us (each pair against every other, as in a
// short list: 132 ms with 200 000 of them to copy).
constexpr int kListThreads = 1024, kListPages = 1 << 20, kListLoads = 4;
__global__ void __launch_bounds__(kListThreads) list_kernel(const __grid_constant__ PageCopyParams p) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ uint32_t targets[];  // a bit per page
  const int first = blockIdx.x * kListPages;
  const uint32_t pairs = (uint32_t)p.num_pairs;
  for (int i = threadIdx.x; i < kListPages / 32; i += kListThreads) targets[i] = 0;
  __syncthreads();
  bool bad = false;
  for (int look = 0; look < 2; ++look) {
    for (uint32_t k0 = 4 * threadIdx.x; k0 < pairs; k0 += 4 * kListThreads * kListLoads) {
      int4 s[kListLoads], d[kListLoads];
#pragma unroll
      for (int u = 0; u < kListLoads; ++u) {
        const uint32_t k = k0 + 4 * kListThreads * u;
        s[u] = d[u] = make_int4(-1, -1, -1, -1);
        if (k + 4 <= pairs) {
          s[u] = __ldg(reinterpret_cast<const int4*>(p.src + k));
          d[u] = __ldg(reinterpret_cast<const int4*>(p.dst + k));
        } else {
          if (k < pairs) s[u].x = __ldg(p.src + k), d[u].x = __ldg(p.dst + k);
          if (k + 1 < pairs) s[u].y = __ldg(p.src + k + 1), d[u].y = __ldg(p.dst + k + 1);
          if (k + 2 < pairs) s[u].z = __ldg(p.src + k + 2), d[u].z = __ldg(p.dst + k + 2);
        }
      }
#pragma unroll
      for (int u = 0; u < kListLoads; ++u) {
        const int sv[4] = {s[u].x, s[u].y, s[u].z, s[u].w}, dv[4] = {d[u].x, d[u].y, d[u].z, d[u].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!copied(p, sv[e], dv[e])) continue;
          const uint32_t at = (uint32_t)((look ? sv[e] : dv[e]) - first);
          if (at >= (uint32_t)kListPages) continue;  // another CTA's page
          const uint32_t bit = 1u << (at & 31);
          bad |= ((look ? targets[at >> 5] : atomicOr(&targets[at >> 5], bit)) & bit) != 0;
        }
      }
    }
    __syncthreads();
  }
  if (__syncthreads_or(bad) && threadIdx.x == 0) flag(p.status, KVQ_FLAG_PAGE_LIST);
}

}  // namespace

// launch_pdl for a kernel with one more integer
static cudaError_t launch_int(void (*kernel)(PoolParams, int), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                              const PoolParams& p, int x) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, x);
}

cudaError_t launch_pages_reorder(const PoolParams& p, cudaStream_t stream) {
  // A CTA holds its columns of every row: as many as fit 128 KB, at most 32,
  // and down to 4 (half a sector a row) while there are fewer CTAs than SMs
  // (256 rows of 190 blocks: 43 us with 32 columns a CTA and 256 threads).
  int cols = 32;
  while (cols > 1 && ((size_t)p.pool.batch * cols * 4 > 128 * 1024 ||
                      (cols > 4 && p.pool.max_blocks_per_seq < 152 * cols)))
    cols >>= 1;
  const size_t smem = (size_t)p.pool.batch * cols * 4;
  cudaError_t e = cudaFuncSetAttribute(reorder_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       128 * 1024);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)((p.pool.max_blocks_per_seq + cols - 1) / cols);
  return launch_int(reorder_kernel, dim3(grid), dim3(1024), smem, stream, p, cols);
}

cudaError_t launch_pages_reserve(const PoolParams& p, cudaStream_t stream) {
  const size_t smem = (size_t)p.pool.batch * 8;
  cudaError_t e = cudaFuncSetAttribute(reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       KVQ_MAX_POOL_BATCH * 8);
  if (e != cudaSuccess) return e;
  int lps = 4;
  while (lps < 32 && lps - 2 < p.num_new / p.pool.page_size) lps *= 2;
  return launch_int(reserve_kernel, dim3(1), dim3(kOne), smem, stream, p, lps);
}

cudaError_t launch_pages_compact(const PoolParams& p, cudaStream_t stream) {
  return launch_pdl(compact_kernel, dim3(1), dim3(kOne), 0, stream, p);
}

cudaError_t launch_pages_copy(const PageCopyParams& p, cudaStream_t stream) {
  cudaError_t e = launch_pdl(copy_kernel, dim3(p.num_pairs, p.layers), dim3(kCopyThreads), 0, stream, p);
  if (e != cudaSuccess || !p.report || p.num_pairs <= kListInline) return e;
  e = cudaFuncSetAttribute(list_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kListPages / 8);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)(((long long)p.num_pages + kListPages - 1) / kListPages);
  return launch_pdl(list_kernel, dim3(grid), dim3(kListThreads), kListPages / 8, stream, p);
}

}  // namespace kvq
