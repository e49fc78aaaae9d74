// Causal attention of several new tokens per sequence over the cache
// (kvq_extend_attn), and the merge of its split partials.
//
// Rows.  The G query heads of a KV head and the new tokens share K and V, so
// a tile's rows are (token, head) pairs, row r = token r / G, head r % G;
// row r attends to positions up to seq_lens_before + r / G.
//
// One pass over the keys with a running maximum and sum per row, in log2
// units: m' = max(m, max_j s_j), l' = 2^(m - m') l + sum_j 2^(s_j - m'),
// o' = 2^(m - m') o + sum_j 2^(s_j - m') v_j; splits over the context write
// (m, l, o) and a merge joins them.
//
// The kernel here, on mma.sync, takes what the tensor-core kernel of
// kvq_extend_tc.cuh does not: head_dim 256 and axis-aware caches.  As there, K
// and V enter as hi + lo, and the probabilities, rounded to fp16, carry a
// factor (2^14: m is the exact maximum here) that keeps small ones in fp16's
// normal range.  Bound by the conversion of a tile before its products, which
// nothing overlaps: it is the form that is right for every cache, kept for the
// shapes that the tensor-core kernel is not written for: D = 256 (the O of its
// two tiles of rows alone would fill tensor memory; one tile would fit, 448 of
// 512 columns) and keys that have a scale per channel.
#include "kvq_extend_tc.cuh"
#include "kvq_host.cuh"
#include "kvq_load.cuh"
#include "kvq_rope.cuh"

namespace kvq {
namespace {

using fast::ex2;
using fast::ldsm_x4;
using fast::ldsm_x4_t;
using fast::mma16816;
using fast::smem_u32;

constexpr int kRows = 64;  // 4 warps of 16 rows
constexpr int kThreads = 128;
constexpr float kLift = 14.f;  // log2 of the factor in the probabilities, l and o

// Keys per tile: K and V rows, hi and lo, as fp16 in shared memory
__host__ __device__ constexpr int tile_keys(int D) { return D == 256 ? 32 : 64; }
__host__ __device__ constexpr size_t extend_smem(int D) {
  return (size_t)(kRows + 4 * tile_keys(D)) * D * 2 + 3 * tile_keys(D) * sizeof(int);
}

// Byte offset of 16-byte chunk c of row r in a [rows][D] fp16 tile; the
// chunk index is XORed with the row so that ldmatrix's 8 rows fall into
// different banks.
template <int D>
__device__ __forceinline__ uint32_t at(int r, int c) {
  return (uint32_t)(r * (2 * D) + ((c ^ (r & 7)) << 4));
}

// One sequence's share of the call: its rows and lengths.
struct Span {
  int before, n, L;
};
__device__ __forceinline__ Span span_of(const ExtendParams& p, int b, bool report) {
  Span s;
  s.before = checked_len(p.v.geom, p.lens_before, b, -1);
  s.n = new_rows_of(p.new_lens, b, p.num_new);
  const long long L = (long long)s.before + s.n;
  const bool bad = s.before < 0 || s.n < 0 || L > p.len_limit;
  if (bad && report && p.status) atomicOr(p.status, KVQ_FLAG_SEQ_LEN);
  s.L = bad ? 0 : (int)L;  // no keys: the rows come out zero
  s.n = max(s.n, 0);
  return s;
}

template <int BITS, int D>
__global__ void __launch_bounds__(kThreads) extend_kernel(const __grid_constant__ ExtendParams p) {
  constexpr int KEYS = tile_keys(D), CH = D / 8, KB = D / 16, NT = KEYS / 8;
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ __align__(128) uint8_t smem[];
  const CacheGeom& c = p.v.geom;
  const int kvh = blockIdx.y, b = blockIdx.z;
  const int split = blockIdx.x % p.splits, tile = blockIdx.x / p.splits;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Span sp = span_of(p, b, threadIdx.x == 0 && blockIdx.x == 0 && kvh == 0);
  const long long r0 = (long long)tile * kRows;
  const long long live_rows = (long long)sp.n * p.G;
  if (r0 >= live_rows) return;

  const uint32_t q_s = smem_u32(smem), k_s = q_s + kRows * D * 2, v_s = k_s + 2 * KEYS * D * 2;
  int* ok_s = reinterpret_cast<int*>(smem + (kRows + 4 * KEYS) * D * 2);
  int* bad_s = ok_s + KEYS;  // [2][KEYS], the tiles in turn: V held an infinity or NaN (set to zero)
  for (int i = threadIdx.x; i < 2 * KEYS; i += kThreads) bad_s[i] = 0;

  // q rows of the tile (zero behind the last)
  for (int i = threadIdx.x; i < kRows * CH; i += kThreads) {
    const int r = i / CH, ch = i % CH;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (r0 + r < live_rows) {
      const int t = (int)((r0 + r) / p.G), h = (int)((r0 + r) % p.G);
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + (((long long)b * p.num_new + t) * p.Hq + (long long)kvh * p.G + h) * D) + ch;
      if (KVQ_IN(c, KVQ_ARRAY_Q, src, 16)) x = *src;
    }
    *reinterpret_cast<uint4*>(smem + at<D>(r, ch)) = x;
  }

  // the tile's last row sees positions below `end`
  const int all_see = sp.L ? sp.before + (int)(r0 / p.G) : -1;  // every row sees the positions up to here
  const int t_last = (int)((min(r0 + kRows, live_rows) - 1) / p.G);
  const int end = sp.L ? min(sp.L, sp.before + t_last + 1) : 0;
  const int k0 = split * p.chunk, k1 = min(end, k0 + p.chunk);

  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  // this lane's two rows: last position seen
  int last[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const long long r = r0 + warp * 16 + (lane >> 2) + 8 * e;
    last[e] = r < live_rows ? sp.before + (int)(r / p.G) : -1;
  }

  int turn = 0;
  for (int ks = k0; ks < k1; ks += KEYS, turn ^= 1) {
    __syncthreads();  // the tile before is used up (and q is in place)
    for (int i = threadIdx.x; i < KEYS * CH; i += kThreads) {
      const int j = i / CH, ch = i % CH, pos = ks + j;
      uint4 kx = make_uint4(0u, 0u, 0u, 0u), kl = kx, vx = kx, vl = kx;
      bool ok = pos < k1;
      if (ok) {
        const long long row = view_row(c, b, kvh, sp.L, pos);
        if (row < 0) {
          ok = false;
          if (ch == 0 && p.status) atomicOr(p.status, KVQ_FLAG_BLOCK_TABLE);
        } else {
          kx = load8<BITS>(p.v, 0, b, kvh, sp.L, pos, row, ch, &kl);
          vx = load8<BITS>(p.v, 1, b, kvh, sp.L, pos, row, ch, &vl);
          // In a tile that some row sees in part an infinite or NaN V must
          // not meet the zero weights of the rows that do not see it.
          if (ks + KEYS - 1 > all_see && (ext::nonfinite2(vx.x) || ext::nonfinite2(vx.y) || ext::nonfinite2(vx.z) ||
                                          ext::nonfinite2(vx.w))) {
            vx = make_uint4(0u, 0u, 0u, 0u);
            bad_s[turn * KEYS + j] = 1;
          }
        }
      }
      *reinterpret_cast<uint4*>(smem + kRows * D * 2 + at<D>(j, ch)) = kx;
      if (BITS != 16) {
        *reinterpret_cast<uint4*>(smem + (kRows + KEYS) * D * 2 + at<D>(j, ch)) = kl;
        *reinterpret_cast<uint4*>(smem + (kRows + 3 * KEYS) * D * 2 + at<D>(j, ch)) = vl;
      }
      *reinterpret_cast<uint4*>(smem + (kRows + 2 * KEYS) * D * 2 + at<D>(j, ch)) = vx;
      if (ch == 0) ok_s[j] = ok;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < KEYS; i += kThreads) bad_s[(turn ^ 1) * KEYS + i] = 0;

    float s[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      uint32_t a[4];
      ldsm_x4(q_s + at<D>(warp * 16 + (lane & 15), kb * 2 + (lane >> 4)), a[0], a[1], a[2], a[3]);
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
#pragma unroll
        for (int part = 0; part < (BITS == 16 ? 1 : 2); ++part) {  // hi, lo
          uint32_t b0, b1, b2, b3;  // keys n*8 .. n*8+15, channels 16 kb .. +15
          ldsm_x4(k_s + part * KEYS * D * 2 + at<D>(n * 8 + (lane & 7) + ((lane >> 4) << 3), kb * 2 + ((lane >> 3) & 1)),
                  b0, b1, b2, b3);
          mma16816(s[n], a[0], a[1], a[2], a[3], b0, b1);
          mma16816(s[n + 1], a[0], a[1], a[2], a[3], b2, b3);
        }
      }
    }

    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = n * 8 + (lane & 3) * 2 + (e & 1);
        const bool see = ok_s[j] && ks + j <= last[e >> 1];
        s[n][e] = !see ? -INFINITY : bad_s[turn * KEYS + j] ? __int_as_float(0x7FFFFFFF) : s[n][e] * p.scale_log2;
        mx[e >> 1] = fmaxf(mx[e >> 1], s[n][e]);
      }
    }
    float alpha[2], base[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
      const float mn = fmaxf(m[e], mx[e]);
      base[e] = mn == -INFINITY ? 0.f : mn - kLift;  // nothing seen yet: every weight is 2^-inf = 0
      alpha[e] = mn == -INFINITY ? 0.f : ex2(m[e] - mn);
      m[e] = mn;
      l[e] *= alpha[e];
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = ex2(s[n][e] - base[e >> 1]);
        l[e >> 1] += s[n][e];
      }
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      o[i][0] *= alpha[0];
      o[i][1] *= alpha[0];
      o[i][2] *= alpha[1];
      o[i][3] *= alpha[1];
    }
#pragma unroll
    for (int kb = 0; kb < KEYS / 16; ++kb) {
      const uint32_t a0 = fast::pack_h2(s[2 * kb][0], s[2 * kb][1]);
      const uint32_t a1 = fast::pack_h2(s[2 * kb][2], s[2 * kb][3]);
      const uint32_t a2 = fast::pack_h2(s[2 * kb + 1][0], s[2 * kb + 1][1]);
      const uint32_t a3 = fast::pack_h2(s[2 * kb + 1][2], s[2 * kb + 1][3]);
#pragma unroll
      for (int n = 0; n < D / 8; n += 2) {
#pragma unroll
        for (int part = 0; part < (BITS == 16 ? 1 : 2); ++part) {  // hi, lo
          uint32_t b0, b1, b2, b3;  // keys 16 kb .. +15, channels n*8 .. +15
          ldsm_x4_t(v_s + part * KEYS * D * 2 + at<D>(kb * 16 + (lane & 15), n + (lane >> 4)), b0, b1, b2, b3);
          mma16816(o[n], a0, a1, a2, a3, b0, b1);
          mma16816(o[n + 1], a0, a1, a2, a3, b2, b3);
        }
      }
    }
  }

#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    const long long r = r0 + warp * 16 + (lane >> 2) + 8 * e;
    if (r >= live_rows) continue;
    const int t = (int)(r / p.G), h = (int)(r % p.G);
    const long long orow = ((long long)b * p.num_new + t) * p.Hq + (long long)kvh * p.G + h;
    if (p.splits == 1) {
      const float inv = l[e] != 0.f ? 1.f / l[e] : 0.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        __half2* d = reinterpret_cast<__half2*>(p.out + orow * D + i * 8 + (lane & 3) * 2);
        if (KVQ_IN(c, KVQ_ARRAY_OUT, d, 4)) *d = __floats2half2_rn(o[i][2 * e] * inv, o[i][2 * e + 1] * inv);
      }
    } else {
      const long long w = orow * p.splits + split;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        float2* d = reinterpret_cast<float2*>(p.ws_o + w * D + i * 8 + (lane & 3) * 2);
        if (KVQ_IN(c, KVQ_ARRAY_WORKSPACE, d, 8)) *d = make_float2(o[i][2 * e], o[i][2 * e + 1]);
      }
      float2* ml = reinterpret_cast<float2*>(p.ws_ml) + w;
      if ((lane & 3) == 0 && KVQ_IN(c, KVQ_ARRAY_WORKSPACE, ml, 8)) *ml = make_float2(m[e], l[e]);
    }
  }
}

// out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s of each live row
// (sequence, new token, head): D / 4 threads a row, four channels each, the
// partials of kMergeSplits splits in flight.  Bound by memory once rows are
// many (a CTA of D threads per row took 135 us for 131072 rows of two splits,
// 134 MB).
constexpr int kMergeSplits = 4;
__global__ void __launch_bounds__(256) extend_merge_kernel(const __grid_constant__ ExtendParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const CacheGeom& c = p.v.geom;
  const int per = c.D / 4;  // 16, 32 or 64
  const long long row = (long long)blockIdx.x * (256 / per) + threadIdx.x / per;
  if (row >= (long long)p.batch * p.num_new * p.Hq) return;
  const long long tok = row / p.Hq;
  const int b = (int)(tok / p.num_new), t = (int)(tok - (long long)b * p.num_new);
  if (t >= new_rows_of(p.new_lens, b, p.num_new)) return;
  const int D = c.D, d = threadIdx.x % per * 4;
  const float2* ml = reinterpret_cast<const float2*>(p.ws_ml) + row * p.splits;
  const float* o = p.ws_o + row * p.splits * D + d;
  float M = -INFINITY, den = 0.f;
  float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < p.splits; s0 += kMergeSplits) {
    float2 v[kMergeSplits];
    float4 x[kMergeSplits];
    float Mn = M;
#pragma unroll
    for (int u = 0; u < kMergeSplits; ++u) {
      const int s = s0 + u;
      v[u] = make_float2(-INFINITY, 0.f);
      x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s < p.splits && KVQ_IN(c, KVQ_ARRAY_WORKSPACE, ml + s, 8) &&
          KVQ_IN(c, KVQ_ARRAY_WORKSPACE, o + (long long)s * D, 16)) {
        v[u] = ml[s];
        x[u] = *reinterpret_cast<const float4*>(o + (long long)s * D);
      }
      Mn = fmaxf(Mn, v[u].x);
    }
    const float base = Mn == -INFINITY ? 0.f : Mn, a = ex2(M - base);
    num = make_float4(num.x * a, num.y * a, num.z * a, num.w * a);
    den *= a;
#pragma unroll
    for (int u = 0; u < kMergeSplits; ++u) {
      if (v[u].x == -INFINITY && v[u].y == 0.f) continue;  // nothing seen there
      const float f = ex2(v[u].x - base);
      num.x = fmaf(f, x[u].x, num.x);
      num.y = fmaf(f, x[u].y, num.y);
      num.z = fmaf(f, x[u].z, num.z);
      num.w = fmaf(f, x[u].w, num.w);
      den = fmaf(f, v[u].y, den);
    }
    M = Mn;
  }
  const float inv = den != 0.f ? 1.f / den : 0.f;
  uint2* to = reinterpret_cast<uint2*>(p.out + row * D + d);
  if (KVQ_IN(c, KVQ_ARRAY_OUT, to, 8))
    *to = make_uint2(fast::pack_h2(num.x * inv, num.y * inv), fast::pack_h2(num.z * inv, num.w * inv));
}

template <int BITS, int D>
cudaError_t run(const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream) {
  static KernelSetup setup;
  int occ = 0;
  cudaError_t e = setup_kernel(extend_kernel<BITS, D>, setup, kThreads, extend_smem(D), &occ);
  if (e != cudaSuccess) return e;
  if (plan) {
    plan->tile_rows = kRows;
    plan->occ = occ;
    return cudaSuccess;
  }
  const long long tiles = ((long long)p->num_new * p->G + kRows - 1) / kRows;
  const dim3 grid((unsigned)(tiles * p->splits), p->v.geom.Hkv, p->batch);
  return launch_pdl(extend_kernel<BITS, D>, grid, dim3(kThreads), extend_smem(D), stream, *p);
}

// Axis-aware caches are INT4 or INT8; of the other formats only head_dim 256
// comes here.
template <int BITS>
cudaError_t run_d(int D, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream) {
  if constexpr (BITS == 4 || BITS == 8) {
    if (D == 64) return run<BITS, 64>(p, plan, stream);
    if (D == 128) return run<BITS, 128>(p, plan, stream);
  }
  return D == 256 ? run<BITS, 256>(p, plan, stream) : cudaErrorInvalidValue;
}

cudaError_t run_any(const CacheGeom& c, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream) {
  switch (c.bits) {
    case 2: return run_d<2>(c.D, p, plan, stream);
    case 4: return run_d<4>(c.D, p, plan, stream);
    case 8: return run_d<8>(c.D, p, plan, stream);
    default: return run_d<16>(c.D, p, plan, stream);
  }
}

}  // namespace

// The tensor-core kernel takes every per-token format at head_dim 64 and 128.
static bool takes_tc(const CacheGeom& c) {
  return !c.kch && (c.D == 64 || c.D == 128) && (!c.nf4 || nf4_table().symmetric);
}

static cudaError_t run_tc_any(const CacheGeom& c, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t s) {
  if (c.nf4) return run_extend_tc_nf4(c.D, nq, p, plan, s);
  switch (c.bits) {
    case 2: return run_extend_tc_int2(c.D, nq, p, plan, s);
    case 4: return run_extend_tc_int4(c.D, nq, p, plan, s);
    case 8: return run_extend_tc_int8(c.D, nq, p, plan, s);
    default: return run_extend_tc_fp16(c.D, nq, p, plan, s);
  }
}

cudaError_t extend_plan(const CacheGeom& c, int num_new, int G, ExtendPlan* plan) {
  plan->kind = !takes_tc(c) ? 0 : (long long)num_new * G <= 128 ? 1 : 2;
  if (plan->kind == 0) return run_any(c, nullptr, plan, nullptr);
  return run_tc_any(c, plan->kind, nullptr, plan, nullptr);
}

cudaError_t launch_extend(const ExtendParams& p, const ExtendPlan& plan, cudaStream_t stream) {
  cudaError_t e = plan.kind == 0 ? run_any(p.v.geom, &p, nullptr, stream)
                                 : run_tc_any(p.v.geom, plan.kind, &p, nullptr, stream);
  if (e == cudaSuccess && p.splits > 1) {
    const long long rows = (long long)p.batch * p.num_new * p.Hq;
    const int per = 256 / (p.v.geom.D / 4);
    e = launch_pdl(extend_merge_kernel, dim3((unsigned)((rows + per - 1) / per)), dim3(256), 0, stream, p);
  }
  return e;
}

}  // namespace kvq
