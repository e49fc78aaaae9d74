// Attention of several new tokens over the cache on the fifth-generation
// tensor cores (head_dim 64 and 128, every per-token format).
//
// Rows.  As in kvq_extend.cu the rows of a tile are (new token, head of the
// KV head's group) pairs.  A CTA takes NQ tiles of 128 rows of one KV head
// and one split of the keys, in steps of 64 keys:
//   S = Q K^T     A = Q, resident in tensor memory for the whole call; B = K
//                 from shared memory
//   P = 2^(S - m) one thread per row: 64 scores from tensor memory to
//                 registers, the probabilities back as fp16 in S's place
//   O += P V      A = P in tensor memory; B = V, whose rows are keys, read
//                 MN-major so that nothing is transposed
// With A in tensor memory the tensor core fetches 64 (QK) or 2 head_dim
// bytes a cycle from shared memory, half its bandwidth or less; with Q in
// shared memory a 64-key step would be bound by fetching Q again.
//
// Warps.  0-3 (and 4-7 with two tiles): softmax, a row per thread.  Then the
// producers, which read the codes, turn them into fp16 and store them in the
// tensor core's swizzled layout (four warps, or eight with one tile).  The
// last warp issues the MMAs.  With two tiles one's softmax runs under the
// other's products.
//
// Precision.  q - z is a whole number (exact in fp16 up to 2048) and s has
// 11 bits, so x_hat = (q - z) s has up to 23: K enters as the sum of two fp16
// numbers, hi = fp16(x_hat) and lo = fp16(x_hat - hi), two products into one
// accumulator.  With hi alone the scores of keys with large channels are off
// by 4e-4 (rms, INT4 groups of 32 with 10x channels) and the outputs by 1e-3,
// five times what rounding the output costs; with both by 3e-4, which the
// fp16 rounding of V and of the probabilities and the output's own rounding
// share.  V enters as hi alone: its errors average out over the keys.  Scores,
// sums and O are fp32.  fp16 caches are exact as they are.
//
// Reference maximum.  m moves only when a tile's maximum exceeds it by 2^8
// (P is at most 256 then), so O in tensor memory is rescaled rarely.
//
// Order of the MMAs.  One thread issues PV(j) and then QK(j + 1) of a tile,
// and MMAs run in the order issued: S may be overwritten as soon as QK(j + 1)
// is issued, and when its completion is seen PV(j) is complete too, so the
// softmax may rescale O until it hands over P(j + 1).
#pragma once

#include "kvq_decode_fast.cuh"
#include "kvq_load.cuh"
#include "kvq_rope.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace ext {

using fast::ex2;

constexpr int kKeys = 64;
constexpr float kLazy = 8.f;  // log2 units the maximum may lead the reference

// KIND: 0 uniform codes (asymmetric or symmetric), 1 NF4, 2 fp16
template <int BITS, int KIND, int D, int NQ>
struct Cfg {
  static constexpr bool LO = KIND != 2;
  static constexpr int SOFT = 4 * NQ;             // softmax warps
  static constexpr int PROD = NQ == 1 ? 8 : 4;    // producer warps
  static constexpr int WARPS = SOFT + PROD + 1;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int MAT = kKeys * D * 2;       // one fp16 tile
  static constexpr int STAGE = (LO ? 3 : 2) * MAT;
  static constexpr int STAGES = D == 128 ? 4 : 6;
  static constexpr int SEGS = D / 32;             // 32-channel segments of a row
  static constexpr int UNITS = 2 * SEGS * kKeys / (PROD * 32);  // segments per producer thread and tile
  // tensor memory columns: per tile S (64, P in its place), O (D), Q (D / 2)
  static constexpr uint32_t COL_S = 0, COL_O = NQ * kKeys, COL_Q = COL_O + NQ * D;
  static constexpr uint32_t COLS = NQ == 2 ? 512 : 256;
  static constexpr size_t SMEM = (size_t)STAGES * STAGE + 1024 + 512;
  static_assert(COL_Q + NQ * D / 2 <= COLS, "tensor memory");
  // channel held at place i of an eight-channel chunk (the unpacking leaves
  // 4-bit and 2-bit codes as pairs (i, i + 4))
  static constexpr bool PAIRED = BITS <= 4;
  __host__ __device__ static constexpr int channel(int i) { return PAIRED ? (i >> 1) + 4 * (i & 1) : i; }
};

// Barriers and flags behind the stages
template <int STAGES>
struct Shared {
  unsigned long long full[STAGES], empty[STAGES];
  unsigned long long q_full[2], s_full[2], p_full[2], o_full[2];
  uint32_t ok[STAGES][2];   // per key: mapped and before the end
  uint32_t bad[STAGES][4][2];  // per segment and key: V held an infinity or NaN (set to zero)
  uint32_t tmem;
  int stop;
};

// ---- producers --------------------------------------------------------

// The codes and headers of 32 channels of one key, as loaded.
template <int BITS>
struct Seg {
  uint32_t w[BITS == 16 ? 1 : BITS];  // 32 * BITS / 32 words
  uint32_t s[2], z[2];                // up to four fp16 scales and zeros
};

template <int BITS, int KIND>
__device__ __forceinline__ void load_seg(const ExtendParams& p, int which, long long row, int seg,
                                         Seg<BITS>& x) {
  const CacheGeom& c = p.v.geom;
#pragma unroll
  for (int i = 0; i < BITS; ++i) x.w[i] = 0;
  x.s[0] = x.s[1] = x.z[0] = x.z[1] = 0;
  if (row < 0) return;
  const uint8_t* src = p.v.codes[which] + row * c.row_bytes + seg * 4 * BITS;
  const int a_codes = which ? KVQ_ARRAY_V_CODES : KVQ_ARRAY_K_CODES;
  if (KVQ_IN(c, a_codes, src, 4 * BITS)) {
    if constexpr (BITS == 2) {
      const uint2 t = __ldg(reinterpret_cast<const uint2*>(src));
      x.w[0] = t.x, x.w[1] = t.y;
    } else {
#pragma unroll
      for (int i = 0; i < BITS / 4; ++i) {
        const uint4 t = __ldg(reinterpret_cast<const uint4*>(src) + i);
        x.w[4 * i] = t.x, x.w[4 * i + 1] = t.y, x.w[4 * i + 2] = t.z, x.w[4 * i + 3] = t.w;
      }
    }
  }
  const int n = c.g >= 32 ? 1 : 32 / c.g;  // groups in the segment: 1, 2 or 4
  const long long h = row * c.ngroups + seg * 32 / c.g;
  const int a_scale = which ? KVQ_ARRAY_V_SCALE : KVQ_ARRAY_K_SCALE;
  const int a_zero = which ? KVQ_ARRAY_V_ZERO : KVQ_ARRAY_K_ZERO;
  const __half* sp = p.v.scale[which] + h;
  if (KVQ_IN(c, a_scale, sp, 2 * n)) {
    if (n == 1) x.s[0] = __ldg(reinterpret_cast<const unsigned short*>(sp));
    else if (n == 2) x.s[0] = __ldg(reinterpret_cast<const uint32_t*>(sp));
    else {
      const uint2 t = __ldg(reinterpret_cast<const uint2*>(sp));
      x.s[0] = t.x, x.s[1] = t.y;
    }
  }
  if (KIND == 0 && !c.sym) {
    const __half* zp = p.v.zero[which] + h;
    if (KVQ_IN(c, a_zero, zp, 2 * n)) {
      if (n == 1) x.z[0] = __ldg(reinterpret_cast<const unsigned short*>(zp));
      else if (n == 2) x.z[0] = __ldg(reinterpret_cast<const uint32_t*>(zp));
      else {
        const uint2 t = __ldg(reinterpret_cast<const uint2*>(zp));
        x.z[0] = t.x, x.z[1] = t.y;
      }
    }
  }
}

__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// The eight codes of chunk ch of a segment as fp16 1024 + q (NF4: as levels)
template <int BITS, int KIND>
__device__ __forceinline__ void biased8(const Seg<BITS>& x, int ch, const uint32_t (&lut)[4], uint32_t (&o)[4]) {
  if constexpr (KIND == 1) {
    fast::nib8_to_h2_nf4(x.w[ch], o, lut);
  } else if constexpr (BITS == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = fast::and_or(x.w[ch] >> (4 * i), 0x000F000Fu, fast::kH1024);
  } else if constexpr (BITS == 2) {
    const uint32_t w = (x.w[ch >> 1] >> (16 * (ch & 1))) & 0xFFFFu;
    const uint32_t v = (w & 0xFFu) | ((w & 0xFF00u) << 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = fast::and_or(v >> (2 * i), 0x00030003u, fast::kH1024);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = fast::prmt_b32(x.w[2 * ch + (i >> 1)], 0x64646464u, (i & 1) ? 0x4342u : 0x4140u);
  }
}

// One segment to fp16 (hi, and lo for K) at its places in the tile:
// blocks of 64 channels, [key][128 bytes], chunks XORed with the key.
template <int BITS, int KIND, int D>
__device__ __forceinline__ void store_seg(const ExtendParams& p, const Seg<BITS>& x, bool is_k, int key, int seg,
                                          uint8_t* hi, uint8_t* lo, const uint32_t (&lut)[4]) {
  const CacheGeom& c = p.v.geom;
  const uint32_t base = (uint32_t)((seg >> 1) * (kKeys * 128) + key * 128);
  const int per = c.g >= 32 ? 4 : c.g / 8;  // chunks per group
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) {
    const int grp = ch / per;
    const uint32_t sw = (grp & 2 ? x.s[1] : x.s[0]) >> (16 * (grp & 1));
    const __half s = __ushort_as_half((unsigned short)(sw & 0xFFFFu));
    __half z = __ushort_as_half(0);
    uint32_t b[4], h[4], l[4];
    biased8<BITS, KIND>(x, ch, lut, b);
    const __half2 s2 = __half2half2(s);
    bool plain = true;  // no product beyond fp16, and 1024 + z a whole number that fp16 holds
    __half2 off = __half2half2(z);
    if constexpr (KIND == 0) {
      const uint32_t zw = (grp & 2 ? x.z[1] : x.z[0]) >> (16 * (grp & 1));
      z = c.sym ? __int2half_rn(1 << (BITS - 1)) : __ushort_as_half((unsigned short)(zw & 0xFFFFu));
      const float zf = __half2float(z), sf = __half2float(s);
      plain = fabsf(zf) <= 1024.f && sf * (fabsf(zf) + (float)((1 << BITS) - 1)) < 65504.f;
      off = __half2half2(__float2half_rn(-1024.f - zf));
    }
    if (plain) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 d = KIND == 1 ? as_h2(b[i]) : __hadd2(as_h2(b[i]), off);
        const __half2 v = __hmul2_rn(d, s2);
        h[i] = as_u32(v);
        l[i] = as_u32(__hfma2(d, s2, __hneg2(v)));  // the product is exact in the fma: what hi left
      }
    } else {  // far zero-points and scales near fp16's end, in fp32
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 q = __half22float2(__hsub2(as_h2(b[i]), as_h2(fast::kH1024)));
        const float zf = __half2float(z), sf = __half2float(s);
        const float a = (q.x - zf) * sf, e = (q.y - zf) * sf;
        h[i] = pack_sat(a, e);
        const float2 v = __half22float2(as_h2(h[i]));
        l[i] = pack_sat(fabsf(a) > 65504.f ? 0.f : a - v.x, fabsf(e) > 65504.f ? 0.f : e - v.y);
      }
    }
    const uint32_t at = base + ((((uint32_t)(seg & 1) * 4 + ch) ^ (key & 7)) << 4);
    *reinterpret_cast<uint4*>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
    if (is_k) *reinterpret_cast<uint4*>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

__device__ __forceinline__ bool nonfinite2(uint32_t w) {
  return (w & 0x7C00u) == 0x7C00u || (w & 0x7C000000u) == 0x7C000000u;
}

// ---- the kernel -------------------------------------------------------

template <int BITS, int KIND, int D, int NQ>
__global__ void __launch_bounds__((Cfg<BITS, KIND, D, NQ>::THREADS), 1)
    extend_tc_kernel(const __grid_constant__ ExtendParams p) {
  using C = Cfg<BITS, KIND, D, NQ>;
  constexpr int ROWS = 128 * NQ;
  pdl_launch_dependents();
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (tc::smem_addr(raw) & 1023)) & 1023);
  auto& sh = *reinterpret_cast<Shared<C::STAGES>*>(smem + C::STAGES * C::STAGE);
  const CacheGeom& c = p.v.geom;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = blockIdx.y, b = blockIdx.z;
  const int split = blockIdx.x % p.splits;
  // row tiles last first: with a causal mask they see the most keys
  const int tile = gridDim.x / p.splits - 1 - blockIdx.x / p.splits;
  pdl_wait();

  const int before = checked_len(c, p.lens_before, b, -1);
  const int n_raw = new_rows_of(p.new_lens, b, p.num_new);
  const int n = max(n_raw, 0);
  const bool fits = before >= 0 && n_raw >= 0 && (long long)before + n <= p.len_limit;
  if (!fits && threadIdx.x == 0 && blockIdx.x == 0 && kvh == 0 && p.status) atomicOr(p.status, KVQ_FLAG_SEQ_LEN);
  const long long live_rows = (long long)n * p.G;
  const long long r0 = (long long)tile * ROWS;
  if (r0 >= live_rows) return;
  const int L = fits ? before + n : 0;
  const int t_first = (int)(r0 / p.G);
  const int t_last = (int)((min(r0 + ROWS, live_rows) - 1) / p.G);
  const int end = L ? before + t_last + 1 : 0;
  const int k0 = split * p.chunk, k1 = min(end, k0 + p.chunk);
  const int tiles = k1 > k0 ? (k1 - k0 + kKeys - 1) / kKeys : 0;
  const int all_see = L ? before + t_first : -1;  // every row sees the positions up to here
  const int nq = (NQ == 2 && live_rows - r0 <= 128) ? 1 : NQ;  // tiles with rows

  static_assert(sizeof(Shared<C::STAGES>) <= 512, "room behind the stages");
  const uint32_t bars = tc::smem_addr(&sh);
  auto full = [&](int s) { return bars + (uint32_t)offsetof(Shared<C::STAGES>, full) + 8 * s; };
  auto empty = [&](int s) { return bars + (uint32_t)offsetof(Shared<C::STAGES>, empty) + 8 * s; };
  auto q_full = [&](int i) { return bars + (uint32_t)offsetof(Shared<C::STAGES>, q_full) + 8 * i; };
  auto s_full = [&](int i) { return bars + (uint32_t)offsetof(Shared<C::STAGES>, s_full) + 8 * i; };
  auto p_full = [&](int i) { return bars + (uint32_t)offsetof(Shared<C::STAGES>, p_full) + 8 * i; };
  auto o_full = [&](int i) { return bars + (uint32_t)offsetof(Shared<C::STAGES>, o_full) + 8 * i; };
  volatile int* stop = &sh.stop;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      tc::mbar_init(full(s), C::PROD);
      tc::mbar_init(empty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(q_full(i), 128);
      tc::mbar_init(s_full(i), 1);
      tc::mbar_init(p_full(i), 128);
      tc::mbar_init(o_full(i), 1);
    }
    sh.stop = 0;
    tc::mbar_init_fence();
  }
  if (warp == C::WARPS - 1) tc::tmem_alloc(tc::smem_addr(&sh.tmem), C::COLS);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sh.tmem;

  if (warp < C::SOFT) {
    // ------------------------------------------------------ softmax rows
    const int i = warp >> 2;
    const long long r = r0 + i * 128 + (warp & 3) * 32 + lane;
    const bool live = r < live_rows;
    const bool any_live = r - lane < live_rows;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + C::COL_S + i * kKeys;
    const uint32_t to = tmem + lanes + C::COL_O + i * D;
    const uint32_t tq = tmem + lanes + C::COL_Q + i * (D / 2);
    const int t = live ? (int)(r / p.G) : 0;
    const long long orow = ((long long)b * p.num_new + t) * p.Hq + (long long)kvh * p.G + (live ? (int)(r % p.G) : 0);
    // (rows behind the last take part with q = 0 and are not written)
    const int last = live ? before + t : 0x7fffffff;
    if (i < nq && tiles) {
      // q to tensor memory, channels in the order the keys are unpacked in
      const uint4* src = reinterpret_cast<const uint4*>(p.q + orow * D);
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        uint32_t w[32];
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          uint4 x = make_uint4(0u, 0u, 0u, 0u);
          if (live && KVQ_IN(c, KVQ_ARRAY_Q, src + h * 8 + ch, 16)) x = src[h * 8 + ch];
          if constexpr (C::PAIRED) {  // (0, 4), (1, 5), (2, 6), (3, 7)
            w[4 * ch] = fast::prmt_b32(x.x, x.z, 0x5410u);
            w[4 * ch + 1] = fast::prmt_b32(x.x, x.z, 0x7632u);
            w[4 * ch + 2] = fast::prmt_b32(x.y, x.w, 0x5410u);
            w[4 * ch + 3] = fast::prmt_b32(x.y, x.w, 0x7632u);
          } else {
            w[4 * ch] = x.x, w[4 * ch + 1] = x.y, w[4 * ch + 2] = x.z, w[4 * ch + 3] = x.w;
          }
        }
        __syncwarp();
        tc::st32(tq + h * 32, w);
      }
      tc::wait_st();
      tc::fence_before();
      tc::mbar_arrive(q_full(i));
    }
    float m = -INFINITY, l = 0.f;  // reference maximum (log2 units) and sum
    bool going = i < nq;
    for (int j = 0; going && j < tiles; ++j) {
      const int st = j % C::STAGES;
      // (the tile's key masks come with its stage, which stays until P is handed over)
      going = tc::mbar_wait(full(st), (j / C::STAGES) & 1, stop) && tc::mbar_wait(s_full(i), j & 1, stop);
      going = __all_sync(0xffffffffu, going);
      if (!going) break;
      tc::fence_after();
      if (any_live) {
        uint32_t u[2][32];
        tc::ld32(ts, u[0]);
        tc::ld32(ts + 32, u[1]);
        tc::wait_ld();
        const int ks = k0 + j * kKeys;
        const uint32_t ok0 = sh.ok[st][0], ok1 = sh.ok[st][1];
        const bool whole = (ok0 & ok1) == 0xFFFFFFFFu && ks + kKeys - 1 <= last;
        if (!__all_sync(0xffffffffu, whole)) {
          uint32_t bad0 = 0, bad1 = 0;
          if constexpr (KIND == 2)
#pragma unroll
            for (int g = 0; g < C::SEGS; ++g) bad0 |= sh.bad[st][g][0], bad1 |= sh.bad[st][g][1];
          const int seen = last - ks;  // keys 0 .. seen of the tile
#pragma unroll
          for (int e = 0; e < 64; ++e) {
            const uint32_t ok = (e < 32 ? ok0 : ok1) >> (e & 31), bad = (e < 32 ? bad0 : bad1) >> (e & 31);
            const bool see = e <= seen && (ok & 1u);
            if (!see) u[e >> 5][e & 31] = 0xFF800000u;             // -inf
            else if (KIND == 2 && (bad & 1u)) u[e >> 5][e & 31] = 0x7FFFFFFFu;    // NaN: its V is not finite
          }
        }
        float mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < 64; ++e) mx = fmaxf(mx, __uint_as_float(u[e >> 5][e & 31]));
        mx *= p.scale_log2;
        const bool moves = mx > m + kLazy;  // m = -inf: any finite maximum
        if (__any_sync(0xffffffffu, moves)) {
          const float mn = moves ? mx : m;
          const float alpha = moves ? ex2(m - mn) : 1.f;
          m = mn;
          l *= alpha;
          if (j) {
#pragma unroll 1
            for (int h = 0; h < D / 16; ++h) {  // rare: few registers
              uint32_t o[16];
              tc::ld16(to + h * 16, o);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tc::st16(to + h * 16, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : m;
        uint32_t w[32];
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
          const float a = ex2(fmaf(__uint_as_float(u[e >> 5][e & 31]), p.scale_log2, -base));
          const float d = ex2(fmaf(__uint_as_float(u[e >> 5][(e & 31) + 1]), p.scale_log2, -base));
          sum[e & 2] += a;
          sum[(e & 2) + 1] += d;
          w[e >> 1] = fast::pack_h2(a, d);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tc::st32(ts, w);
        tc::wait_st();
      }
      tc::fence_before();
      tc::mbar_arrive(p_full(i));
    }
    if (going && tiles) going = __all_sync(0xffffffffu, tc::mbar_wait(o_full(i), 0, stop));
    tc::fence_after();
    if (going && any_live) {
      const float inv = l != 0.f ? 1.f / l : 0.f;
      const long long w = orow * p.splits + split;
#pragma unroll
      for (int h = 0; h < D / 32; ++h) {
        uint32_t o[32];
        if (tiles) {
          tc::ld32(to + h * 32, o);
          tc::wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        float x[32];  // place i of a chunk holds channel(i)
#pragma unroll
        for (int e = 0; e < 32; ++e) x[(e & ~7) + C::channel(e & 7)] = __uint_as_float(o[e]);
        if (live && p.splits == 1) {
          uint4* d = reinterpret_cast<uint4*>(p.out + orow * D + h * 32);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (KVQ_IN(c, KVQ_ARRAY_OUT, d + e, 16))
              d[e] = make_uint4(fast::pack_h2(x[8 * e] * inv, x[8 * e + 1] * inv),
                                fast::pack_h2(x[8 * e + 2] * inv, x[8 * e + 3] * inv),
                                fast::pack_h2(x[8 * e + 4] * inv, x[8 * e + 5] * inv),
                                fast::pack_h2(x[8 * e + 6] * inv, x[8 * e + 7] * inv));
        } else if (live) {
          float4* d = reinterpret_cast<float4*>(p.ws_o + w * D + h * 32);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (KVQ_IN(c, KVQ_ARRAY_WORKSPACE, d + e, 16))
              d[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        }
        __syncwarp();
      }
      if (p.splits > 1 && live) {
        float2* ml = reinterpret_cast<float2*>(p.ws_ml) + w;
        if (KVQ_IN(c, KVQ_ARRAY_WORKSPACE, ml, 8)) *ml = make_float2(m, l);
      }
    }
  } else if (warp < C::SOFT + C::PROD) {
    // ------------------------------------------------------ producers
    const int tid = threadIdx.x - C::SOFT * 32;
    constexpr int PT = C::PROD * 32;
    // this thread's key, and segment and K / V of its unit u; the keys of a
    // warp are consecutive, so its 16-byte stores hit all banks
    const int key = tid & (kKeys - 1);
    auto seg_of = [&](int u) { return ((u * PT + tid) / kKeys) % C::SEGS; };
    auto which_of = [&](int u) { return (u * PT + tid) / (kKeys * C::SEGS); };
    auto row_at = [&](int j) -> long long {
      const int pos = k0 + j * kKeys + key;
      if (pos >= k1) return -1;
      const long long row = token_row(c, b, kvh, pos);
      return row < 0 ? -2 : row;
    };
    auto note_keys = [&](int st, long long row) {  // the first two warps hold key = lane, 32 + lane
      const uint32_t ok = __ballot_sync(0xffffffffu, row >= 0);
      if (lane == 0) sh.ok[st][tid >> 5] = ok;
      if (row == -2 && p.status) atomicOr(p.status, KVQ_FLAG_BLOCK_TABLE);
    };
    if constexpr (KIND != 2) {
      uint32_t lut[4] = {0u, 0u, 0u, 0u};
      if constexpr (KIND == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // magnitudes 0..7 are levels 8..15: bytes apart
          const uint32_t h = __half_as_ushort(__float2half_rn(p.v.nf4_level[8 + i]));
          lut[i >> 2] |= (h & 0xFFu) << (8 * (i & 3));
          lut[2 + (i >> 2)] |= (h >> 8) << (8 * (i & 3));
        }
      }
      Seg<BITS> x[C::UNITS];
      long long row = -1;
      auto load_all = [&](int j) {
        row = row_at(j);
#pragma unroll
        for (int u = 0; u < C::UNITS; ++u) load_seg<BITS, KIND>(p, which_of(u), row, seg_of(u), x[u]);
      };
      if (tiles) load_all(0);
      for (int j = 0; j < tiles; ++j) {
        const int st = j % C::STAGES;
        if (!__all_sync(0xffffffffu, tc::mbar_wait(empty(st), ((j / C::STAGES) & 1) ^ 1, stop))) break;
        uint8_t* base = smem + st * C::STAGE;
        Seg<BITS> y[C::UNITS];
#pragma unroll
        for (int u = 0; u < C::UNITS; ++u) y[u] = x[u];
        const long long key_row = row;
        if (j + 1 < tiles) load_all(j + 1);
        if (tid < 64) note_keys(st, key_row);
#pragma unroll
        for (int u = 0; u < C::UNITS; ++u) {
          const bool is_k = which_of(u) == 0;
          store_seg<BITS, KIND, D>(p, y[u], is_k, key, seg_of(u), base + (is_k ? 0 : 2 * C::MAT),
                                   base + C::MAT, lut);
        }
        tc::fence_async_shared();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(full(st));
      }
    } else {
      // fp16 rows: straight to their places, one tile ahead of the arrival
      for (int j = 0; j <= tiles; ++j) {
        if (j < tiles) {
          const int st = j % C::STAGES;
          if (!__all_sync(0xffffffffu, tc::mbar_wait(empty(st), ((j / C::STAGES) & 1) ^ 1, stop))) break;
          const uint32_t base = tc::smem_addr(smem + st * C::STAGE);
          const long long row = row_at(j);
          if (tid < 64) note_keys(st, row);
#pragma unroll
          for (int u = 0; u < C::UNITS; ++u) {
            const int seg = seg_of(u), which = which_of(u);
            const uint8_t* src = p.v.codes[which] + max(row, 0ll) * c.row_bytes + seg * 64;
            const uint32_t dst = base + which * C::MAT + (seg >> 1) * (kKeys * 128) + key * 128;
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
              const uint8_t* sp = src + ch * 16;
              fast::cp_async16(dst + ((((seg & 1) * 4 + ch) ^ (key & 7)) << 4), sp,
                               row >= 0 && KVQ_IN(c, which ? KVQ_ARRAY_V_CODES : KVQ_ARRAY_K_CODES, sp, 16));
            }
          }
        }
        fast::cp_async_commit();
        fast::cp_async_wait<1>();
        if (j > 0) {
          const int st = (j - 1) % C::STAGES;
          // in a tile that some row sees in part, an infinite or NaN V must
          // not meet the zero weights of the rows that do not see it
          const bool partly = k0 + j * kKeys - 1 > all_see;
#pragma unroll
          for (int u = 0; u < C::UNITS; ++u) {
            if (which_of(u) == 0) continue;  // (a warp's units are all K or all V)
            const int seg = seg_of(u);
            bool bad = false;
            if (partly) {
              uint8_t* row = smem + st * C::STAGE + C::MAT + (seg >> 1) * (kKeys * 128) + key * 128;
#pragma unroll
              for (int ch = 0; ch < 4; ++ch) {
                uint4* v = reinterpret_cast<uint4*>(row + ((((seg & 1) * 4 + ch) ^ (key & 7)) << 4));
                const uint4 q = *v;
                if (nonfinite2(q.x) || nonfinite2(q.y) || nonfinite2(q.z) || nonfinite2(q.w)) {
                  bad = true;
                  *v = make_uint4(0u, 0u, 0u, 0u);
                }
              }
            }
            const uint32_t keys = __ballot_sync(0xffffffffu, bad);
            if (lane == 0) sh.bad[st][seg][(tid >> 5) & 1] = keys;
          }
          tc::fence_async_shared();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(full(st));
        }
      }
    }
  } else if (lane == 0 && tiles) {
    // ------------------------------------------------------ MMA issue
    constexpr uint32_t id_qk = tc::idesc_f16(kKeys, false), id_pv = tc::idesc_f16(D, true);
    const uint32_t data = tc::smem_addr(smem);
    auto qk = [&](int i, int j) {
      const uint32_t base = data + (j % C::STAGES) * C::STAGE;
      const uint32_t d = tmem + C::COL_S + i * kKeys, a = tmem + C::COL_Q + i * (D / 2);
#pragma unroll
      for (int part = 0; part < (C::LO ? 2 : 1); ++part)
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc::mma_ts(d, a + kk * 8,
                     tc::smem_desc(base + part * C::MAT + (kk >> 2) * (kKeys * 128) + (kk & 3) * 32, 16, 1024), id_qk,
                     part || kk);
      tc::commit(s_full(i));
    };
    auto pv = [&](int i, int j) {
      const uint32_t base = data + (j % C::STAGES) * C::STAGE + (C::LO ? 2 : 1) * C::MAT;
      const uint32_t d = tmem + C::COL_O + i * D, a = tmem + C::COL_S + i * kKeys;
#pragma unroll
      for (int kk = 0; kk < kKeys / 16; ++kk)
        tc::mma_ts(d, a + kk * 8, tc::smem_desc(base + kk * 2048, kKeys * 128, 1024), id_pv, j || kk);
    };
    bool ok = tc::mbar_wait(full(0), 0, stop);
    for (int i = 0; ok && i < nq; ++i) {
      ok = tc::mbar_wait(q_full(i), 0, stop);
      tc::fence_after();
      if (ok) qk(i, 0);
    }
    for (int j = 0; ok && j < tiles; ++j) {
      for (int i = 0; ok && i < nq; ++i) {
        ok = tc::mbar_wait(p_full(i), j & 1, stop);
        tc::fence_after();
        if (!ok) break;
        pv(i, j);
        if (i == nq - 1) tc::commit(empty(j % C::STAGES));
        if (j + 1 < tiles) {
          if (i == 0) ok = tc::mbar_wait(full((j + 1) % C::STAGES), ((j + 1) / C::STAGES) & 1, stop);
          if (ok) qk(i, j + 1);
        } else {
          tc::commit(o_full(i));
        }
      }
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (warp == C::WARPS - 1) {
    tc::fence_after();
    tc::tmem_dealloc(tmem, C::COLS);
  }
  if (threadIdx.x == 0 && sh.stop && p.status) atomicOr(p.status, KVQ_FLAG_TIMEOUT);
}

template <int BITS, int KIND, int D, int NQ>
cudaError_t run_nq(const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream) {
  using C = Cfg<BITS, KIND, D, NQ>;
  static KernelSetup setup;
  int occ = 0;
  const cudaError_t e = setup_kernel(extend_tc_kernel<BITS, KIND, D, NQ>, setup, C::THREADS, C::SMEM, &occ);
  if (e != cudaSuccess) return e;
  if (plan) {
    plan->tile_rows = 128 * NQ;
    plan->occ = occ;
    return cudaSuccess;
  }
  const long long tiles = ((long long)p->num_new * p->G + 128 * NQ - 1) / (128 * NQ);
  const dim3 grid((unsigned)(tiles * p->splits), p->v.geom.Hkv, p->batch);
  return launch_pdl(extend_tc_kernel<BITS, KIND, D, NQ>, grid, dim3(C::THREADS), C::SMEM, stream, *p);
}

// One instance file per format calls this for its BITS and KIND.
template <int BITS, int KIND>
cudaError_t run_tc(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream) {
  if (D == 64) return nq == 1 ? run_nq<BITS, KIND, 64, 1>(p, plan, stream) : run_nq<BITS, KIND, 64, 2>(p, plan, stream);
  return nq == 1 ? run_nq<BITS, KIND, 128, 1>(p, plan, stream) : run_nq<BITS, KIND, 128, 2>(p, plan, stream);
}

}  // namespace ext

cudaError_t run_extend_tc_int2(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream);
cudaError_t run_extend_tc_int4(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream);
cudaError_t run_extend_tc_int8(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream);
cudaError_t run_extend_tc_nf4(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream);
cudaError_t run_extend_tc_fp16(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream);

}  // namespace kvq
