// Attention of 16 or 32 rows over codes that stay in registers (INT4, INT8 and
// NF4 caches at head_dim 64 and 128): the members of a shared prefix where they
// are few.
//
// Rows are (sequence, new token, head of the KV head's group) triples, as in
// kvq_extend_tc.cuh.  There the codes pass through shared memory as fp16 sums
// of two numbers, 64 KB written and read per 64 keys whatever the number of
// rows, about 1900 cycles (30 a key).  Here a code is one logic operation away
// from an fp16 subnormal c 2^-24 (kvq_decode_fast.cuh), scale and zero-point
// stay out of the products, and every code is unpacked once for 32 rows:
//   S = Q C_K^T  m16n8k16, A = q fragments from shared memory, B = the codes of
//                eight keys; per group of channels s (sum q c - z sum q) in
//                fp32, the zero-point term as the accumulator's start
//   O += P C_V   A = the probabilities, fp16, times a group's scale per key; B =
//                V's codes with the keys in pairs (ldmatrix.trans); sum p s z of
//                each group by one more product against its zero-points, taken
//                off at the end
// q, K's scales and V's scales enter times powers of two that keep them where fp16
// has its bits, whatever their size; they are taken back in fp32.
// A warp has a pipeline of 32-key tiles to itself and its own running maximum
// and sum per row; the four of a block are joined at the end, and the block
// leaves a partial.
//
// What bounds it: latency, of unpacking, products and softmax in turn with two or
// three warps a scheduler (32 heads x 32 rows over 4096 keys, INT4: 46 % of the
// issue slots, 18 % of the tensor pipe, 0.7 TB/s; 23 us by itself, cold).  Against
// the kernel of kvq_extend_tc.cuh, the whole call with tails of 64 keys, 8 KV heads
// of 128 over INT4, each with its best splits: 8 rows over 512, 4096, 16384 keys 8.2,
// 11.5, 20.7 us (12.1, 15.9, 25.3 there), 32 rows 9.7, 16.0, 27.2 (12.7, 17.7, 28.6),
// 64 rows 11.3, 19.1, 37.1 (12.9, 17.9, 29.4).  Tiles of 16 rows against tiles of 32:
// 32 rows of 8 heads over 512 keys 9.7 against 12.1 us (INT8: 9.9, 14.8), of 32 heads
// over 16384 78.6 against 69.3.  Sixteen keys are taken at a time: 32 held more
// registers than there are (108 spilled accesses a tile).
#pragma once

#include "kvq_decode_fast.cuh"
#include "kvq_load.cuh"
#include "kvq_prefix.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace rows {

using namespace fast;

// KIND: 0 integer codes, 1 NF4
template <int BITS, int KIND, int D, int MT>
struct RowCfg {
  static constexpr int ROWS = 16 * MT;
  static constexpr int ROWB = D * BITS / 8;
  static constexpr int CHUNKS = ROWB / 16;       // 16-byte chunks of a row
  static constexpr int RPL = 128 / ROWB;
  static constexpr int DPC = 128 / BITS;         // channels of a chunk
  static constexpr int FPC = DPC / 8;            // n-tiles of V, of a chunk
  static constexpr int KPC = DPC / 16;           // k-blocks of K, of a chunk
  static constexpr int KB = D / 16;
  static constexpr int MAXNG = D / 32;           // groups (of 32 channels or more)
  static constexpr int HDRB = 2 * MAXNG;
  static constexpr int CODE_TILE = kTT * ROWB, HDR_TILE = kTT * HDRB;
  static constexpr int STAGE = 2 * CODE_TILE + 4 * HDR_TILE;
  static constexpr int KROW = kTT, VROW = kTT + 8;  // entries of a group's row (bank offsets)
  // the zero-point term of the scores, a product over (part, group) slots
  static constexpr int NZ = KIND == 0 ? (3 * MAXNG + 15) / 16 : 0, ZROW = 16 * NZ + 8;
  static constexpr int XHDR = MAXNG * (KROW * 4 + 2 * VROW * 2) + kTT * (NZ ? ZROW * 2 : 0);
  // q of one unit: fragments, sums, the rows' tokens
  static constexpr int Q_FRAG = MT * (KB + NZ) * 32 * 16, Q_SUM = MAXNG * ROWS * 4;
  static constexpr int Q_BYTES = Q_FRAG + Q_SUM + ROWS * 4;
  static constexpr int FIXED = Q_BYTES;
  // Blocks an SM: the tile of 16 rows leaves registers for three where its stages
  // fit (32 heads over 16384 keys, INT4: 49.6 -> 42.8 us with three, over 4096
  // 20.7 -> 20.3; a block of 32 rows needs all of its 255 registers).
  static constexpr int CTAS = MT == 1 && BITS == 4 && D == 128 ? 3 : 2;
  static constexpr int STAGES_FIT = (((CTAS == 3 ? 75 : 112) * 1024 - FIXED) / kWarps - XHDR) / STAGE;
  static constexpr int STAGES = STAGES_FIT > 4 ? 4 : STAGES_FIT;
  static constexpr int WARP_BYTES = STAGES * STAGE + XHDR;
  static constexpr int RED = D + 4;              // floats of a row in the join
  static constexpr int PIPE = kWarps * WARP_BYTES;
  static constexpr int JOIN = kWarps * ROWS * (RED + 2) * 4;
  static constexpr int SMEM = FIXED + (PIPE > JOIN ? PIPE : JOIN);
  static_assert(STAGES >= 2, "a tile in flight beside the one in use");
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "the blocks an SM is to hold");
  __device__ static __forceinline__ uint32_t at(int t, int c) {
    return (uint32_t)(t * ROWB + ((c ^ ((t / RPL) & (CHUNKS - 1))) << 4));
  }
};

// How far (log2 units) a tile's maximum may lead the reference, and the factor that
// the probabilities carry, so that they keep fp16's 11 bits down to 2^-21 of the
// row's reference.
constexpr float kSlackRows = 2.f;
constexpr float kLiftRows = 7.f;

// A probability enters times V's scale, as fp16.  V's scales may be of any size, so
// a warp takes those of a group times a power of two, exactly: the largest seen
// comes to 2^4 .. 2^6.  A product is then at most 2^(2 + 7 + 6), and that of the
// reference with the largest scale is 2^11 at least: the bits of smaller ones last
// to 2^-25 of it (without the power, INT8 groups at 0.02 lost theirs from 2^-8 of the
// row's largest on: 14 times the bound where one heavy key's V was small).  A group's
// power, as the fp16 exponent that its scales stay within: it only rises, and the
// group's sums come down with it.  All the powers together cost 2 % (32 heads over
// 4096 keys, the whole call 36.5 -> 37.1 us; 37.8 with the maxima worked out in each
// tile instead of a vote).
struct ScalePower {
  // the exponent of a scale, and the one to allow for it: a binade more
  __device__ static __forceinline__ uint32_t field(uint32_t bits) { return (bits & 0x7FFFu) >> 10; }
  __device__ static __forceinline__ float factor(uint32_t allowed) { return __uint_as_float((147u - allowed) << 23); }    // 2^(20 - allowed)
  __device__ static __forceinline__ float inverse(uint32_t allowed) { return __uint_as_float((107u + allowed) << 23); }
};

// A block takes a prefix, a KV head, a tile of rows and a split.
template <int BITS, int KIND, int D, int MT>
__global__ void __launch_bounds__(kWarps * 32, RowCfg<BITS, KIND, D, MT>::CTAS) rows_kernel(const __grid_constant__ ExtendParams p) {
  using C = RowCfg<BITS, KIND, D, MT>;
  constexpr float kSub = KIND == 1 ? 1.f : 16777216.f;  // 2^24: codes enter as c 2^-24
  constexpr int NT = C::CHUNKS * C::FPC;                // n-tiles of V: D / 8
  extern __shared__ __align__(128) uint8_t smem[];
  const CacheGeom& geo = p.v.geom;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rho = lane >> 2, j = lane & 3;
  uint32_t lut[4] = {0u, 0u, 0u, 0u};
  if constexpr (KIND == 1) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t h = __half_as_ushort(__float2half_rn(p.v.nf4_level[8 + k]));
      lut[k >> 2] |= (h & 0xFFu) << (8 * (k & 3));
      lut[2 + (k >> 2)] |= (h >> 8) << (8 * (k & 3));
    }
  }
  pdl_wait();
  say_started(p.started);

  // ---- which rows, which keys ----
  const int kvh = blockIdx.y, split = blockIdx.x % p.splits;
  const PrefixTile pt = prefix_tile(p.plan, blockIdx.x / p.splits, p.num_new * p.G, C::ROWS);
  const int b = pt.n;
  if (b < 0) return;
  const int end = prefix_len(p.plan, b, p.len_limit);
  if (split * p.chunk >= end) return;  // (the join knows which splits hold keys)
  const int r0 = pt.tile * C::ROWS;
  int own_tok;  // of row lane mod ROWS
  const int live_rows = prefix_rows(p.plan, pt, p.new_lens, p.num_new, p.G, (long long)r0 + (lane & (C::ROWS - 1)), &own_tok);
  if (r0 >= live_rows) return;
  const int k0 = split * p.chunk, k1 = min(end, k0 + p.chunk);
  const int ntiles = k1 > k0 ? (k1 - k0 + kTT - 1) / kTT : 0;
  const int nmine = ntiles > warp ? (ntiles - warp + kWarps - 1) / kWarps : 0;

  uint4* const q_frag = reinterpret_cast<uint4*>(smem);  // [MT][KB][lane], then [MT][NZ][lane]
  float* const q_sum = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(q_frag) + C::Q_FRAG);  // [group][row]
  int* const toks = reinterpret_cast<int*>(q_sum + C::MAXNG * C::ROWS);
  uint8_t* const pipe = smem + C::FIXED;
  uint8_t* const mine = pipe + warp * C::WARP_BYTES;
  const uint32_t mine_s = smem_u32(mine);
  uint8_t* const x = mine + C::STAGES * C::STAGE;  // header scratch
  float* const ksc = reinterpret_cast<float*>(x);  // [group][key]: K's scale, times 2^24
  uint16_t* const vs = reinterpret_cast<uint16_t*>(x + C::MAXNG * C::KROW * 4);  // [group][key]
  uint16_t* const vz = vs + C::MAXNG * C::VROW;
  uint16_t* const kz = vz + C::MAXNG * C::VROW;  // [key][slot]: scale times zero-point, see below

  // ---- the pipeline ----
  const int NG = geo.ngroups;  // groups, of 2^lcpg chunks
  const int lcpg = __ffs(C::CHUNKS / NG) - 1, cmask = (1 << lcpg) - 1;
  const bool zeros = KIND == 0 && !geo.sym;
  bool unmapped = false;
  uint32_t mask_of[C::STAGES];  // keys that do not count, of this tile and the next ones
#pragma unroll
  for (int s = 0; s < C::STAGES; ++s) mask_of[s] = 0;
  auto issue = [&](int it, int stage) -> uint32_t {
    uint32_t bad = 0xffffffffu;
    if (it < nmine) {
      const int start = k0 + (warp + it * kWarps) * kTT;
      const int n = min(kTT, k1 - start);
      const long long row = lane < n ? token_row(geo, b, kvh, start + lane) : -1;
      unmapped |= lane < n && row < 0;
      const uint32_t kc = mine_s + stage * C::STAGE, vc = kc + C::CODE_TILE, hd = vc + C::CODE_TILE;
#pragma unroll
      for (int k = 0; k < C::CHUNKS; ++k) {
        const int c = lane + 32 * k, tok = c / C::CHUNKS, part = c % C::CHUNKS;
        const long long r = __shfl_sync(0xffffffffu, row, tok);
        const long long off = r >= 0 ? r * C::ROWB + part * 16 : 0;
        const uint32_t to = C::at(tok, part);
        cp_async16(kc + to, p.v.codes[0] + off, r >= 0 && KVQ_IN(geo, KVQ_ARRAY_K_CODES, p.v.codes[0] + off, 16));
        cp_async16(vc + to, p.v.codes[1] + off, r >= 0 && KVQ_IN(geo, KVQ_ARRAY_V_CODES, p.v.codes[1] + off, 16));
      }
      const long long h = row >= 0 ? row * NG : 0;
      auto header = [&](auto bytes) {
        constexpr int N = decltype(bytes)::value;
        const uint32_t to = hd + lane * N;
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          if ((a & 1) && !zeros) continue;
          const __half* from = (a & 1 ? p.v.zero : p.v.scale)[a >> 1] + h;
          const int array = a == 0 ? KVQ_ARRAY_K_SCALE : a == 1 ? KVQ_ARRAY_K_ZERO : a == 2 ? KVQ_ARRAY_V_SCALE : KVQ_ARRAY_V_ZERO;
          cp_async_small<N>(to + a * C::HDR_TILE, from, row >= 0 && KVQ_IN(geo, array, from, N));
        }
      };
      if (NG == 2) header(std::integral_constant<int, 4>{});
      else header(std::integral_constant<int, 8>{});
      bad = __ballot_sync(0xffffffffu, row < 0);
    }
    cp_async_commit();
    return bad;
  };
#pragma unroll
  for (int s = 0; s < C::STAGES; ++s) mask_of[s] = issue(s, s);

  // ---- q as fragments, its channels in the order the codes are unpacked in ----
  //
  // Integer codes: a row of q enters times a power of two, which the softmax takes
  // back, so that its largest channel comes to 2^7 .. 2^8.  The sums over groups then
  // fit fp16's range (as q stood, 32 channels above 2047 did not), and q / 16 is exact
  // but for channels below 2^-17 of the largest.
  if (warp == 0 && lane < C::ROWS) toks[lane] = own_tok;
  constexpr int QI = (MT * C::CHUNKS + kWarps - 1) / kWarps;  // chunks of rows rho and rho + 8 that a warp takes
  uint32_t qx[QI][2][4];
  uint16_t* const tops = reinterpret_cast<uint16_t*>(q_sum);  // [chunk][row]: the largest finite channel
  static_assert(C::CHUNKS * 2 <= C::MAXNG * 4, "they fit where the sums come to lie");
#pragma unroll
  for (int n = 0; n < QI; ++n) {
    const int i = n * kWarps + warp, mt = i / C::CHUNKS, c = i % C::CHUNKS;
    if (i >= MT * C::CHUNKS) break;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      qx[n][hh][0] = qx[n][hh][1] = qx[n][hh][2] = qx[n][hh][3] = 0u;
      const int r = mt * 16 + rho + 8 * hh;
      const int tok = __shfl_sync(0xffffffffu, own_tok, r);
      if (r0 + r < live_rows) {
        const __half* from = p.q + ((long long)tok * p.Hq + (long long)kvh * p.G + (r0 + r) % p.G) * D + c * C::DPC + j * (C::DPC / 4);
        if constexpr (BITS == 4) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (KVQ_IN(geo, KVQ_ARRAY_Q, from, 16)) v = __ldg(reinterpret_cast<const uint4*>(from));
          qx[n][hh][0] = v.x, qx[n][hh][1] = v.y, qx[n][hh][2] = v.z, qx[n][hh][3] = v.w;
        } else {
          uint2 v = make_uint2(0u, 0u);
          if (KVQ_IN(geo, KVQ_ARRAY_Q, from, 8)) v = __ldg(reinterpret_cast<const uint2*>(from));
          qx[n][hh][0] = v.x, qx[n][hh][1] = v.y;
        }
      }
      if constexpr (KIND == 0) {
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 2 * (C::DPC / 8); ++e) {
          const uint32_t h = qx[n][hh][e >> 1] >> (16 * (e & 1)) & 0x7FFFu;
          top = max(top, h < 0x7C00u ? h : 0u);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        if (j == 0) tops[c * C::ROWS + r] = (uint16_t)top;
      }
    }
  }
  if constexpr (KIND == 0) __syncthreads();
  float unit[MT][2];                      // scores to log2 units
  uint32_t lift[MT][2], lift_odd[MT][2];  // the row's power (fp16, twice), and where channels meet 16 c
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      // (2^-60: scores reach 2^41, so that below it all weights are alike; with the powers
      // `unit` is then 2^-115 at least, and not 0 times a masked key's infinity)
      unit[mt][hh] = fmaxf(p.scale_log2, 0x1p-60f);
      lift[mt][hh] = lift_odd[mt][hh] = 0x3C003C00u;  // 1
      if constexpr (KIND == 0) {
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < C::CHUNKS; ++c) top = max(top, (uint32_t)tops[c * C::ROWS + mt * 16 + rho + 8 * hh]);
        const int a = min(22 - (int)(top >> 10), 15);  // -8 .. 15
        unit[mt][hh] *= __int_as_float((127 - a) << 23);
        lift[mt][hh] = (uint32_t)(15 + a) * 0x04000400u;
        lift_odd[mt][hh] = (uint32_t)(11 + a) * 0x04000400u;
      }
    }
#pragma unroll
  for (int n = 0; n < QI; ++n) {
    const int i = n * kWarps + warp, mt = i / C::CHUNKS, c = i % C::CHUNKS;
    if (i >= MT * C::CHUNKS) break;
    const __half2 f0 = u32_as_h2(mt ? lift[MT - 1][0] : lift[0][0]), f1 = u32_as_h2(mt ? lift[MT - 1][1] : lift[0][1]);
    uint4* const to = q_frag + (mt * C::KB + c * C::KPC) * 32 + lane;
    if constexpr (BITS == 4) {
      // channels 8j + (0, 4, 1, 5), then + (2, 6, 3, 7); the odd ones meet
      // nibbles held as 16 c
      const __half2 g0 = u32_as_h2(mt ? lift_odd[MT - 1][0] : lift_odd[0][0]);
      const __half2 g1 = u32_as_h2(mt ? lift_odd[MT - 1][1] : lift_odd[0][1]);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        uint4 f;
        f.x = h2_as_u32(__hmul2(u32_as_h2(prmt_b32(qx[n][0][kk], qx[n][0][2 + kk], 0x5410u)), f0));
        f.y = h2_as_u32(__hmul2(u32_as_h2(prmt_b32(qx[n][1][kk], qx[n][1][2 + kk], 0x5410u)), f1));
        f.z = h2_as_u32(__hmul2(u32_as_h2(prmt_b32(qx[n][0][kk], qx[n][0][2 + kk], 0x7632u)), g0));
        f.w = h2_as_u32(__hmul2(u32_as_h2(prmt_b32(qx[n][1][kk], qx[n][1][2 + kk], 0x7632u)), g1));
        to[32 * kk] = f;
      }
    } else {
      to[0] = make_uint4(h2_as_u32(__hmul2(u32_as_h2(qx[n][0][0]), f0)), h2_as_u32(__hmul2(u32_as_h2(qx[n][1][0]), f1)),
                         h2_as_u32(__hmul2(u32_as_h2(qx[n][0][1]), f0)), h2_as_u32(__hmul2(u32_as_h2(qx[n][1][1]), f1)));
    }
  }
  __syncthreads();
  // The sum of q over each group of channels, by a product with ones (16 where
  // the fragment holds q / 16).
  for (int mt = warp; KIND == 0 && mt < MT; mt += kWarps) {
    constexpr uint32_t one = 0x3C003C00u, odd = BITS == 4 ? 0x4C004C00u : one;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C::CHUNKS; ++c) {
#pragma unroll
      for (int kk = 0; kk < C::KPC; ++kk) {
        const uint4 a = q_frag[(mt * C::KB + c * C::KPC + kk) * 32 + lane];
        mma16816(acc, a.x, a.y, a.z, a.w, one, odd);
      }
      if ((c & cmask) == cmask) {
        if (j == 0) {
          q_sum[(c >> lcpg) * C::ROWS + mt * 16 + rho] = acc[0];
          q_sum[(c >> lcpg) * C::ROWS + mt * 16 + rho + 8] = acc[2];
        }
        acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
      }
    }
  }
  __syncthreads();
  // The scores' zero-point term - sum_g Q_g (s_g z_g) is a product as well: both
  // factors as sums of two fp16 numbers, of which hi hi, hi lo and lo hi are
  // taken (2^-22 of it is left out).  Slot k = part M + g holds (hi, lo, hi) of
  // s z against (hi, hi, lo) of - Q.
  if constexpr (KIND == 0) {
    for (int i = warp * 32 + lane; i < MT * C::NZ * 32; i += kWarps * 32) {
      const int l = i & 31, nz = (i >> 5) % C::NZ, mt = (i >> 5) / C::NZ;
      uint32_t f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t w = 0;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int k = 16 * nz + 2 * (l & 3) + hh + 8 * (e >> 1), part = k / C::MAXNG, g = k % C::MAXNG;
          if (part > 2 || g >= NG) continue;
          const float v = -q_sum[g * C::ROWS + mt * 16 + (l >> 2) + 8 * (e & 1)];
          const __half hi = __float2half_rn(v);
          const __half h = part == 2 ? __float2half_rn(v - __half2float(hi)) : hi;
          w |= (uint32_t)__half_as_ushort(h) << (16 * hh);
        }
        f[e] = w;
      }
      q_frag[(MT * C::KB + mt * C::NZ + nz) * 32 + l] = make_uint4(f[0], f[1], f[2], f[3]);
    }
    for (int k = 0; k < C::ZROW / 8; ++k) *reinterpret_cast<uint4*>(kz + lane * C::ZROW + 8 * k) = make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();

  // ---- running state ----
  uint32_t power = 0;  // of each group, a byte (ScalePower)
  // K's scales enter times a power of two as well, so that the largest s z seen comes
  // to 2^12 .. 2^14 and both of its parts keep their bits (keys of 1e-4: the second
  // part was gone); `unit` takes it back.  Its exponent field, 0: all zero so far.
  uint32_t power_k = 0;
  float lift_k = 1.f;
  // Group g's entry of four (registers: the index is a constant but for the rows of
  // two groups in a kernel for four).
  auto of_chunk = [&](const float (&x)[C::MAXNG], int chunk) {
    const int full = chunk * C::MAXNG / C::CHUNKS, half = chunk * 2 / C::CHUNKS;
    return NG == C::MAXNG ? x[full] : x[half];
  };
  float o[MT][NT][4], cz[MT][4], m_ref[MT][2], l_run[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int n = 0; n < NT; ++n) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.f;
    cz[mt][0] = cz[mt][1] = cz[mt][2] = cz[mt][3] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m_ref[mt][e] = -INFINITY;
      l_run[mt][e] = 0.f;
    }
  }
  int stage = 0;
#pragma unroll 1
  for (int it = 0; it < nmine; ++it) {
    cp_async_wait<C::STAGES - 1>();
    __syncwarp();
    const uint8_t* const st = mine + stage * C::STAGE;
    const uint32_t kc = mine_s + stage * C::STAGE, vc = kc + C::CODE_TILE;
    uint32_t bad = mask_of[0];
    // headers: a lane its key's, to [group][key]
    {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(st + 2 * C::CODE_TILE) + lane * NG;
      constexpr uint16_t half_range = BITS == 4 ? 0x4800u : 0x5800u;  // 8, 128
      float sz[C::MAXNG];
      uint32_t top_k = 0;
      bool over = false;  // a scale, or K's scale times zero-point, beyond what its power allows
#pragma unroll
      for (int g = 0; g < C::MAXNG; ++g) {
        sz[g] = 0.f;
        if (g >= NG) break;
        over |= ScalePower::field(h[C::HDR_TILE + g]) > (power >> (8 * g) & 255u);
        if constexpr (KIND == 0) {
          sz[g] = __half2float(__ushort_as_half(h[g])) * __half2float(__ushort_as_half(zeros ? h[C::HDR_TILE / 2 + g] : half_range));
          const uint32_t bits = __float_as_uint(fabsf(sz[g]));
          top_k = max(top_k, bits < 0x7F800000u ? bits : 0u);
        }
      }
      over |= top_k >> 23 > power_k;
      if (__any_sync(0xffffffffu, over)) {
        uint32_t allowed = power;
#pragma unroll
        for (int g = 0; g < C::MAXNG; ++g) {
          if (g >= NG) break;
          const uint32_t top = ScalePower::field(__reduce_max_sync(0xffffffffu, h[C::HDR_TILE + g] & 0x7FFFu));
          if (top > (power >> (8 * g) & 255u)) allowed = (allowed & ~(255u << (8 * g))) | (top + 1) << (8 * g);
        }
        // the sums so far come down with their groups' powers
        float down[C::MAXNG];
#pragma unroll
        for (int g = 0; g < C::MAXNG; ++g)
          down[g] = ScalePower::factor(allowed >> (8 * g) & 255u) * ScalePower::inverse(power >> (8 * g) & 255u);
        power = allowed;
        // (cz: group g's column, of lanes j = g / 2)
        const float c0 = C::MAXNG == 4 && j == 1 ? down[C::MAXNG - 2] : down[0];
        const float c1 = C::MAXNG == 4 && j == 1 ? down[C::MAXNG - 1] : down[1];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          cz[mt][0] *= c0, cz[mt][1] *= c1, cz[mt][2] *= c0, cz[mt][3] *= c1;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float f = of_chunk(down, n / C::FPC);
            o[mt][n][0] *= f, o[mt][n][1] *= f, o[mt][n][2] *= f, o[mt][n][3] *= f;
          }
        }
        if constexpr (KIND == 0) {
          const uint32_t top = __reduce_max_sync(0xffffffffu, top_k) >> 23;  // at most 159
          if (top > power_k) {
            const uint32_t next = max(top + 1u, 100u);  // (of less than 2^-27 a few bits go)
            const float f = __uint_as_float((next - (power_k ? power_k : 140u) + 127u) << 23);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) unit[mt][0] *= f, unit[mt][1] *= f;
            power_k = next;
            lift_k = __uint_as_float((267u - power_k) << 23);
          }
        }
      }
#pragma unroll
      for (int g = 0; g < C::MAXNG; ++g) {
        if (g >= NG) break;
        ksc[g * C::KROW + lane] = __half2float(__ushort_as_half(h[g])) * (kSub * lift_k);
        vs[g * C::VROW + lane] =
            __half_as_ushort(__float2half_rn(__half2float(__ushort_as_half(h[C::HDR_TILE + g])) *
                                             ScalePower::factor(power >> (8 * g) & 255u)));
        if constexpr (KIND == 0) {
          const float y = sz[g] * lift_k;
          const __half hi = __float2half_rn(y);
          uint16_t* const to = kz + lane * C::ZROW + g;
          to[0] = to[2 * C::MAXNG] = __half_as_ushort(hi);
          to[C::MAXNG] = __half_as_ushort(__float2half_rn(y - __half2float(hi)));
          vz[g * C::VROW + lane] = zeros ? h[3 * C::HDR_TILE / 2 + g] : half_range;
        }
      }
    }
    __syncwarp();

    // sixteen keys at a time: few registers beside the rows' sums
#pragma unroll 1
    for (int ks = 0; ks < 2; ++ks) {
      // scores (log2 units): s[mt][u] = rows rho, rho + 8 x keys 16 ks + 8 u + 2j, + 1
      float s[MT][2][4];
      {
        uint32_t w[2][C::CHUNKS];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int tok = 16 * ks + 8 * u + (lane & 7);
          if constexpr (C::CHUNKS == 2) {
            ldsm_x2(kc + C::at(tok, (lane >> 3) & 1), w[u][0], w[u][1]);
          } else {
#pragma unroll
            for (int c4 = 0; c4 < C::CHUNKS; c4 += 4)
              ldsm_x4(kc + C::at(tok, c4 + (lane >> 3)), w[u][c4], w[u][c4 + 1], w[u][c4 + 2], w[u][c4 + 3]);
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int u = 0; u < 2; ++u) s[mt][u][0] = s[mt][u][1] = s[mt][u][2] = s[mt][u][3] = 0.f;
        if constexpr (KIND == 0) {
#pragma unroll
          for (int nz = 0; nz < C::NZ; ++nz) {
            uint32_t z[2][2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint16_t* const from = kz + (16 * ks + 8 * u + rho) * C::ZROW + 16 * nz + 2 * j;
              z[u][0] = *reinterpret_cast<const uint32_t*>(from);
              z[u][1] = *reinterpret_cast<const uint32_t*>(from + 8);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const uint4 a = q_frag[(MT * C::KB + mt * C::NZ + nz) * 32 + lane];
              mma16816(s[mt][0], a.x, a.y, a.z, a.w, z[0][0], z[0][1]);
              mma16816(s[mt][1], a.x, a.y, a.z, a.w, z[1][0], z[1][1]);
            }
          }
        }
        float acc[MT][2][4];
#pragma unroll
        for (int c = 0; c < C::CHUNKS; ++c) {
          if ((c & cmask) == 0) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int u = 0; u < 2; ++u) acc[mt][u][0] = acc[mt][u][1] = acc[mt][u][2] = acc[mt][u][3] = 0.f;
          }
          uint32_t h[2][4];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if constexpr (BITS == 4) {
              nib8_to_h2<KIND == 1, true>(w[u][c], h[u], lut);
            } else {
              h[u][0] = byte2_to_h2_biased<0x4140, true>(w[u][c]);
              h[u][1] = byte2_to_h2_biased<0x4342, true>(w[u][c]);
            }
          }
#pragma unroll
          for (int kk = 0; kk < C::KPC; ++kk)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const uint4 a = q_frag[(mt * C::KB + c * C::KPC + kk) * 32 + lane];
              mma16816(acc[mt][0], a.x, a.y, a.z, a.w, h[0][2 * kk], h[0][2 * kk + 1]);
              mma16816(acc[mt][1], a.x, a.y, a.z, a.w, h[1][2 * kk], h[1][2 * kk + 1]);
            }
          if ((c & cmask) == cmask) {  // a group's last chunk: times its scales
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float2 sc = *reinterpret_cast<const float2*>(ksc + (c >> lcpg) * C::KROW + 16 * ks + 8 * u + 2 * j);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                  const float2 y = tc::fma2(make_float2(acc[mt][u][e], acc[mt][u][e + 1]), sc,
                                            make_float2(s[mt][u][e], s[mt][u][e + 1]));
                  s[mt][u][e] = y.x, s[mt][u][e + 1] = y.y;
                }
            }
          }
        }
      }
      if (bad) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int t = 16 * ks + 8 * u + 2 * j + (e & 1);
              if (bad >> t & 1u) s[mt][u][e] = -INFINITY;
            }
      }

      // softmax, the reference moved only where it is exceeded by kSlackRows
      uint32_t pa[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float top[2];
        top[0] = fmaxf(fmaxf(s[mt][0][0], s[mt][0][1]), fmaxf(s[mt][1][0], s[mt][1][1])) * unit[mt][0];
        top[1] = fmaxf(fmaxf(s[mt][0][2], s[mt][0][3]), fmaxf(s[mt][1][2], s[mt][1][3])) * unit[mt][1];
        if (__any_sync(0xffffffffu, top[0] > m_ref[mt][0] + kSlackRows || top[1] > m_ref[mt][1] + kSlackRows)) {
          float alpha[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
            top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
            const bool moves = top[e] > m_ref[mt][e] + kSlackRows;
            alpha[e] = moves ? ex2(m_ref[mt][e] - top[e]) : 1.f;
            m_ref[mt][e] = moves ? top[e] : m_ref[mt][e];
            l_run[mt][e] *= alpha[e];
            cz[mt][2 * e] *= alpha[e], cz[mt][2 * e + 1] *= alpha[e];
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
            o[mt][n][0] *= alpha[0], o[mt][n][1] *= alpha[0], o[mt][n][2] *= alpha[1], o[mt][n][3] *= alpha[1];
        }
        const float ma = m_ref[mt][0] == -INFINITY ? 0.f : -m_ref[mt][0] + kLiftRows;
        const float mb = m_ref[mt][1] == -INFINITY ? 0.f : -m_ref[mt][1] + kLiftRows;
        float2 sum[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float2 a = tc::fma2(make_float2(s[mt][u][0], s[mt][u][1]), make_float2(unit[mt][0], unit[mt][0]), make_float2(ma, ma));
          float2 d = tc::fma2(make_float2(s[mt][u][2], s[mt][u][3]), make_float2(unit[mt][1], unit[mt][1]), make_float2(mb, mb));
          a = make_float2(ex2(a.x), ex2(a.y));
          d = make_float2(ex2(d.x), ex2(d.y));
          pa[mt][2 * u] = pack_h2(a.x, a.y);
          pa[mt][2 * u + 1] = pack_h2(d.x, d.y);
          sum[0] = u ? tc::add2(sum[0], a) : a;
          sum[1] = u ? tc::add2(sum[1], d) : d;
        }
        l_run[mt][0] += sum[0].x + sum[0].y;
        l_run[mt][1] += sum[1].x + sum[1].y;
      }

      // weighted V
      const uint16_t* const vsk = vs + 16 * ks + 2 * j;
      uint32_t ps[MT][4];
#pragma unroll
      for (int c = 0; c < C::CHUNKS; c += 2) {
        uint32_t v[4];
        const int mm = lane >> 3, tok = 16 * ks + ((mm & 1) << 3) + (lane & 7);
        ldsm_x4_t(vc + C::at(tok, c + (mm >> 1)), v[0], v[1], v[2], v[3]);
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          const int chunk = c + cc, g = chunk >> lcpg;
          if ((chunk & cmask) == 0) {  // a new group: its scales, and its zero-points' sums
            const __half2 lo = u32_as_h2(*reinterpret_cast<const uint32_t*>(vsk + g * C::VROW));
            const __half2 hi = u32_as_h2(*reinterpret_cast<const uint32_t*>(vsk + g * C::VROW + 8));
            uint32_t z0 = 0u, z1 = 0u;
            if (KIND == 0 && rho == g) {
              z0 = *reinterpret_cast<const uint32_t*>(vz + g * C::VROW + 16 * ks + 2 * j);
              z1 = *reinterpret_cast<const uint32_t*>(vz + g * C::VROW + 16 * ks + 8 + 2 * j);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              ps[mt][0] = h2_as_u32(__hmul2(u32_as_h2(pa[mt][0]), lo));
              ps[mt][1] = h2_as_u32(__hmul2(u32_as_h2(pa[mt][1]), lo));
              ps[mt][2] = h2_as_u32(__hmul2(u32_as_h2(pa[mt][2]), hi));
              ps[mt][3] = h2_as_u32(__hmul2(u32_as_h2(pa[mt][3]), hi));
              if constexpr (KIND == 0) mma16816(cz[mt], ps[mt][0], ps[mt][1], ps[mt][2], ps[mt][3], z0, z1);
            }
          }
          const uint32_t x0 = v[2 * cc], x1 = v[2 * cc + 1];  // keys 0-7, 8-15 of the sixteen
          uint32_t lo[4], hi[4];
          if constexpr (BITS == 4) {
            nib8_to_h2<KIND == 1, true>(x0, lo, lut);
            nib8_to_h2<KIND == 1, true>(x1, hi, lut);
          } else {
            lo[0] = byte2_to_h2_sub<0x4240>(x0), lo[1] = byte2_to_h2_sub<0x4341>(x0);
            hi[0] = byte2_to_h2_sub<0x4240>(x1), hi[1] = byte2_to_h2_sub<0x4341>(x1);
          }
#pragma unroll
          for (int f = 0; f < C::FPC; ++f)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              mma16816(o[mt][chunk * C::FPC + f], ps[mt][0], ps[mt][1], ps[mt][2], ps[mt][3], lo[f], hi[f]);
        }
      }
    }
    __syncwarp();
    // the stage's next tile; the masks move up by one
    const uint32_t next = issue(it + C::STAGES, stage);
#pragma unroll
    for (int k = 0; k + 1 < C::STAGES; ++k) mask_of[k] = mask_of[k + 1];
    mask_of[C::STAGES - 1] = next;
    stage = stage + 1 == C::STAGES ? 0 : stage + 1;
  }
  cp_async_wait<0>();
  if (unmapped && p.status) atomicOr(p.status, KVQ_FLAG_BLOCK_TABLE);

  // ---- the sums, zero-points taken off: in place, four (INT8: two) channels of
  // a row side by side ----
  float up[C::MAXNG];
#pragma unroll
  for (int g = 0; g < C::MAXNG; ++g) up[g] = ScalePower::inverse(power >> (8 * g) & 255u);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l_run[mt][e] += __shfl_xor_sync(0xffffffffu, l_run[mt][e], 1);
      l_run[mt][e] += __shfl_xor_sync(0xffffffffu, l_run[mt][e], 2);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int f = n % C::FPC, g = (n / C::FPC) >> lcpg;
      const float back = of_chunk(up, n / C::FPC), fac = back * (kSub * (BITS == 4 && KIND == 0 && (f & 1) ? 0.0625f : 1.f));
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // group g's sum lies in column g: lane g / 2, one of its two
        float corr = 0.f;
        if constexpr (KIND == 0) {
          const float c0 = __shfl_sync(0xffffffffu, cz[mt][2 * e], (rho << 2) | (g >> 1));
          const float c1 = __shfl_sync(0xffffffffu, cz[mt][2 * e + 1], (rho << 2) | (g >> 1));
          corr = ((g & 1) ? c1 : c0) * back;
        }
        o[mt][n][2 * e] = o[mt][n][2 * e] * fac - corr;
        o[mt][n][2 * e + 1] = o[mt][n][2 * e + 1] * fac - corr;
      }
    }
  }
  // where channels chunk DPC + FPC (2j + c) .. of row mt 16 + rho + 8 e go
  auto put = [&](float* to, int mt, int chunk, int e, int c) {
    const int n = chunk * C::FPC, i = 2 * e + c;
    if constexpr (C::FPC == 4)
      *reinterpret_cast<float4*>(to) = make_float4(o[mt][n][i], o[mt][n + 1][i], o[mt][n + 2][i], o[mt][n + 3][i]);
    else
      *reinterpret_cast<float2*>(to) = make_float2(o[mt][n][i], o[mt][n + 1][i]);
  };
  auto partial_at = [&](int r) {
    return ((long long)toks[r] * p.Hq + (long long)kvh * p.G + (r0 + r) % p.G) * p.splits + split;
  };
  __syncthreads();  // every warp is done with its pipeline: the join takes its place
  float* const red = reinterpret_cast<float*>(pipe);  // [warp][row][RED]
  float2* const ml = reinterpret_cast<float2*>(red + kWarps * C::ROWS * C::RED);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = warp * C::ROWS + mt * 16 + rho + 8 * e;
      if (j == 0) ml[r] = make_float2(m_ref[mt][e], l_run[mt][e]);
#pragma unroll
      for (int chunk = 0; chunk < C::CHUNKS; ++chunk)
#pragma unroll
        for (int c = 0; c < 2; ++c) put(red + r * C::RED + chunk * C::DPC + C::FPC * (2 * j + c), mt, chunk, e, c);
    }
  __syncthreads();
  for (int i = threadIdx.x; i < C::ROWS * (D / 4); i += kWarps * 32) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    if (r0 + r >= live_rows) break;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * C::ROWS + r].x);
    const float base = M == -INFINITY ? 0.f : M;
    float l = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 y = ml[w * C::ROWS + r];
      const float4 a = *reinterpret_cast<const float4*>(red + (w * C::ROWS + r) * C::RED + d);
      const float f = ex2(y.x - base);
      l = fmaf(f, y.y, l);
      v = make_float4(fmaf(f, a.x, v.x), fmaf(f, a.y, v.y), fmaf(f, a.z, v.z), fmaf(f, a.w, v.w));
    }
    const long long at = partial_at(r);
    float4* to = reinterpret_cast<float4*>(p.ws_o + at * D + d);
    if (KVQ_IN(geo, KVQ_ARRAY_WORKSPACE, to, 16)) *to = v;
    float2* tml = reinterpret_cast<float2*>(p.ws_ml) + at;
    if (d == 0 && KVQ_IN(geo, KVQ_ARRAY_WORKSPACE, tml, 8)) *tml = make_float2(M, l);
  }
}

template <int BITS, int KIND, int D, int MT>
cudaError_t run(const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream) {
  using C = RowCfg<BITS, KIND, D, MT>;
  static KernelSetup setup;
  int occ = 0;
  const cudaError_t e = setup_kernel(rows_kernel<BITS, KIND, D, MT>, setup, kWarps * 32, C::SMEM, &occ);
  if (e != cudaSuccess) return e;
  if (plan) {
    plan->tile_rows = C::ROWS;
    plan->occ = occ;
    plan->lift = kLiftRows;
    return cudaSuccess;
  }
  const long long each = (long long)p->num_new * p->G;
  const dim3 grid((unsigned)(prefix_tiles_bound(p->plan.B, p->plan.N, each, C::ROWS) * p->splits), p->v.geom.Hkv);
  return launch_pdl(rows_kernel<BITS, KIND, D, MT>, grid, dim3(kWarps * 32), C::SMEM, stream, *p);
}

// One instance file per format calls this for its BITS and KIND; mt: 16 rows
// or 32.
template <int BITS, int KIND>
cudaError_t run_rows(int D, int mt, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream) {
  if (D == 64) return mt == 1 ? run<BITS, KIND, 64, 1>(p, plan, stream) : run<BITS, KIND, 64, 2>(p, plan, stream);
  return mt == 1 ? run<BITS, KIND, 128, 1>(p, plan, stream) : run<BITS, KIND, 128, 2>(p, plan, stream);
}
}  // namespace rows
}  // namespace kvq
