// Attention of several new tokens over the cache on the fifth-generation
// tensor cores (head_dim 64 and 128, every per-token format).
//
// Rows.  As in kvq_extend.cu the rows of a tile are (new token, head of the
// KV head's group) pairs.  A CTA takes two tiles of 128 rows of one KV head
// and one split of the keys, in steps of 64 keys; a call of at most 128 rows
// takes one tile in two streams that share the key tiles out between them and
// are joined at the end (NQ = 1):
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
// Warps.  0 and 3 issue the MMAs, a tile each; 1 and 2 copy codes and headers
// to a ring in shared memory; from 4 on softmax, a row per thread (four warps a
// tile); the eight producers behind turn the ring's codes into fp16 in the
// tensor core's swizzled layout, four of them K's and four V's (fp16 caches:
// they copy rows).  One tile's (or stream's) softmax runs under the other's
// products.
//
// What bounds it.  256 rows of 128 channels over codes: the tensor core, 2048
// cycles a 64-key step of about 2600 (K and V each in two parts): INT4, 4096
// tokens after 12288, 32 / 8 heads (the late chunk below), 1.03 ms by itself
// (profiler), 937 TFLOP/s of the formula's; calls in turn, each with the merge
// of its two splits (47 us), 1.07 to 1.13 ms by the inputs and the power.  Over
// fp16: the softmax, about 2000 cycles a step (512 of them a warp's exponentials
// alone, and two warps share a scheduler's unit) where the products take 1280:
// 0.88 ms, 1088 TFLOP/s, calls in turn.  At most 128 rows: the conversion, about
// 1300 of 1900 cycles a step, bound by its own latency with two warps a
// scheduler: 17 tokens over 32768 (INT8) 42 us by itself, 44 in turn.
// (Figures "a -> b" below are of the step that brought them: calls in turn, on
// one set of inputs.)
//
// Precision.  q - z is a whole number of up to 12 bits (exact in fp16 up to
// 2048) and s has 11, so x_hat = (q - z) s has up to 23 and is, like s, a whole
// number of 2^-24: K and V enter as sums of two fp16 numbers, hi = fp16(x_hat)
// and lo = x_hat - hi, which fp16 holds exactly (at most 2^11 units of s's last
// bit); two products into one accumulator.  (NF4: a level times s has bits below
// 2^-24 where s < 2; lo is off by up to 2^-25.)  With hi alone for both, the outputs of keys with large
// channels (INT4 groups of 32, 10x channels) are off by 1.0e-3 to 1.3e-3
// relative, five times what rounding the output costs (2.1e-4); with K's lo by
// 3.2e-4, with both by 2.7e-4: the output's own rounding and that of the
// probabilities to fp16, whose errors average out over the keys.  Scores, sums
// and O are fp32.  fp16 caches are exact as they are.
//
// Reference maximum.  m moves only when a tile's maximum exceeds it by 2^8,
// so O in tensor memory is rescaled rarely.  P carries a factor 2^7 that the
// division by the sum takes out: at most 2^15 it stays within fp16, and keys
// 2^-21 of the largest still have all 11 bits (a long context can hold enough
// of them to matter).
//
// Order of the MMAs.  One lane issues PV(j) and then QK(j + 1) of a tile,
// and MMAs run in the order issued: S may be overwritten as soon as QK(j + 1)
// is issued, and when its completion is seen PV(j) is complete too, so the
// softmax may rescale O until it hands over P(j + 1).  PV(j) starts with the
// first 32 keys' P (late chunk below: 1.14 -> 1.05 ms, fp16 1.00 -> 0.90).
// Where tensor memory holds two S per tile (SB), QK(j + 2) follows PV(j)
// instead, and a rescale waits for PV(j - 1) by itself.
#pragma once

#include "kvq_decode_fast.cuh"
#include "kvq_load.cuh"
#include "kvq_rope.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace ext {

using fast::ex2;

constexpr int kKeys = 64;
template <int N>
struct Int {
  static constexpr int value = N;
};
constexpr float kLazy = 8.f;  // log2 units the maximum may lead the reference
constexpr float kLift = 7.f;  // log2 of the factor in P, l and O

// KIND: 0 uniform codes (asymmetric or symmetric), 1 NF4, 2 fp16
template <int BITS, int KIND, int D, int NQ>
struct Cfg {
  static constexpr bool LO = KIND != 2;
  static constexpr bool DUAL = NQ == 1;           // one tile of rows, the key tiles shared between two streams
  static constexpr int ROWS = 128 * NQ;
  static constexpr int SOFT = 8;                  // softmax warps
  static constexpr int PROD = 8;                  // producer warps
  static constexpr int LOAD = LO ? 2 : 1;         // loader warps, K and V (fp16: the warp that passes stages on)
  // warps 0 and 3 issue the MMAs, 1 .. LOAD load; softmax from 4 on (a warp reads
  // the tensor memory lanes of its number modulo 4), producers behind
  static constexpr int SOFT0 = 4, PROD0 = SOFT0 + SOFT, WARPS = PROD0 + PROD;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int MAT = kKeys * D * 2;       // one fp16 tile
  // A stage holds K and V of a key tile, hi and lo.  Quantized formats fill
  // and free the two by themselves, so that K of a tile to come is converted
  // under the softmax, and two stages do.
  static constexpr int HALF = (LO ? 2 : 1) * MAT, STAGE = 2 * HALF;
  static constexpr int STAGES = !LO ? 4 : D == 128 ? 2 : 3;
  static constexpr int K_STEP = LO ? HALF : STAGE, V_AT = LO ? STAGES * HALF : HALF, V_STEP = K_STEP;
  // q passes through the V tiles (fp16: the stages) from this one on
  static constexpr int Q_STAGE = STAGES - (SOFT * 4096 + V_STEP - 1) / V_STEP;
  static constexpr int Q_AT = (LO ? V_AT : 0) + Q_STAGE * V_STEP;
  static constexpr int SEGS = D / 32;             // 32-channel segments of a row
  // A producer warp works on items: the whole rows of KPI keys of K or V, a
  // segment per lane.
  static constexpr int KPI = 32 / SEGS;
  static constexpr int ITEMS = 2 * kKeys / KPI;   // of a tile
  static constexpr int MINE = ITEMS / PROD;       // of a warp and tile
  // Codes and headers arrive in a ring of DEPTH tiles by bulk copies (one to
  // three tiles of latency covered); fp16 rows go to their stage.
  static constexpr int DEPTH = !LO ? 0 : D == 128 ? (BITS == 8 ? 3 : 4) : 6;
  static constexpr int CODES = LO ? kKeys * D * BITS / 8 : 0;  // bytes of a tile's K (or V) codes
  static constexpr int HDR = kKeys * D / 4 + 16;  // most bytes of one header array, from a 16-byte boundary on
  static constexpr int RAW = LO ? 2 * CODES + 4 * HDR : 0;     // K codes, V codes, K scale, K zero, V scale, V zero
  // arrivals that fill a ring slot (fp16: a stage's copies and key masks), and a stage
  static constexpr int RAW_FULL = LO ? LOAD : PROD * 32, FULL = LO ? PROD / 2 : 1;
  static constexpr int SLOTS = LO ? DEPTH : STAGES;
  // Two S per tile where tensor memory has room for them: at head_dim 64, and
  // at 128 with q in shared memory, which only fp16 caches leave the room for.
  static constexpr bool Q_SMEM = !LO && D == 128 && !DUAL;
  static constexpr int SB = !DUAL && (D == 64 || Q_SMEM) ? 2 : 1;
  // Whether the tiles' MMA warps take turns: with one S per tile, which keeps
  // the tiles a softmax apart; with two they only wait for one another (fp16
  // 0.89 -> 0.88 ms, prompts of 2048 219 -> 211 us without).
  static constexpr bool TURNS = !DUAL && SB == 1;
  // tensor memory columns: per tile S (64 each, P in its place), O (D), Q (D / 2)
  static constexpr uint32_t COL_S = 0, COL_O = 2 * SB * kKeys, COL_Q = COL_O + 2 * D, COLS = 512;
  static constexpr int Q_BYTES = Q_SMEM ? 2 * 128 * D * 2 : 0;  // behind the ring, on a 1024-byte boundary
  static_assert(!Q_SMEM || DEPTH == 0, "q follows the stages");
  static constexpr size_t SMEM = (size_t)STAGES * STAGE + (size_t)DEPTH * RAW + Q_BYTES + 1024 + 2048;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(COL_Q + (Q_SMEM ? 0 : 2 * D / 2) <= COLS, "tensor memory");
  static_assert((size_t)STAGES * STAGE >= (DUAL ? (size_t)128 * D * 4 : 0) + SOFT * 4096, "scratch in the stages");
  // channel held at place i of an eight-channel chunk (the unpacking leaves
  // 4-bit and 2-bit codes as pairs (i, i + 4))
  static constexpr bool PAIRED = BITS <= 4;
  __host__ __device__ static constexpr int channel(int i) { return PAIRED ? (i >> 1) + 4 * (i & 1) : i; }
};

// Barriers and flags behind the stages
constexpr int kMaxDepth = 6;
template <int STAGES>
struct Shared {
  unsigned long long raw_full[kMaxDepth], raw_empty[kMaxDepth];
  uint32_t raw_ok[kMaxDepth][2];
  unsigned long long full[2][STAGES], empty[2][STAGES];  // K, V (fp16: full[0] and empty[1], both at once)
  unsigned long long q_full[2], s_full[4], p_half[4], p_full[4], o_full[2], o_step[2], turn[2], merge;  // s, p: [tile][S]
  unsigned long long done[2];  // a tile's (stream's) products when its warp gives up
  int loaded[2];               // key tiles whose K, V copies were issued
  float2 ml[128];           // the second stream's maximum and sum per row
  uint32_t ok[2 * STAGES][2];  // per key: mapped and before the end (a K tile is freed before the softmax has read these)
  alignas(4) uint8_t bad[STAGES][kKeys];  // per key: V held an infinity or NaN (set to zero)
  uint32_t tmem;
  int stop;
};

// ---- producers --------------------------------------------------------

// The codes and headers of 32 channels of one key.
template <int BITS>
struct Seg {
  uint32_t w[BITS == 16 ? 1 : BITS];  // 32 * BITS / 32 words
  uint32_t s[2], z[2];                // up to four fp16 scales and zeros
};

// Reads one lane's segment from the ring: `codes` of the item's first key,
// scales and zeros of its key.  Lanes of the upper 64 channels take their
// chunks in the order 2, 3, 0, 1 (swap), so that the stores of a warp fall
// into different banks.
template <int BITS, int KIND, int NG>
__device__ __forceinline__ void take_item(const uint8_t* codes, const uint8_t* s, const uint8_t* z, bool zeros,
                                          int lane, bool swap, Seg<BITS>& x) {
  constexpr int SB = 4 * BITS;
  if constexpr (SB == 8) {
    const uint2 t = *reinterpret_cast<const uint2*>(codes + lane * 8);
    x.w[0] = swap ? t.y : t.x;
    x.w[1] = swap ? t.x : t.y;
  } else {
    uint32_t w[BITS];
#pragma unroll
    for (int i = 0; i < SB / 16; ++i) {
      const uint4 t = *reinterpret_cast<const uint4*>(codes + lane * SB + i * 16);
      w[4 * i] = t.x, w[4 * i + 1] = t.y, w[4 * i + 2] = t.z, w[4 * i + 3] = t.w;
    }
#pragma unroll
    for (int i = 0; i < BITS; ++i) x.w[i] = swap ? w[(i + BITS / 2) % BITS] : w[i];
  }
  x.s[0] = x.s[1] = x.z[0] = x.z[1] = 0;
  if constexpr (NG == 1) {
    x.s[0] = *reinterpret_cast<const unsigned short*>(s);
    if (zeros) x.z[0] = *reinterpret_cast<const unsigned short*>(z);
  } else if constexpr (NG == 2) {
    x.s[0] = *reinterpret_cast<const uint32_t*>(s);
    if (zeros) x.z[0] = *reinterpret_cast<const uint32_t*>(z);
    if (swap) x.s[0] = fast::prmt_b32(x.s[0], 0u, 0x1032u), x.z[0] = fast::prmt_b32(x.z[0], 0u, 0x1032u);
  } else {
    uint2 t = *reinterpret_cast<const uint2*>(s);
    x.s[0] = swap ? t.y : t.x, x.s[1] = swap ? t.x : t.y;
    if (zeros) {
      t = *reinterpret_cast<const uint2*>(z);
      x.z[0] = swap ? t.y : t.x, x.z[1] = swap ? t.x : t.y;
    }
  }
}

__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// A group's conversion: d = q - z from the unpacked codes, hi = fp16(d s).
struct Group {
  __half2 s, off, off16;  // scale; -(1024 + z); -(64 + z)
  __half z;
  bool plain;             // 1024 + z a number that fp16 holds, no product beyond fp16
};
template <int BITS, int KIND>
__device__ __forceinline__ Group group_of(uint32_t sw, uint32_t zw, int sym) {
  Group g;
  g.s = as_h2(fast::prmt_b32(sw, 0u, 0x1010u));
  g.z = __ushort_as_half(0);
  g.plain = true;
  g.off = g.off16 = g.s;
  if constexpr (KIND == 0) {
    // (symmetric codes: z = 2^(bits-1), as fp16)
    constexpr uint32_t half_range = BITS == 2 ? 0x40004000u : BITS == 4 ? 0x48004800u : 0x58005800u;
    const __half2 z = as_h2(sym ? half_range : fast::prmt_b32(zw, 0u, 0x1010u));
    g.z = __low2half(z);
    g.off = __hneg2(__hadd2(z, as_h2(fast::kH1024)));
    g.off16 = __hneg2(__hadd2(z, as_h2(0x54005400u)));
    const __half2 az = __habs2(z);
    const __half2 most = __hmul2(__hadd2(az, as_h2(BITS == 8 ? 0x5BF85BF8u : BITS == 4 ? 0x4B804B80u : 0x42004200u)), g.s);
    g.plain = __hle(__low2half(az), __ushort_as_half(0x6400)) && __hlt(__low2half(most), __ushort_as_half(0x7BD0));
  }
  return g;
}

// d of the eight codes of chunk ch of a segment, in fp16 pairs
template <int BITS, int KIND>
__device__ __forceinline__ void codes8(const Seg<BITS>& x, int ch, const Group& g, const uint32_t (&lut)[4],
                                       __half2 (&d)[4]) {
  if constexpr (KIND == 1) {
    uint32_t o[4];
    fast::nib8_to_h2_nf4(x.w[ch], o, lut);
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = as_h2(o[i]);
  } else if constexpr (BITS == 4) {
    // low nibbles as 1024 + q; high ones, left in place, as 1024 + 16 q
    const __half2 k16 = as_h2(fast::kH1_16);
    const uint32_t w = x.w[ch], v = w >> 8;
    d[0] = __hadd2(as_h2(fast::and_or(w, 0x000F000Fu, fast::kH1024)), g.off);
    d[1] = __hfma2(as_h2(fast::and_or(w, 0x00F000F0u, fast::kH1024)), k16, g.off16);
    d[2] = __hadd2(as_h2(fast::and_or(v, 0x000F000Fu, fast::kH1024)), g.off);
    d[3] = __hfma2(as_h2(fast::and_or(v, 0x00F000F0u, fast::kH1024)), k16, g.off16);
  } else if constexpr (BITS == 2) {
    const uint32_t w = (x.w[ch >> 1] >> (16 * (ch & 1))) & 0xFFFFu;
    const uint32_t v = (w & 0xFFu) | ((w & 0xFF00u) << 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = __hadd2(as_h2(fast::and_or(v >> (2 * i), 0x00030003u, fast::kH1024)), g.off);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      d[i] = __hadd2(as_h2(fast::prmt_b32(x.w[2 * ch + (i >> 1)], 0x64646464u, (i & 1) ? 0x4342u : 0x4140u)), g.off);
  }
}

// One segment to fp16, hi and lo, at its places in the tile: blocks
// of 64 channels, [key][128 bytes], 16-byte chunks XORed with the key.
// NG: groups in the segment.  swap (0 or 2): x holds its chunks in that order.
template <int BITS, int KIND, int NG, int UNROLL>
__device__ __forceinline__ void store_seg(const Seg<BITS>& x, int key, int seg, int sym, int swap, uint8_t* hi,
                                          uint8_t* lo, const uint32_t (&lut)[4]) {
  const uint32_t base = (uint32_t)((seg >> 1) * (kKeys * 128) + key * 128);
  const uint32_t turn = (uint32_t)(((seg & 1) * 4) ^ swap ^ (key & 7));
  Group g[NG];
  bool plain = true;
#pragma unroll
  for (int n = 0; n < NG; ++n) {
    g[n] = group_of<BITS, KIND>(x.s[n >> 1] >> (16 * (n & 1)), x.z[n >> 1] >> (16 * (n & 1)), sym);
    plain = plain && g[n].plain;
  }
  if (plain) {
    // A small loop, its words shifted on.  One chunk a turn where the softmax
    // of 256 rows runs beside it, whose code shares the instruction caches
    // (late prompt chunk: 1.135 ms, two a turn 1.163); two a turn where few
    // rows wait for the conversion (16 x 5 tokens over ragged 8000, calls in turn
    // on one cache: 98 us, one a turn 105).
    Seg<BITS> y = x;
    Group gc = g[0];
#pragma unroll UNROLL
    for (int ch = 0; ch < 4; ++ch) {
      __half2 d[4], v[4];
      codes8<BITS, KIND>(y, 0, gc, lut, d);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __hmul2_rn(d[i], gc.s);
      const uint32_t at = base + ((turn ^ ch) << 4);
      *reinterpret_cast<uint4*>(hi + at) = make_uint4(as_u32(v[0]), as_u32(v[1]), as_u32(v[2]), as_u32(v[3]));
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __hfma2(d[i], gc.s, __hneg2(v[i]));  // exact inside: what hi left
      *reinterpret_cast<uint4*>(lo + at) = make_uint4(as_u32(v[0]), as_u32(v[1]), as_u32(v[2]), as_u32(v[3]));
      if constexpr (BITS == 2) {
        y.w[0] = __funnelshift_r(y.w[0], y.w[1], 16);
        y.w[1] >>= 16;
      } else {
#pragma unroll
        for (int i = 0; i + BITS / 4 < BITS; ++i) y.w[i] = y.w[i + BITS / 4];
      }
      if constexpr (NG > 1) {
        if (NG == 4 || ch == 1) {
          y.s[0] = __funnelshift_r(y.s[0], y.s[1], 16), y.s[1] >>= 16;
          y.z[0] = __funnelshift_r(y.z[0], y.z[1], 16), y.z[1] >>= 16;
          gc = group_of<BITS, KIND>(y.s[0], y.z[0], sym);
        }
      }
    }
  } else {  // far zero-points and scales near fp16's end, in fp32
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) {
      const Group& gc = g[ch / (4 / NG)];
      uint32_t h[4], l[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int q = BITS <= 4 ? i + 4 * e : 2 * i + e;  // the code at this place
          const uint32_t c = BITS == 8   ? x.w[2 * ch + (q >> 2)] >> (8 * (q & 3))
                             : BITS == 4 ? x.w[ch] >> (4 * q)
                                         : x.w[ch >> 1] >> (16 * (ch & 1) + 2 * q);
          a[e] = ((float)(c & ((1u << BITS) - 1u)) - __half2float(gc.z)) * __low2float(gc.s);
        }
        h[i] = pack_sat(a[0], a[1]);
        l[i] = pack_rest(a[0], a[1], h[i]);
      }
      const uint32_t at = base + ((turn ^ ch) << 4);
      *reinterpret_cast<uint4*>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
    }
  }
}

__device__ __forceinline__ bool nonfinite2(uint32_t w) {
  return (w & 0x7C00u) == 0x7C00u || (w & 0x7C000000u) == 0x7C000000u;
}

// ---- the kernel -------------------------------------------------------

// (ExtendParams::started)
__device__ __forceinline__ void end_after_prefixes(const ExtendParams& p) {
  if (p.started && threadIdx.x == 0 && blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1 && blockIdx.z == gridDim.z - 1)
    wait_beside(p.started, true);
}

// PRE: over shared prefixes (rows of all members of a prefix, which see all of
// its keys; partials only).
template <int BITS, int KIND, int D, int NQ, bool PRE>
__global__ void __launch_bounds__((Cfg<BITS, KIND, D, NQ>::THREADS), 1)
    extend_tc_kernel(const __grid_constant__ ExtendParams p) {
  using C = Cfg<BITS, KIND, D, NQ>;
  constexpr int ROWS = C::ROWS, STEP = C::DUAL ? 2 : 1;  // key tiles from one of a stream's to its next
  if (!PRE) pdl_launch_dependents();
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (tc::smem_addr(raw) & 1023)) & 1023);
  auto& sh = *reinterpret_cast<Shared<C::STAGES>*>(smem + C::STAGES * C::STAGE + C::DEPTH * C::RAW + C::Q_BYTES);
  const CacheGeom& c = p.v.geom;
  const int warp = tc::uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int kvh = blockIdx.y;
  const int split = blockIdx.x % p.splits;
  if constexpr (PRE) {
    pdl_wait();
    say_started(p.started);
  } else {
    start_beside(p.started);
  }

  int b, before, end, all_see;  // all_see: every row sees the positions up to here
  PrefixTile pt{};              // (PRE)
  int own_tok = 0;              // (PRE) the token of this lane's row of the tile
  long long live_rows, r0;
  if constexpr (PRE) {
    pt = prefix_tile(p.plan, blockIdx.x / p.splits, p.num_new * p.G, ROWS);
    b = tc::uniform(pt.n);
    if (b < 0) return;
    end = tc::uniform(prefix_len(p.plan, b, p.len_limit));
    if (split * p.chunk >= end) return;  // the join knows which splits hold keys
    r0 = (long long)tc::uniform(pt.tile) * ROWS;
    const int soft = max(warp - C::SOFT0, 0) & 7;  // a softmax warp's rows
    const long long own = r0 + (C::DUAL ? (soft & 3) : soft) * 32 + lane;
    live_rows = tc::uniform(prefix_rows(p.plan, pt, p.new_lens, p.num_new, p.G, own, &own_tok));
    if (r0 >= live_rows) return;
    before = all_see = 0x7fffffff;
  } else {
    // row tiles last first: with a causal mask they see the most keys
    const int tile = gridDim.x / p.splits - 1 - blockIdx.x / p.splits;
    b = blockIdx.z;
    before = tc::uniform(checked_len(c, p.lens_before, b, -1));
    const int n_raw = tc::uniform(new_rows_of(p.new_lens, b, p.num_new));
    const int n = max(n_raw, 0);
    const bool fits = before >= 0 && n_raw >= 0 && (long long)before + n <= p.len_limit;
    if (!fits && threadIdx.x == 0 && blockIdx.x == 0 && kvh == 0 && p.status) atomicOr(p.status, KVQ_FLAG_SEQ_LEN);
    live_rows = (long long)n * p.G;
    r0 = (long long)tile * ROWS;
    if (r0 >= live_rows) {
      end_after_prefixes(p);
      return;
    }
    const int L = fits ? before + n : 0;
    const int t_first = (int)(r0 / p.G);
    const int t_last = (int)((min(r0 + ROWS, live_rows) - 1) / p.G);
    end = L ? before + t_last + 1 : 0;
    all_see = L ? before + t_first : -1;
  }
  const int k0 = split * p.chunk, k1 = min(end, k0 + p.chunk);
  const int tiles = k1 > k0 ? (k1 - k0 + kKeys - 1) / kKeys : 0;
  const int nq = (!C::DUAL && live_rows - r0 <= 128) ? 1 : 2;  // tiles of rows, or streams

  static_assert(sizeof(Shared<C::STAGES>) <= 2048, "room behind the stages");
  const uint32_t bars = tc::smem_addr(&sh);
  // which S a tile's n-th step uses, and its barriers' phase
  auto buf = [](int n) { return C::SB == 2 ? n & 1 : 0; };
  auto phase = [](int n) { return C::SB == 2 ? n >> 1 & 1 : n & 1; };
  auto full = [&](int v, int s) { return bars + (uint32_t)offsetof(Shared<C::STAGES>, full) + 8 * (v * C::STAGES + s); };
  auto empty = [&](int v, int s) { return bars + (uint32_t)offsetof(Shared<C::STAGES>, empty) + 8 * (v * C::STAGES + s); };
  auto raw_full = [&](int s) { return bars + (uint32_t)offsetof(Shared<C::STAGES>, raw_full) + 8 * s; };
  auto raw_empty = [&](int s) { return bars + (uint32_t)offsetof(Shared<C::STAGES>, raw_empty) + 8 * s; };
  auto q_full = [&](int i) { return bars + (uint32_t)offsetof(Shared<C::STAGES>, q_full) + 8 * i; };
  auto s_full = [&](int i, int n) { return bars + (uint32_t)offsetof(Shared<C::STAGES>, s_full) + 8 * (2 * i + buf(n)); };
  auto o_step = [&](int i) { return bars + (uint32_t)offsetof(Shared<C::STAGES>, o_step) + 8 * i; };
  auto p_half = [&](int i, int n) { return bars + (uint32_t)offsetof(Shared<C::STAGES>, p_half) + 8 * (2 * i + buf(n)); };
  auto p_full = [&](int i, int n) { return bars + (uint32_t)offsetof(Shared<C::STAGES>, p_full) + 8 * (2 * i + buf(n)); };
  auto turn = [&](int i) { return bars + (uint32_t)offsetof(Shared<C::STAGES>, turn) + 8 * i; };
  const uint32_t merge = bars + (uint32_t)offsetof(Shared<C::STAGES>, merge);
  auto o_full = [&](int i) { return bars + (uint32_t)offsetof(Shared<C::STAGES>, o_full) + 8 * i; };
  auto done = [&](int i) { return bars + (uint32_t)offsetof(Shared<C::STAGES>, done) + 8 * i; };
  volatile int* stop = &sh.stop;
  // (debug builds: a wait that is to run out)
  auto runs_out = [&](int wait, int j) {
    if (!KVQ_FAILS(c, wait, j)) return false;
    *stop = 1;
    return true;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2 * C::STAGES; ++s) {
      tc::mbar_init(full(0, s), C::FULL);
      tc::mbar_init(empty(0, s), C::DUAL ? 1 : nq);
    }
    for (int s = 0; s < C::SLOTS; ++s) {
      tc::mbar_init(raw_full(s), C::RAW_FULL);
      tc::mbar_init(raw_empty(s), C::PROD);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(q_full(i), 128);
      for (int n = 0; n < C::SB; ++n) {
        tc::mbar_init(s_full(i, n), 1);
        tc::mbar_init(p_half(i, n), 4);
        tc::mbar_init(p_full(i, n), 4);
      }
      tc::mbar_init(o_step(i), 1);
      tc::mbar_init(o_full(i), 1);
      tc::mbar_init(turn(i), 1);
      tc::mbar_init(done(i), 1);
      sh.loaded[i] = 0;
    }
    tc::mbar_init(merge, 4);
    sh.stop = 0;
    tc::mbar_init_fence();
  }
  if (warp == 0) tc::tmem_alloc(tc::smem_addr(&sh.tmem), C::COLS);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tc::uniform(sh.tmem);

  // where a dense header array's rows begin in their first 16 bytes (the same for every tile)
  const int mis = c.layout == KVQ_DENSE
                      ? (int)((((long long)b * c.Hkv + kvh) * c.slots + k0) * (2 * c.ngroups) & 15) : 0;
  // row of a position of this split: -1 behind its end, -2 unmapped
  auto row_of = [&](int pos) -> long long {
    if (pos >= k1) return -1;
    const long long row = token_row(c, b, kvh, pos);
    return row < 0 ? -2 : row;
  };
  auto note_keys = [&](uint32_t* to, int j) {  // which keys of tile j count; one warp
    const int pos = k0 + j * kKeys + lane;
    const long long r0k = row_of(pos), r1k = row_of(pos + 32);
    const uint32_t a = __ballot_sync(0xffffffffu, r0k >= 0), d = __ballot_sync(0xffffffffu, r1k >= 0);
    if (lane == 0) to[0] = a, to[1] = d;
    if ((r0k == -2 || r1k == -2) && p.status) atomicOr(p.status, KVQ_FLAG_BLOCK_TABLE);
  };

  if (warp >= C::SOFT0 && warp < C::PROD0) {
    // ------------------------------------------------------ softmax rows
    const int i = (warp - C::SOFT0) >> 2;
    const int row0 = (int)r0 + (C::DUAL ? 0 : i * 128) + (warp & 3) * 32;  // the warp's first row
    const int r = row0 + lane;
    const bool live = r < live_rows;
    const bool any_live = row0 < live_rows;
    // 32 rows of 128 bytes in the stages' memory, before they are first
    // filled and after the last product
    uint8_t* scratch = smem + C::Q_AT + (warp - C::SOFT0) * 4096;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts0 = tmem + lanes + C::COL_S + i * C::SB * kKeys;
    const uint32_t to = tmem + lanes + C::COL_O + i * D;
    const uint32_t tq = tmem + lanes + C::COL_Q + i * (D / 2);
    // this lane's row in q, out and the partials
    const int t = live ? r / p.G : 0;
    const long long orow = (PRE ? (long long)own_tok : (long long)b * p.num_new + t) * p.Hq + (long long)kvh * p.G +
                           (live ? r % p.G : 0);
    // (rows behind the last take part with q = 0 and are not written)
    const int last = live && !PRE ? before + t : 0x7fffffff;
    const int mine = C::DUAL ? (tiles + 1 - i) / 2 : tiles;  // this stream's key tiles
    if (i < nq && mine) {
      // q to tensor memory, channels in the order the keys are unpacked in: 64
      // channels at a time through the warp's scratch, whole lines from global
      // memory (a lane reading its own row takes a line's tag per lane and
      // load: 7000 cycles for the tile)
      // (Set-up and writing out run once a block, their instructions fetched
      // anew: rolled loops.)
      uint4 x[D / 64][8];
#pragma unroll
      for (int it = 0; it < 8; ++it) {  // (all loads, then the stores)
        long long row;
        if constexpr (PRE || !C::LO) {
          row = __shfl_sync(0xffffffffu, orow, it * 4 + (lane >> 3));
        } else {  // (late chunks over codes: 1095 us by shuffles, 1070 so)
          const int own = min(row0 + it * 4 + (lane >> 3), (int)live_rows - 1), t2 = own / p.G;
          row = ((long long)b * p.num_new + t2) * p.Hq + (long long)kvh * p.G + (own - t2 * p.G);
        }
        const uint4* src = reinterpret_cast<const uint4*>(p.q + row * D) + (lane & 7);
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          x[h][it] = KVQ_IN(c, KVQ_ARRAY_Q, src + h * 8, 16) ? __ldg(src + h * 8) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        // in shared memory for good (Q_SMEM, swizzled as K), or on its way
        uint8_t* const at = C::Q_SMEM
                                ? smem + C::STAGES * C::STAGE + ((i * 2 + h) * 128 + (warp & 3) * 32) * 128
                                : scratch;
#pragma unroll
        for (int it = 0; it < 8; ++it) {
          const int rr = it * 4 + (lane >> 3);
          if (row0 + rr >= live_rows) x[h][it] = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(at + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4)) = x[h][it];
        }
        if constexpr (!C::Q_SMEM) {
          __syncwarp();
          uint32_t w[32];
#pragma unroll
          for (int ch = 0; ch < 8; ++ch) {
            const uint4 y = *reinterpret_cast<const uint4*>(scratch + lane * 128 + ((ch ^ (lane & 7)) << 4));
            if constexpr (C::PAIRED) {  // (0, 4), (1, 5), (2, 6), (3, 7)
              w[4 * ch] = fast::prmt_b32(y.x, y.z, 0x5410u);
              w[4 * ch + 1] = fast::prmt_b32(y.x, y.z, 0x7632u);
              w[4 * ch + 2] = fast::prmt_b32(y.y, y.w, 0x5410u);
              w[4 * ch + 3] = fast::prmt_b32(y.y, y.w, 0x7632u);
            } else {
              w[4 * ch] = y.x, w[4 * ch + 1] = y.y, w[4 * ch + 2] = y.z, w[4 * ch + 3] = y.w;
            }
          }
          tc::st32(tq + h * 32, w);
          __syncwarp();
        }
      }
      if constexpr (C::Q_SMEM) tc::fence_async_shared();
      else tc::wait_st();
      tc::fence_before();
      tc::mbar_arrive(q_full(i));
    }
    float m = -INFINITY, l = 0.f;  // reference maximum (log2 units) and sum
    bool going = i < nq;
#pragma unroll 1
    for (int n = 0; going && n < mine; ++n) {
      const int j = C::DUAL ? 2 * n + i : n, st = j % C::STAGES;
      const uint32_t ts = ts0 + buf(n) * kKeys;
      // (S follows the stage's arrival, so its key masks are there too; they
      // stay until P is handed over)
      going = __all_sync(0xffffffffu, !(warp == C::SOFT0 && runs_out(KVQ_WAIT_SOFTMAX, j)) &&
                                           tc::mbar_wait(s_full(i, n), phase(n), stop));
      if (!going) break;
      tc::fence_after();
      if (any_live) {
        uint32_t u[2][32];
        tc::ld32(ts, u[0]);
        tc::ld32(ts + 32, u[1]);
        const int ks = k0 + j * kKeys;
        const uint32_t ok0 = sh.ok[j % (2 * C::STAGES)][0], ok1 = sh.ok[j % (2 * C::STAGES)][1];
        // (a tile that the block's first row sees in part may hold V rows set to
        // zero, which count for every row that sees them)
        const bool checked = KIND == 2 && ks + kKeys - 1 > all_see;
        const bool spoilt = checked && reinterpret_cast<const unsigned short*>(sh.bad[st])[lane];
        const bool whole =
            __all_sync(0xffffffffu, (ok0 & ok1) == 0xFFFFFFFFu && ks + kKeys - 1 <= last && !spoilt);
        tc::wait_ld();
        if (!whole) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t bad = 0;
            if (checked) {
#pragma unroll
              for (int g = 0; g < 8; ++g) {
                const uint32_t v = reinterpret_cast<const uint32_t*>(sh.bad[st])[h * 8 + g];
                bad |= ((v & 1u) | (v >> 7 & 2u) | (v >> 14 & 4u) | (v >> 21 & 8u)) << (4 * g);
              }
            }
            const int seen = last - ks - 32 * h;  // keys 0 .. seen of these
            const uint32_t see = (h ? ok1 : ok0) & (seen >= 31 ? 0xFFFFFFFFu : seen < 0 ? 0u : (2u << seen) - 1u);
            bad &= see;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (!(see >> e & 1u)) u[h][e] = 0xFF800000u;                   // -inf
              else if (KIND == 2 && (bad >> e & 1u)) u[h][e] = 0x7FFFFFFFu;  // NaN: its V is not finite
            }
          }
          __syncwarp();
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 64; e += 2)
          top[(e >> 1) & 3] = tc::max3(top[(e >> 1) & 3], __uint_as_float(u[e >> 5][e & 31]),
                                       __uint_as_float(u[e >> 5][(e & 31) + 1]));
        const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale_log2;
        const bool moves = mx > m + kLazy;  // m = -inf: any finite maximum
        if (__any_sync(0xffffffffu, moves)) {
          const float mn = moves ? mx : m;
          const float alpha = moves ? ex2(m - mn) : 1.f;
          m = mn;
          l *= alpha;
          // (with one S, its arrival says that the products before are done)
          if (C::SB == 2 && n) going = __all_sync(0xffffffffu, tc::mbar_wait(o_step(i), (n - 1) & 1, stop));
          if (C::SB == 2) tc::fence_after();
          if (n) {
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
        const float base = m == -INFINITY ? 0.f : m - kLift;
        const float2 sl2 = make_float2(p.scale_log2, p.scale_log2), nb2 = make_float2(-base, -base);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int h = 0; h < 4; ++h) {  // (P overwrites scores already in registers)
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const int k = 16 * h + e;
            float2 x = make_float2(__uint_as_float(u[k >> 5][k & 31]), __uint_as_float(u[k >> 5][(k & 31) + 1]));
            x = tc::fma2(x, sl2, nb2);
            x.x = ex2(x.x);
            x.y = ex2(x.y);
            sum[(e >> 1) & 1] = tc::add2(sum[(e >> 1) & 1], x);
            w[e >> 1] = fast::pack_h2(x.x, x.y);
          }
          tc::st8(ts + 8 * h, w);
          if (h == 1) {  // the first 32 keys' products may start
            tc::wait_st();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(p_half(i, n));
          }
        }
        tc::wait_st();
        sum[0] = tc::add2(sum[0], sum[1]);
        l += sum[0].x + sum[0].y;
      } else if (lane == 0) {
        tc::mbar_arrive(p_half(i, n));
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(p_full(i, n));
    }
    // both tiles' (streams') products are done with the stages
    for (int k = 0; k < nq && going; ++k)
      if (C::DUAL ? k < tiles : tiles > 0) going = __all_sync(0xffffffffu, tc::mbar_wait(o_full(k), 0, stop));
    tc::fence_after();
    // The second stream hands its sum over in the stages' memory: chunk c of
    // row r at r, c ^ (r & 7).
    const int rr = (warp & 3) * 32 + lane;
    uint8_t* const other = smem + rr * (D * 4);
    float a0 = 1.f, a1 = 0.f;  // the streams' factors
    if (C::DUAL && going && tiles > 1) {
      if (i == 1) {
        if (any_live) {
#pragma unroll 1
          for (int h = 0; h < D / 16; ++h) {
            uint32_t o[16];
            tc::ld16(to + h * 16, o);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4*>(other + (((h * 4 + e) ^ (rr & 7)) << 4)) =
                  make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          sh.ml[rr] = make_float2(m, l);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(merge);
      } else {
        going = __all_sync(0xffffffffu, tc::mbar_wait(merge, 0, stop));
        if (going && any_live) {
          const float2 x = sh.ml[rr];
          const float mn = fmaxf(m, x.x), base = mn == -INFINITY ? 0.f : mn;
          a0 = ex2(m - base);
          a1 = ex2(x.x - base);
          l = l * a0 + x.y * a1;
          m = mn;
        }
      }
    }
    if (going && any_live && !(C::DUAL && i)) {
      const float inv = l != 0.f ? 1.f / l : 0.f;
      scratch = smem + (C::DUAL ? 128 * D * 4 : 0) + (warp - C::SOFT0) * 4096;
#pragma unroll 1
      for (int h = 0; h < D / 32; ++h) {
        uint32_t o[32];
        if (mine) {
          tc::ld32(to + h * 32, o);
          tc::wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        if (C::DUAL && tiles > 1) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 y = *reinterpret_cast<const float4*>(other + (((h * 8 + e) ^ (rr & 7)) << 4));
            const float z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int g = 0; g < 4; ++g)
              o[4 * e + g] = __float_as_uint(__uint_as_float(o[4 * e + g]) * a0 + z[g] * a1);
          }
        }
        float x[32];  // place i of a chunk holds channel(i)
#pragma unroll
        for (int e = 0; e < 32; ++e) x[(e & ~7) + C::channel(e & 7)] = __uint_as_float(o[e]);
        // through the scratch, so that lanes write whole lines of a row
        const bool halves = !PRE && !p.partials;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (halves && e >= 4) continue;
          uint4 y;
          if (halves)
            y = make_uint4(fast::pack_h2(x[8 * (e & 3)] * inv, x[8 * (e & 3) + 1] * inv),
                           fast::pack_h2(x[8 * (e & 3) + 2] * inv, x[8 * (e & 3) + 3] * inv),
                           fast::pack_h2(x[8 * (e & 3) + 4] * inv, x[8 * (e & 3) + 5] * inv),
                           fast::pack_h2(x[8 * (e & 3) + 6] * inv, x[8 * (e & 3) + 7] * inv));
          else
            y = make_uint4(__float_as_uint(x[4 * e]), __float_as_uint(x[4 * e + 1]), __float_as_uint(x[4 * e + 2]),
                           __float_as_uint(x[4 * e + 3]));
          *reinterpret_cast<uint4*>(scratch + lane * 128 + ((e ^ (lane & 7)) << 4)) = y;
        }
        __syncwarp();
        const int per = halves ? 4 : 8, ch = lane & (per - 1);  // lanes a row takes
#pragma unroll 4
        for (int rr = lane / per; rr < 32; rr += 32 / per) {
          const long long row = __shfl_sync(0xffffffffu, orow, rr);
          if (row0 + rr >= live_rows) continue;
          const uint4 y = *reinterpret_cast<const uint4*>(scratch + rr * 128 + ((ch ^ (rr & 7)) << 4));
          if (halves) {
            uint4* d = reinterpret_cast<uint4*>(p.out + row * D + h * 32) + ch;
            if (KVQ_IN(c, KVQ_ARRAY_OUT, d, 16)) *d = y;
          } else {
            uint4* d = reinterpret_cast<uint4*>(p.ws_o + (row * p.splits + split) * D + h * 32) + ch;
            if (KVQ_IN(c, KVQ_ARRAY_WORKSPACE, d, 16)) *d = y;
          }
        }
        __syncwarp();
      }
      if ((PRE || p.partials) && live) {
        float2* ml = reinterpret_cast<float2*>(p.ws_ml) + orow * p.splits + split;
        if (KVQ_IN(c, KVQ_ARRAY_WORKSPACE, ml, 8)) *ml = make_float2(m, l);
      }
    }
  } else if (warp >= C::PROD0) {
    // ------------------------------------------------------ producers
    const int tid = threadIdx.x - C::PROD0 * 32, pw = tid >> 5;
    bool ok = true;
    auto wait_q = [&] {  // before the stages are filled that q passes through
      for (int k = 0; k < nq; ++k)
        if (C::DUAL ? k < tiles : tiles > 0) ok = ok && tc::mbar_wait(q_full(k), 0, stop);
      ok = __all_sync(0xffffffffu, ok);
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
      const int is_v = pw >= C::PROD / 2;  // half the warps turn K, half V
      const int seg = lane % C::SEGS, key_l = lane / C::SEGS;
      const int swap = seg >= 2 ? 2 : 0;
      const bool zeros = KIND == 0 && !c.sym;
      const int hb = 2 * c.ngroups, hseg = 2 * (seg * 32 / c.g);
      // (NG, groups per segment, is fixed for the call: one small loop runs)
      auto convert = [&](auto ng) {
        constexpr int NG = decltype(ng)::value;
        int st = 0, ph = 1, slot = 0, rph = 0;
#pragma unroll 1
        for (int j = 0; j < tiles; ++j) {
          ok = !(pw == (is_v ? C::PROD / 2 : 0) && runs_out(is_v ? KVQ_WAIT_V : KVQ_WAIT_K, j)) &&
               tc::mbar_wait(raw_full(slot), rph, stop);
          const uint8_t* ring = smem + C::STAGES * C::STAGE + slot * C::RAW;
          const uint32_t ok0 = sh.raw_ok[slot][0], ok1 = sh.raw_ok[slot][1];
          const bool all = (ok0 & ok1) == 0xFFFFFFFFu;
          if (ok) ok = tc::mbar_wait(empty(is_v, st), ph, stop);
          ok = __all_sync(0xffffffffu, ok);
          if (ok && is_v && j == C::Q_STAGE) wait_q();
          if (!ok) break;
          if (pw == 0 && lane == 0)
            sh.ok[j % (2 * C::STAGES)][0] = ok0, sh.ok[j % (2 * C::STAGES)][1] = ok1;
          uint8_t* const to = smem + (is_v ? C::V_AT + st * C::V_STEP : st * C::K_STEP);
#pragma unroll 1
          for (int u = 0; u < C::MINE; ++u) {
            const int key0 = (u * (C::PROD / 2) + (pw & (C::PROD / 2 - 1))) * C::KPI, key = key0 + key_l;
            const uint8_t* h = ring + 2 * C::CODES + is_v * 2 * C::HDR + mis + key * hb + hseg;
            Seg<BITS> x;
            take_item<BITS, KIND, NG>(ring + is_v * C::CODES + key0 * (D * BITS / 8), h, h + C::HDR, zeros, lane, swap, x);
            if (!all && !((key < 32 ? ok0 : ok1) >> (key & 31) & 1u))  // not a key: zeros, whatever the ring held
              x.s[0] = x.s[1] = x.z[0] = x.z[1] = 0;
            store_seg<BITS, KIND, NG, C::DUAL ? 2 : 1>(x, key, seg, c.sym, swap, to, to + C::MAT, lut);
          }
          tc::fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            tc::mbar_arrive(full(is_v, st));
            tc::mbar_arrive(raw_empty(slot));
          }
          if (++st == C::STAGES) st = 0, ph ^= 1;
          if (++slot == C::DEPTH) slot = 0, rph ^= 1;
        }
      };
      if (c.g >= 32) convert(Int<1>{});
      else if (c.g == 16) convert(Int<2>{});
      else convert(Int<4>{});
    } else {
      // fp16 rows: straight to their places, a row by consecutive lanes (a row
      // per lane took a tag per lane and copy: 2050 cycles of issue a tile).
      constexpr int CH = D / 8, RPP = C::PROD * 32 / CH;  // chunks of a row, rows a pass
      const int ch = tid % CH, sub = tid / CH;
      // Where a warp's eight keys of a tile lie, a lane per key, looked up a tile
      // ahead: a page takes a division and a load from the table.
      constexpr int SPW = 32 / CH;  // rows a warp has in a pass
      static_assert(SPW * (kKeys / RPP) == 8, "eight keys a warp and tile");
      auto own_row = [&](int j) { return row_of(k0 + j * kKeys + (lane & 7) / SPW * RPP + pw * SPW + (lane & 7) % SPW); };
      long long ahead = own_row(0);
#pragma unroll 1
      for (int j = 0; j < tiles; ++j) {
        const int st = j % C::STAGES;
        const long long rows8 = ahead;
        ok = __all_sync(0xffffffffu, !(pw == 0 && runs_out(KVQ_WAIT_K, j)) &&
                                         tc::mbar_wait(empty(1, st), ((j / C::STAGES) & 1) ^ 1, stop));
        if (ok && j == C::Q_STAGE) wait_q();
        if (!ok) break;
        uint8_t* const stage = smem + st * C::STAGE;
        const uint32_t base = tc::smem_addr(stage) + (ch >> 3) * (kKeys * 128);
#pragma unroll 4
        for (int pass = 0; pass < kKeys / RPP; ++pass) {
          const int key = pass * RPP + sub;
          const long long row = __shfl_sync(0xffffffffu, rows8, pass * SPW + lane / CH);
          const uint32_t dst = base + key * 128 + (((ch & 7) ^ (key & 7)) << 4);
          const long long o = max(row, 0ll) * (2 * D) + ch * 16;
          fast::cp_async16(dst, p.v.codes[0] + o, row >= 0 && KVQ_IN(c, KVQ_ARRAY_K_CODES, p.v.codes[0] + o, 16));
          fast::cp_async16(dst + C::MAT, p.v.codes[1] + o, row >= 0 && KVQ_IN(c, KVQ_ARRAY_V_CODES, p.v.codes[1] + o, 16));
        }
        ahead = own_row(j + 1);  // (-1 behind the last tile)
        if (k0 + (j + 1) * kKeys - 1 <= all_see) {
          tc::mbar_arrive_copies(raw_full(st));
          continue;
        }
        // in a tile that some row sees in part, an infinite or NaN V must not
        // meet the zero weights of the rows that do not see it
        fast::cp_async_commit();
        fast::cp_async_wait<0>();
#pragma unroll 2
        for (int pass = 0; pass < kKeys / RPP; ++pass) {
          const int key = pass * RPP + sub;
          uint4* v = reinterpret_cast<uint4*>(stage + C::MAT + (ch >> 3) * (kKeys * 128) + key * 128 +
                                              (((ch & 7) ^ (key & 7)) << 4));
          const uint4 q = *v;
          const bool bad = nonfinite2(q.x) || nonfinite2(q.y) || nonfinite2(q.z) || nonfinite2(q.w);
          if (bad) *v = make_uint4(0u, 0u, 0u, 0u);
          const uint32_t row_bad = __ballot_sync(0xffffffffu, bad) >> (lane & ~(CH - 1)) & ((1u << CH) - 1u);
          if (ch == 0) sh.bad[st][key] = row_bad != 0;
        }
        tc::mbar_arrive(raw_full(st));
      }
      fast::cp_async_commit();
      fast::cp_async_wait<0>();  // nothing in flight when the block ends
    }
  } else if (warp >= 1 && warp <= C::LOAD) {
    // ------------------------------------------------------ loaders
    bool ok = true;
    if constexpr (KIND != 2) {
      if (p.started) tc::fence_async();  // (start_beside, for the bulk copies too)
      // A tile's rows come in runs of consecutive rows: one in a dense cache,
      // one per page (or part of one) in a paged one; lane r finds run r.
      const int which = warp - 1;
      const bool zeros = KIND == 0 && !c.sym, paged = c.layout == KVQ_PAGED;
      const uint32_t hb = 2 * c.ngroups;
      constexpr uint32_t RB = D * BITS / 8;
      const long long hdr_bytes = (long long)p.batch * c.Hkv * c.slots * hb;  // dense: of a header array, at least
      const uint8_t* const codes = p.v.codes[which];
      const uint8_t* const scale = reinterpret_cast<const uint8_t*>(p.v.scale[which]);
      const uint8_t* const zero = reinterpret_cast<const uint8_t*>(p.v.zero[which]);
      int slot = 0, ph = 1, j = 0;
#pragma unroll 1
      for (; j < tiles; ++j) {
        const int p0 = k0 + j * kKeys, p1 = min(p0 + kKeys, k1);
        int start = p0, end = p1;
        if (paged) {
          const int blk = p0 / c.slots + lane;
          start = min(max(p0, blk * c.slots), p1);  // (at most nine runs)
          end = min(p1, (blk + 1) * c.slots);
          if (lane > 8) start = end = p1;
        } else if (lane) {
          start = p1;
        }
        const int rows = end - start;
        const long long row = rows > 0 ? token_row(c, b, kvh, start) : -1;
        bool live = row >= 0;
        live = live && KVQ_IN(c, KVQ_ARRAY_K_CODES + which, codes + row * RB, (long long)rows * RB) &&
               KVQ_IN(c, which ? KVQ_ARRAY_V_SCALE : KVQ_ARRAY_K_SCALE, scale + row * hb, (long long)rows * hb) &&
               (!zeros || KVQ_IN(c, which ? KVQ_ARRAY_V_ZERO : KVQ_ARRAY_K_ZERO, zero + row * hb, (long long)rows * hb));
        // Whole 16-byte pieces: in a page, rows rounded up to 8 (the page has
        // them); a dense header array starts mis bytes into one and is copied
        // to the end of its last one, which holds the rows that follow.  Behind
        // the last of all rows there may be nothing: that piece is copied by
        // hand (its loads wait for memory: 900 cycles a tile when every tile
        // did it).
        const uint32_t up = paged ? (rows + 7) & ~7 : rows;
        const bool by_hand = !paged && row >= 0 && (row + rows) * hb + 15 > hdr_bytes;
        const uint32_t hdr = paged ? up * hb : (mis + rows * hb + (by_hand ? 0 : 15)) & ~15u;
        const uint32_t total = __reduce_add_sync(0xffffffffu, live ? up * RB + (zeros ? 2 : 1) * hdr : 0u);
        ok = __all_sync(0xffffffffu, !runs_out(which ? KVQ_WAIT_LOAD_V : KVQ_WAIT_LOAD_K, j) &&
                                         tc::mbar_wait(raw_empty(slot), ph, stop));
        if (!ok) break;
        uint8_t* const at = smem + C::STAGES * C::STAGE + slot * C::RAW;
        uint8_t* const at_h = at + 2 * C::CODES + 2 * which * C::HDR;
        if (which == 0) {  // which keys there are
          uint32_t d0 = 0, d1 = 0;
          if (rows > 0 && !live) {
            const int k = start - p0, n = end - p0;  // keys k .. n - 1 have no row
            d0 = (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u) & ~(k >= 32 ? 0xFFFFFFFFu : (1u << k) - 1u);
            d1 = (n > 32 ? (n >= 64 ? 0xFFFFFFFFu : (1u << (n - 32)) - 1u) : 0u) &
                 ~(k > 32 ? (1u << (k - 32)) - 1u : 0u);
            if (row < 0 && p.status) atomicOr(p.status, KVQ_FLAG_BLOCK_TABLE);
          }
          const int n = p1 - p0;
          d0 = __reduce_or_sync(0xffffffffu, d0);
          d1 = __reduce_or_sync(0xffffffffu, d1);
          if (lane == 0) {
            sh.raw_ok[slot][0] = (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u) & ~d0;
            sh.raw_ok[slot][1] = (n > 32 ? (n >= 64 ? 0xFFFFFFFFu : (1u << (n - 32)) - 1u) : 0u) & ~d1;
          }
        }
        uint32_t todo = __ballot_sync(0xffffffffu, live);
        const int n = mis + (p1 - p0) * (int)hb;
        if (__any_sync(0xffffffffu, by_hand) && (n & 15) && todo) {
          const int x = (n & ~15) + 2 * lane;
          const long long from = (((long long)b * c.Hkv + kvh) * c.slots + p0) * hb - mis + x;
          if (x >= mis && x < n) {
            *reinterpret_cast<unsigned short*>(at_h + x) = *reinterpret_cast<const unsigned short*>(scale + from);
            if (zeros)
              *reinterpret_cast<unsigned short*>(at_h + C::HDR + x) = *reinterpret_cast<const unsigned short*>(zero + from);
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_expect(raw_full(slot), total);
        __syncwarp();
        const uint32_t dst = tc::smem_addr(at) + which * C::CODES, dst_h = tc::smem_addr(at_h);
        while (todo) {
          const int r = __ffs(todo) - 1;
          todo &= todo - 1;
          const long long row_r = __shfl_sync(0xffffffffu, row, r);
          const uint32_t key = __shfl_sync(0xffffffffu, start, r) - p0;
          const uint32_t up_r = __shfl_sync(0xffffffffu, up, r), hdr_r = __shfl_sync(0xffffffffu, hdr, r);
          tc::bulk_load(dst + key * RB, codes + row_r * RB, up_r * RB, raw_full(slot));
          if (hdr_r) {
            tc::bulk_load(dst_h + key * hb, scale + row_r * hb - mis, hdr_r, raw_full(slot));
            if (zeros) tc::bulk_load(dst_h + C::HDR + key * hb, zero + row_r * hb - mis, hdr_r, raw_full(slot));
          }
        }
        if (++slot == C::DEPTH) slot = 0, ph ^= 1;
      }
      if (lane == 0) sh.loaded[which] = j;
    } else {
      // The rows of a stage have landed: make them visible to the tensor core
      // and pass the stage on.  (Not the producers' job: the fence would wait
      // for their later copies; nor the MMA warp's: for its products.)
#pragma unroll 1
      for (int j = 0; j < tiles && ok; ++j) {
        const int st = j % C::STAGES;
        // (the softmax is at most STAGES tiles behind, so that the slot is free)
        note_keys(sh.ok[j % (2 * C::STAGES)], j);
        ok = __all_sync(0xffffffffu, !runs_out(KVQ_WAIT_LOAD_K, j) &&
                                         tc::mbar_wait(raw_full(st), (j / C::STAGES) & 1, stop));
        tc::fence_async_shared();
        if (ok && lane == 0) tc::mbar_arrive(full(0, st));
        __syncwarp();
      }
    }
  } else if ((warp == 0 || warp == 3) && tiles) {
    // ------------------------------------------------------ MMA issue
    // A warp per tile of rows: what one does between its products (waiting,
    // descriptors) runs under the other's.
    const int i = warp == 0 ? 0 : 1;
    constexpr uint32_t id_qk = tc::idesc_f16(kKeys, false), id_pv = tc::idesc_f16(D, true);
    const uint32_t t0 = tmem;
    const uint32_t data = tc::smem_addr(smem);
    constexpr uint32_t hi = tc::desc_hi(1024);
    const uint32_t k_lo = tc::desc_lo(data, 16);
    const uint32_t v_lo = tc::desc_lo(data + C::V_AT, kKeys * 128);
    const uint32_t s0 = t0 + C::COL_S + i * C::SB * kKeys, d_o = t0 + C::COL_O + i * D, a_q = t0 + C::COL_Q + i * (D / 2);
    const uint32_t q_lo = tc::desc_lo(data + C::STAGES * C::STAGE + i * (128 * D * 2), 16);  // (Q_SMEM)
    auto qk = [&](int st, int at) {  // the at-th step's scores
      const uint32_t d_s = s0 + buf(at) * kKeys;
      const uint32_t kd = k_lo + st * (C::K_STEP / 16);
      // hi, then lo: the tiles follow one another in 64-channel blocks
#pragma unroll
      for (int n = 0; n < (C::LO ? 2 : 1) * (D / 64); ++n)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          if constexpr (C::Q_SMEM)
            tc::mma_ss(d_s, q_lo + n * (128 * 128 / 16) + kk * 2, kd + n * (kKeys * 128 / 16) + kk * 2, hi, id_qk, n || kk);
          else
            tc::mma_ts(d_s, a_q + ((n * 4) & (D / 16 - 1)) * 8 + kk * 8, kd + n * (kKeys * 128 / 16) + kk * 2, hi, id_qk,
                       n || kk);
      tc::commit(s_full(i, at));
      if (C::LO) tc::commit(empty(0, st));
    };
    auto wait = [&](uint32_t bar, int parity) { return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, stop)); };
    // the warps take turns (TURNS), so that one tile's softmax runs under the
    // other tile's products and not beside its softmax
    auto pass = [&] {
      if (C::TURNS && nq == 2 && lane == 0) tc::mbar_arrive(turn(1 - i));
      __syncwarp();
    };
    const int j0 = C::DUAL ? i : 0;  // this stream's first key tile
    if (i < nq && j0 < tiles && wait(full(0, j0), 0) && wait(q_full(i), 0) && (!C::TURNS || i == 0 || wait(turn(1), 0))) {
      tc::fence_after();
      qk(j0, 0);
      bool ahead = C::SB == 2 && 1 < tiles;  // the second S filled too
      if (ahead) ahead = wait(full(0, 1), 0);
      if (ahead) {
        tc::fence_after();
        qk(1, 1);
      }
      pass();
      int st = j0, tp = i;  // stage of key tile j; phase of the turn
#pragma unroll 1
      for (int j = j0, n = 0;; j += STEP, ++n) {
        const int next = j + C::SB * STEP;  // the tile whose scores follow
        const bool more = next < tiles, last_one = j + STEP >= tiles;
        const int st1 = next % C::STAGES;
        const uint32_t d_s = s0 + buf(n) * kKeys;
        if (C::SB == 2 && !last_one && n == 0 && !ahead) break;
        if (i == 0 && more && runs_out(KVQ_WAIT_SCORES, next)) break;
        if (!C::DUAL && more && !wait(full(0, st1), (next / C::STAGES) & 1)) break;
        if (C::LO && !wait(full(1, st), (j / C::STAGES) & 1)) break;
        if (!wait(p_half(i, n), phase(n))) break;
        if (C::TURNS && nq == 2 && !wait(turn(i), tp)) break;
        tp ^= 1;
        tc::fence_after();
        const uint32_t vd = v_lo + st * (C::V_STEP / 16);
        auto pv = [&](int half) {
#pragma unroll
          for (int part = 0; part < (C::LO ? 2 : 1); ++part)
#pragma unroll
            for (int e = 0; e < kKeys / 32; ++e) {
              const int kk = half * (kKeys / 32) + e;
              tc::mma_ts(d_o, d_s + kk * 8, vd + part * (C::MAT / 16) + kk * (2048 / 16), hi, id_pv, n || part || kk);
            }
        };
        pv(0);
        if (i == 0 && runs_out(KVQ_WAIT_SUM, j)) break;
        if (!wait(p_full(i, n), phase(n))) break;
        tc::fence_after();
        pv(1);
        if (C::SB == 2) tc::commit(o_step(i));
        if (last_one) {
          tc::commit(o_full(i));
          pass();
          break;
        }
        tc::commit(empty(1, st));
        if (C::DUAL && !wait(full(0, st1), (next / C::STAGES) & 1)) break;
        if (more) qk(st1, n + C::SB);
        pass();
        st = (j + STEP) % C::STAGES;
      }
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (sh.stop) {
    // Given up: no product may read shared or tensor memory, and no copy land,
    // after the block has ended.  Copies of the last DEPTH tiles may be in
    // flight (a tile before has been converted); where one loader got further
    // than the other, the other's arrival is made up for.
    if (warp == 0 || warp == 3) {
      tc::commit(done(warp == 3));
      tc::mbar_drain(done(warp == 3), 0);
    }
    if (C::LO && threadIdx.x == 32) {
      const int most = max(sh.loaded[0], sh.loaded[1]), both = min(sh.loaded[0], sh.loaded[1]);
      for (int t = max(most - C::SLOTS, 0); t < most; ++t) {
        if (t >= both) tc::mbar_arrive(raw_full(t % C::SLOTS));
        tc::mbar_drain(raw_full(t % C::SLOTS), (t / C::SLOTS) & 1);
      }
    }
    if (threadIdx.x == 0 && p.status) atomicOr(p.status, KVQ_FLAG_TIMEOUT);
    __syncwarp();
    __syncthreads();
  }
  if (warp == 0) {
    tc::fence_after();
    tc::tmem_dealloc(tmem, C::COLS);
  }
  if constexpr (!PRE) end_after_prefixes(p);
}

template <int BITS, int KIND, int D, int NQ, bool PRE>
cudaError_t run_nq(const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream) {
  using C = Cfg<BITS, KIND, D, NQ>;
  static KernelSetup setup;
  int occ = 0;
  const cudaError_t e = setup_kernel(extend_tc_kernel<BITS, KIND, D, NQ, PRE>, setup, C::THREADS, C::SMEM, &occ);
  if (e != cudaSuccess) return e;
  if (plan) {
    plan->tile_rows = 128 * NQ;
    plan->occ = occ;
    plan->lift = kLift;
    return cudaSuccess;
  }
  const long long each = (long long)p->num_new * p->G;
  const long long tiles = PRE ? prefix_tiles_bound(p->plan.B, p->plan.N, each, 128 * NQ) : (each + 128 * NQ - 1) / (128 * NQ);
  const dim3 grid((unsigned)(tiles * p->splits), p->v.geom.Hkv, PRE ? 1 : p->batch);
  return launch_pdl(extend_tc_kernel<BITS, KIND, D, NQ, PRE>, grid, dim3(C::THREADS), C::SMEM, stream, *p);
}

// Two instance files per format call this for its BITS and KIND.
template <int BITS, int KIND, bool PRE = false>
cudaError_t run_tc(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream) {
  if (D == 64)
    return nq == 1 ? run_nq<BITS, KIND, 64, 1, PRE>(p, plan, stream) : run_nq<BITS, KIND, 64, 2, PRE>(p, plan, stream);
  return nq == 1 ? run_nq<BITS, KIND, 128, 1, PRE>(p, plan, stream) : run_nq<BITS, KIND, 128, 2, PRE>(p, plan, stream);
}

}  // namespace ext

cudaError_t run_extend_tc_int2(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream);
cudaError_t run_extend_tc_int4(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream);
cudaError_t run_extend_tc_int8(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream);
cudaError_t run_extend_tc_nf4(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream);
cudaError_t run_extend_tc_fp16(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream);
cudaError_t run_prefix_tc_int2(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream);
cudaError_t run_prefix_tc_int4(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream);
cudaError_t run_prefix_tc_int8(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream);
cudaError_t run_prefix_tc_nf4(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream);
cudaError_t run_prefix_tc_fp16(int D, int nq, const ExtendParams* p, ExtendPlan* plan, cudaStream_t stream);

}  // namespace kvq
