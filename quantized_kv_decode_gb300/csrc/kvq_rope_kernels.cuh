// Kernels of the rotary positions: rotation of q and k, and the rotation fused
// into the quantizing append, by one position a token (kvq_rope.cu) or by one
// an axis (kvq_rope_axes.cu).
#pragma once

#include <type_traits>

#include "kvq_quant.cuh"
#include "kvq_rope.cuh"

namespace kvq {
namespace {

using rope::Turn;

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // tokens per CTA

// The position of token t of sequence b, or a skip: bad lengths are flagged.
struct Token {
  int b, t;
  long long pos;
  bool live;
};
__device__ __forceinline__ Token token_of(const RopeParams& p, long long i) {
  Token k;
  k.b = (int)(i / p.num_new);
  k.t = (int)(i - (long long)k.b * p.num_new);
  const int n = new_rows_of(p.new_lens, k.b, p.num_new);
  k.live = k.t < n;
  k.pos = 0;
  uint32_t flags = n < 0 ? KVQ_FLAG_SEQ_LEN : 0u;
  if (p.positions) {
    if (k.live) k.pos = __ldg(p.positions + i);
  } else {
    const int before = __ldg(p.seq_lens_before + k.b);
    if (before < 0) {
      flags |= KVQ_FLAG_SEQ_LEN;
      k.live = false;
    }
    k.pos = (long long)before + k.t;
  }
  if (flags && p.status && k.t == 0) atomicOr(p.status, flags);
  return k;
}

__device__ __forceinline__ const RopeParams& rope_of(const RopeParams& p) { return p; }
__device__ __forceinline__ const RopeParams& rope_of(const RopeAppendParams& p) { return p.r; }

// Whether the pairs of a launch turn by their own axis' position.
template <class Params>
constexpr bool kAxes = std::is_same_v<Params, RopeAxesParams>;

// The position that pair i of token `at` turns by.
template <class Params>
__device__ __forceinline__ long long turn_position(const Params& pp, const Token& tok, long long at, int i) {
  if constexpr (kAxes<Params>) return __ldg(pp.at + at * pp.num_axes + pp.axis[i]);
  else return tok.pos;
}

// Turns of the CTA's tokens into shared memory, [token][pair], and the
// tokens' positions (live or not).
template <class Params>
__device__ __forceinline__ void fill_turns(const Params& pp, long long first, int count,
                                           Turn* turns, Token* toks) {
  const RopeParams& p = rope_of(pp);
  const int pairs = p.rope.rotary_dim >> 1;
  if (threadIdx.x < count) toks[threadIdx.x] = token_of(p, first + threadIdx.x);
  __syncthreads();
  for (int i = threadIdx.x; i < count * pairs; i += blockDim.x) {
    const int k = i / pairs;
    const long long pos = turn_position(pp, toks[k], first + k, i - k * pairs);
    turns[i] = rope::turn_of((unsigned long long)pos * p.rope.turns[i - k * pairs], p.rope.amplitude);
  }
  __syncthreads();
}

// ---- the general form: any even rotary_dim -------------------------------

// Rotates rows r0, r0 + step, ... of one token's [heads][D] block: each row
// is cut into items, the pairs and then the channels behind them, copied
// unless in place.  An item's inputs are read before its outputs are written
// and no other item touches them, so src may be dst.
__device__ __forceinline__ void rotate_rows(const RopeParams& p, const Turn* turns, const __half* src, __half* dst,
                                            int heads, int item, int r0, int step) {
  const int rd = p.rope.rotary_dim, pairs = rd >> 1;
  const bool inter = p.rope.interleaved != 0;
  for (int row = r0; row < heads; row += step) {
    const __half* s = src + (long long)row * p.D;
    __half* d = dst + (long long)row * p.D;
    if (item < pairs) {
      const int c0 = inter ? 2 * item : item, c1 = inter ? c0 + 1 : c0 + pairs;
      __half y0, y1;
      rope::rotate_exact(turns[item], s[c0], s[c1], y0, y1);
      d[c0] = y0;
      d[c1] = y1;
    } else if (s != d) {
      d[pairs + item] = s[pairs + item];
    }
  }
}
__device__ __forceinline__ int rope_items(const RopeParams& p) { return p.D - (p.rope.rotary_dim >> 1); }

// Grid: x = groups of `tokens` tokens, y = slices of the rows of a token.
template <class Params>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ Params pp, int tokens) {
  pdl_launch_dependents();
  pdl_wait();
  const RopeParams& p = rope_of(pp);
  extern __shared__ __align__(16) Turn turns[];
  __shared__ Token toks[kMaxTokens];
  const long long total = (long long)p.batch * p.num_new;
  const long long first = (long long)blockIdx.x * tokens;
  const int count = (int)min((long long)tokens, total - first);
  fill_turns(pp, first, count, turns, toks);
  const int pairs = p.rope.rotary_dim >> 1;
  const int items = rope_items(p);  // at most 255
  const int rows = kThreads / items;  // rows per pass
  const int r = threadIdx.x / items;
  if (r >= rows) return;
  const int item = threadIdx.x - r * items;
  for (int k = 0; k < count; ++k) {
    if (!toks[k].live) continue;
    const long long at = first + k;
    if (p.Hq)
      rotate_rows(p, turns + k * pairs, p.q + at * p.Hq * p.D, p.q_out + at * p.Hq * p.D, p.Hq, item,
                  r + rows * blockIdx.y, rows * gridDim.y);
    if (p.Hk)
      rotate_rows(p, turns + k * pairs, p.k + at * p.Hk * p.D, p.k_out + at * p.Hk * p.D, p.Hk, item,
                  r + rows * blockIdx.y, rows * gridDim.y);
  }
}

// The 8 channels of chunk `ch` of a rotated row.
__device__ __forceinline__ uint4 rotated_chunk(const RopeParams& p, const CacheGeom& c, const Turn* turns,
                                               const __half* row, int ch) {
  const int rd = p.rope.rotary_dim, pairs = rd >> 1;
  const bool inter = p.rope.interleaved != 0;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  const uint4* own = reinterpret_cast<const uint4*>(row) + ch;
  if (KVQ_IN(c, KVQ_ARRAY_K_NEW, own, 16)) v = __ldg(own);
  uint4 o = v;
  __half* y = reinterpret_cast<__half*>(&o);
  const __half* x = reinterpret_cast<const __half*>(&v);
  __half skip;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int d = ch * 8 + e;
    if (d >= rd) continue;
    const bool second = inter ? (d & 1) : d >= pairs;
    const int i = inter ? d >> 1 : (second ? d - pairs : d);
    const __half* op = row + (inter ? (d ^ 1) : (second ? i : d + pairs));
    const __half other = KVQ_IN(c, KVQ_ARRAY_K_NEW, op, 2) ? *op : __ushort_as_half(0);
    if (second) rope::rotate_exact(turns[i], other, x[e], skip, y[e]);
    else rope::rotate_exact(turns[i], x[e], other, y[e], skip);
  }
  return o;
}

// Grid as rope_kernel.  K rows are rotated and quantized, V rows quantized
// (quantize8, as in append_kernel: a thread per 8 channels, a group's lanes
// adjacent), q rows rotated.  KIND: 0 asymmetric, 1 symmetric, 2 NF4.
template <int BITS, int KIND, class Params>
__global__ void __launch_bounds__(kThreads)
    rope_append_kernel(const __grid_constant__ Params pp, int tokens) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ __align__(16) Turn turns[];
  __shared__ Token toks[kMaxTokens];
  const RopeParams& p = pp.r;
  const AppendParams& a = pp.a;
  const CacheGeom& c = a.geom;
  const long long total = (long long)p.batch * p.num_new;
  const long long first = (long long)blockIdx.x * tokens;
  const int count = (int)min((long long)tokens, total - first);
  fill_turns(pp, first, count, turns, toks);
  const int pairs = p.rope.rotary_dim >> 1;

  const int chunks = c.D / 8;  // 8, 16 or 32: whole rows per warp
  const int rows = kThreads / chunks;
  const int ch = threadIdx.x % chunks, r0 = threadIdx.x / chunks;
  const long long limit = c.layout == KVQ_DENSE ? c.slots : (long long)c.max_blocks * c.slots;
  uint32_t flags = 0;
  // rows of all tokens: [token][which][kv head]
  const int per_token = 2 * c.Hkv, all = count * per_token;
  for (int base = rows * blockIdx.y; base < all; base += rows * gridDim.y) {
    const int i = base + r0;
    const int k = min(i, all - 1) / per_token;
    const int w = min(i, all - 1) - k * per_token;
    const int which = w >= c.Hkv, kvh = w - which * c.Hkv;
    const Token tok = toks[k];
    const bool live = i < all && tok.live;
    long long row = -1;
    if (live) {
      if (tok.pos >= limit) {
        flags |= KVQ_FLAG_SEQ_LEN;
      } else {
        row = token_row(c, tok.b, kvh, (int)tok.pos);
        if (row < 0) flags |= KVQ_FLAG_BLOCK_TABLE;
      }
    }
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (row >= 0) {
      const __half* src = a.src[which] + ((first + k) * c.Hkv + kvh) * (long long)c.D;
      if (which) {
        const uint4* sp = reinterpret_cast<const uint4*>(src) + ch;
        if (KVQ_IN(c, KVQ_ARRAY_V_NEW, sp, 16)) v = __ldg(sp);
      } else {
        v = rotated_chunk(p, c, turns + k * pairs, src, ch);
      }
    }
    const int a_codes = which ? KVQ_ARRAY_V_CODES : KVQ_ARRAY_K_CODES;
    uint8_t* dst = a.codes[which] + row * c.row_bytes + ch * BITS;
    if constexpr (BITS == 16) {
      if (row >= 0 && KVQ_IN(c, a_codes, dst, 16)) *reinterpret_cast<uint4*>(dst) = v;
    } else {
      const int tpg = c.g / 8;
      // every lane: the group uses shuffles
      const Quant8 qz = KIND == 2 ? quantize8_nf4(v, tpg, a.nf4_mid) : quantize8<BITS, KIND == 1>(v, tpg);
      if (row < 0) continue;
      flags |= qz.flags;
      if (KVQ_IN(c, a_codes, dst, BITS)) {
        if constexpr (BITS == 2) *reinterpret_cast<uint16_t*>(dst) = (uint16_t)qz.w0;
        else if constexpr (BITS == 4) *reinterpret_cast<uint32_t*>(dst) = qz.w0;
        else *reinterpret_cast<uint2*>(dst) = make_uint2(qz.w0, qz.w1);
      }
      if (ch % tpg == 0) {
        const long long h = row * c.ngroups + ch / tpg;
        if (KVQ_IN(c, which ? KVQ_ARRAY_V_SCALE : KVQ_ARRAY_K_SCALE, a.scale[which] + h, 2))
          a.scale[which][h] = qz.s;
        if constexpr (KIND == 0)
          if (KVQ_IN(c, which ? KVQ_ARRAY_V_ZERO : KVQ_ARRAY_K_ZERO, a.zero[which] + h, 2))
            a.zero[which][h] = qz.z;
      }
    }
  }
  if (flags && p.status) atomicOr(p.status, flags);

  if (p.Hq) {
    const int items = rope_items(p);
    const int qrows = kThreads / items, r = threadIdx.x / items;
    if (r >= qrows) return;
    for (int k = 0; k < count; ++k)
      if (toks[k].live)
        rotate_rows(p, turns + k * pairs, p.q + (first + k) * p.Hq * p.D, p.q_out + (first + k) * p.Hq * p.D, p.Hq,
                    threadIdx.x - r * items, r + qrows * blockIdx.y, qrows * gridDim.y);
  }
}

template <typename Params>
cudaError_t launch2(void (*kernel)(Params, int), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                    const Params& p, int tokens) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, tokens);
}

// ---- the vector form: a warp per token ----------------------------------
//
// A warp computes its token's turns once (two pairs a lane) and then walks
// the token's rows: K rows (rotated and quantized), V rows (quantized), q
// rows and, without a cache, k rows (rotated).  A lane keeps the same
// channels in every row of a kind, so their turns stay in its registers, and
// it has two rows' loads in flight (four: 198 us where two take 131, fewer
// warps and more code).  With few tokens a token's rows are spread over
// `slices` warps.  BITS 0: no append.
//
// 4 x 8192 tokens, 32 q and 8 KV heads of 128: rotation 131 us, 5.1 TB/s (0.76
// of a plain copy); with the INT8 append 264 us, bound by the instructions of
// the quantizer; 8 tokens of 32 + 32 heads 3.7 us.
constexpr int kWarps = 4;

// Lanes a row of q or k takes: a lane handles two chunks (half layout) or one.
__host__ __device__ __forceinline__ int row_items(int rd, bool inter, int D) {
  return inter ? D / 8 : rd / 16 + ((D - rd) / 8 + 1) / 2;
}

template <int BITS, int KIND, bool INTER, class Params>
__global__ void __launch_bounds__(kWarps * 32)
    rope_warp_kernel(const __grid_constant__ Params pp, int slices) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ Turn turn_s[kWarps][KVQ_ROPE_MAX_PAIRS];
  const RopeParams& p = pp.r;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * kWarps + warp;
  const long long at = w / slices;  // token
  const int slice = (int)(w - at * slices);
  if (at >= (long long)p.batch * p.num_new) return;
  const Token tok = token_of(p, at);
  if (!tok.live) return;
  Turn* turn = turn_s[warp];
  const int rd = p.rope.rotary_dim, pairs = rd >> 1;
  // Pair i of the P pairs of item k at i * items + k: the lanes of a row read
  // consecutive turns.
  constexpr int P = INTER ? 4 : 8;
  const int rot = pairs / P;
  for (int i = lane; i < pairs; i += 32)
    turn[(i & (P - 1)) * rot + i / P] =
        rope::turn_of((unsigned long long)turn_position(pp, tok, at, i) * p.rope.turns[i], p.rope.amplitude);
  __syncwarp();
  const float e = fmaxf((float)p.rope.amplitude * 0x1p-61f, 1.f) * (1.0625f * 0x1p-24f);
  int next = slice;  // this warp's next pass, counted over all kinds

  if constexpr (BITS != 0) {
    const AppendParams& a = pp.a;
    const CacheGeom& c = a.geom;
    const int chunks = c.D / 8, rpp = 32 / chunks;  // whole rows per pass
    const int ch = lane % chunks, sub = lane / chunks;
    const int passes = (c.Hkv + rpp - 1) / rpp;
    const long long limit = c.layout == KVQ_DENSE ? c.slots : (long long)c.max_blocks * c.slots;
    uint32_t flags = tok.pos >= limit ? KVQ_FLAG_SEQ_LEN : 0u;
    // this lane's chunk: turned with its partner chunk (half layout), or by
    // itself (interleaved)
    const bool turned = ch * 8 < rd, upper = !INTER && ch * 8 >= pairs;
    const int item = INTER ? ch : (upper ? ch - rot : ch);
#pragma unroll 1
    for (int pass = next; pass < 2 * passes; pass += slices) {
      next = pass + slices;
      const int which = pass >= passes;
      const int kvh = (which ? pass - passes : pass) * rpp + sub;
      long long row = -1;
      if (kvh < c.Hkv && tok.pos < limit) {
        row = token_row(c, tok.b, kvh, (int)tok.pos);
        if (row < 0) flags |= KVQ_FLAG_BLOCK_TABLE;
      }
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (row >= 0) {
        const __half* src = a.src[which] + (at * c.Hkv + kvh) * c.D;
        const uint4* own = reinterpret_cast<const uint4*>(src) + ch;
        if (KVQ_IN(c, which ? KVQ_ARRAY_V_NEW : KVQ_ARRAY_K_NEW, own, 16)) v = __ldg(own);
        if (!which && turned) {
          uint4 u = make_uint4(0u, 0u, 0u, 0u), o0, o1;
          if constexpr (!INTER) {
            const uint4* oth = reinterpret_cast<const uint4*>(src + ch * 8 + (upper ? -pairs : pairs));
            if (KVQ_IN(c, KVQ_ARRAY_K_NEW, oth, 16)) u = __ldg(oth);
          }
          const uint4 x0 = upper ? u : v, x1 = upper ? v : u;
          rope::rotate_chunk<P, INTER>(turn + item, rot, e, x0, x1, o0, o1);
          v = upper ? o1 : o0;
        }
      }
      const int a_codes = which ? KVQ_ARRAY_V_CODES : KVQ_ARRAY_K_CODES;
      uint8_t* dst = a.codes[which] + row * c.row_bytes + ch * BITS;
      if constexpr (BITS == 16) {
        if (row >= 0 && KVQ_IN(c, a_codes, dst, 16)) *reinterpret_cast<uint4*>(dst) = v;
      } else {
        const int tpg = c.g / 8;
        __syncwarp();
        // every lane: the group uses shuffles
        const Quant8 qz = KIND == 2 ? quantize8_nf4(v, tpg, a.nf4_mid) : quantize8<BITS, KIND == 1>(v, tpg);
        if (row < 0) continue;
        flags |= qz.flags;
        if (KVQ_IN(c, a_codes, dst, BITS)) {
          if constexpr (BITS == 2) *reinterpret_cast<uint16_t*>(dst) = (uint16_t)qz.w0;
          else if constexpr (BITS == 4) *reinterpret_cast<uint32_t*>(dst) = qz.w0;
          else *reinterpret_cast<uint2*>(dst) = make_uint2(qz.w0, qz.w1);
        }
        if (ch % tpg == 0) {
          const long long h = row * c.ngroups + ch / tpg;
          if (KVQ_IN(c, which ? KVQ_ARRAY_V_SCALE : KVQ_ARRAY_K_SCALE, a.scale[which] + h, 2))
            a.scale[which][h] = qz.s;
          if constexpr (KIND == 0)
            if (KVQ_IN(c, which ? KVQ_ARRAY_V_ZERO : KVQ_ARRAY_K_ZERO, a.zero[which] + h, 2))
              a.zero[which][h] = qz.z;
        }
      }
    }
    if (flags && p.status) atomicOr(p.status, flags);
    next = next >= 2 * passes ? next - 2 * passes : next;
  }

  // q and k rows: items of two partner chunks (half layout) or of one chunk,
  // then the chunks behind the turned channels by twos (or one), copied
  // unless in place
  const int items = row_items(rd, INTER, p.D);
  const int rpp = 32 / items, sub = lane / items, item = lane - sub * items;
  const bool turns = item < rot;
  const int c0 = turns ? item * 8 : rd + (item - rot) * (INTER ? 8 : 16);
  const int c1 = turns ? pairs : 8;  // the second chunk, half layout
  const bool two = !INTER && (turns || c0 + 8 < p.D);
  constexpr int UN = 2;  // rows in flight
  const int rows = p.Hq + p.Hk, step = slices * rpp;
  if (sub >= rpp) return;
#pragma unroll 1
  for (int r0 = next * rpp + sub; r0 < rows; r0 += UN * step) {
    uint4 x0[UN], x1[UN];
    long long at_row[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int r = r0 + u * step;
      if (r >= rows) continue;
      const bool is_k = r >= p.Hq;
      at_row[u] = (is_k ? at * p.Hk + (r - p.Hq) : at * p.Hq + r) * p.D + c0;
      const __half* src = (is_k ? p.k : p.q) + at_row[u];
      x0[u] = *reinterpret_cast<const uint4*>(src);
      if (two) x1[u] = *reinterpret_cast<const uint4*>(src + c1);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int r = r0 + u * step;
      if (r >= rows) continue;
      __half* dst = (r >= p.Hq ? p.k_out : p.q_out) + at_row[u];
      if (!turns) {
        if (dst != (r >= p.Hq ? p.k : p.q) + at_row[u]) {
          *reinterpret_cast<uint4*>(dst) = x0[u];
          if (two) *reinterpret_cast<uint4*>(dst + c1) = x1[u];
        }
        continue;
      }
      uint4 y0, y1;
      rope::rotate_chunk<P, INTER>(turn + item, rot, e, x0[u], x1[u], y0, y1);
      *reinterpret_cast<uint4*>(dst) = y0;
      if (!INTER) *reinterpret_cast<uint4*>(dst + pairs) = y1;
    }
  }
}

template <int BITS, int KIND, class Params>
cudaError_t launch_warp(const Params& p, cudaStream_t stream) {
  const long long total = (long long)p.r.batch * p.r.num_new;
  // passes of a token's rows, and warps sharing them while the grid is small:
  // eight warps an SM already cover a memory latency, and each slice computes
  // the token's turns again (4096 tokens: 20 us with one slice, 23, 28 and 40
  // with 2, 4 and 8; 512 tokens: 7.1 us with 4, 10.5 with 16)
  const int rd = p.r.rope.rotary_dim;
  const bool inter = p.r.rope.interleaved != 0;
  const int rpp = 32 / row_items(rd, inter, p.r.D);
  long long passes = (p.r.Hq + p.r.Hk + rpp - 1) / rpp;
  if (BITS) {
    const int k = 32 / (p.r.D / 8);
    passes += 2 * ((p.a.geom.Hkv + k - 1) / k);
  }
  long long slices = 1;
  while (slices < passes && total * slices < 1216) slices *= 2;
  // An append's tokens take about as much beside the turns (the quantizer): two warps
  // a token where one leaves the SMs half empty (INT8, all of 1300, 2000 tokens 30.6,
  // 27.1 us with one, 21.3, 21.9 with two; 4096, 8190, 12288 39.7, 74.1, 107.3 and
  // 41.3, 76.4, 112.3), and up to 12288 for padded batches, which hold fewer tokens
  // than they have room for (a fifth of 4096, 8190, 12288: 35.5, 38.1, 38.8 and 20.4,
  // 23.3, 32.5; half of them 34.2, 40.4, 63.9 and 22.1, 41.8, 61.2).
  if (BITS && slices == 1 && passes > 1 && total <= (p.r.new_lens ? 12288 : 2432)) slices = 2;
  const long long warps = total * slices;
  const dim3 grid((unsigned)((warps + kWarps - 1) / kWarps));
  return inter ? launch2(rope_warp_kernel<BITS, KIND, true, Params>, grid, kWarps * 32, 0, stream, p, (int)slices)
               : launch2(rope_warp_kernel<BITS, KIND, false, Params>, grid, kWarps * 32, 0, stream, p, (int)slices);
}

// Tokens per CTA and slices of a token's rows: up to kMaxTokens tokens share
// a CTA once the grid fills the device several times over (fewer CTAs repeat
// the launch overhead); with few tokens their rows are spread over CTAs.
inline void rope_grid(long long total, int rows_per_token, int rows_per_pass, int* tokens, dim3* grid) {
  int n = 1;
  while (n < kMaxTokens && total / (2 * n) >= 1216) n *= 2;
  long long slices = 1;
  const long long passes = ((long long)n * rows_per_token + rows_per_pass - 1) / rows_per_pass;
  while (slices * 2 <= passes && total / n * slices * 2 <= 608) slices *= 2;
  *tokens = n;
  *grid = dim3((unsigned)((total + n - 1) / n), (unsigned)slices);
}

inline size_t turn_bytes(const kvq_rope& r, int tokens) {
  return (size_t)tokens * (r.rotary_dim / 2) * sizeof(Turn);  // at most 16 KB
}

// Whether the vector form applies: pairs in whole 16-byte chunks
inline bool rope_vec(const kvq_rope& r) { return r.interleaved ? r.rotary_dim % 8 == 0 : r.rotary_dim % 16 == 0; }

// Launches the form that takes the rotation, for tokens of one format.
template <int BITS, int KIND, class Params>
cudaError_t launch_append_bits(const Params& p, cudaStream_t s) {
  if (rope_vec(p.r.rope)) return launch_warp<BITS, KIND>(p, s);
  int tokens;
  dim3 grid;
  rope_grid((long long)p.a.batch * p.a.num_new, p.r.Hq + 2 * p.a.geom.Hkv, 16, &tokens, &grid);
  return launch2(rope_append_kernel<BITS, KIND, Params>, grid, kThreads, turn_bytes(p.r.rope, tokens), s, p, tokens);
}

template <class Params>
cudaError_t launch_append_any(const Params& p, cudaStream_t stream) {
  const CacheGeom& c = p.a.geom;
  if ((long long)p.a.batch * p.a.num_new == 0) return cudaSuccess;
  switch (c.bits * 4 + (c.nf4 ? 2 : (c.sym ? 1 : 0))) {
    case 8:  return launch_append_bits<2, 0>(p, stream);
    case 9:  return launch_append_bits<2, 1>(p, stream);
    case 16: return launch_append_bits<4, 0>(p, stream);
    case 17: return launch_append_bits<4, 1>(p, stream);
    case 18: return launch_append_bits<4, 2>(p, stream);
    case 32: return launch_append_bits<8, 0>(p, stream);
    case 33: return launch_append_bits<8, 1>(p, stream);
    default: return launch_append_bits<16, 0>(p, stream);
  }
}

}  // namespace
}  // namespace kvq
