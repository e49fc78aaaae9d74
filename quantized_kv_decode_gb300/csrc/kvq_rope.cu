// Rotary positions: rotation of q and k (kvq_rope_apply), and the rotation
// fused into the quantizing append (kvq_rope_append).
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

// Turns of the CTA's tokens into shared memory, [token][pair], and the
// tokens' positions (live or not).
__device__ __forceinline__ void fill_turns(const RopeParams& p, long long first, int count,
                                           Turn* turns, Token* toks) {
  const int pairs = p.rope.rotary_dim >> 1;
  if (threadIdx.x < count) toks[threadIdx.x] = token_of(p, first + threadIdx.x);
  __syncthreads();
  for (int i = threadIdx.x; i < count * pairs; i += blockDim.x) {
    const int k = i / pairs;
    turns[i] = rope::turn_of((unsigned long long)toks[k].pos * p.rope.turns[i - k * pairs],
                             p.rope.amplitude);
  }
  __syncthreads();
}

// Rotates rows r0, r0 + step, ... of one token's [heads][D] block: each row
// is cut into items, VEC: pairs of 8-channel chunks (or one chunk of 4
// interleaved pairs), else single pairs; then the channels behind the
// rotated ones, copied unless in place.  An item's inputs are read before
// its outputs are written and no other item touches them, so src may be dst.
template <bool VEC>
__device__ __forceinline__ void rotate_rows(const RopeParams& p, const Turn* turns,
                                            const __half* src, __half* dst, int heads, int item,
                                            int items, int r0, int step) {
  const int rd = p.rope.rotary_dim, pairs = rd >> 1;
  const bool inter = p.rope.interleaved != 0;
  const int per = VEC ? 8 : 1;  // channels of a pass-through item
  const int rot = VEC ? (inter ? rd / 8 : rd / 16) : pairs;
  for (int row = r0; row < heads; row += step) {
    const __half* s = src + (long long)row * p.D;
    __half* d = dst + (long long)row * p.D;
    if (item < rot) {
      if constexpr (VEC) {
        uint4 v[2], o[2];
        const int c0 = inter ? item * 8 : item * 8, c1 = c0 + pairs;
        v[0] = *reinterpret_cast<const uint4*>(s + c0);
        const __half* x = reinterpret_cast<const __half*>(v);
        __half* y = reinterpret_cast<__half*>(o);
        if (inter) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            rope::rotate_exact(turns[item * 4 + e], x[2 * e], x[2 * e + 1], y[2 * e], y[2 * e + 1]);
          *reinterpret_cast<uint4*>(d + c0) = o[0];
        } else {
          v[1] = *reinterpret_cast<const uint4*>(s + c1);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            rope::rotate_exact(turns[c0 + e], x[e], x[8 + e], y[e], y[8 + e]);
          *reinterpret_cast<uint4*>(d + c0) = o[0];
          *reinterpret_cast<uint4*>(d + c1) = o[1];
        }
      } else {
        const int c0 = inter ? 2 * item : item, c1 = inter ? c0 + 1 : c0 + pairs;
        __half y0, y1;
        rope::rotate_exact(turns[item], s[c0], s[c1], y0, y1);
        d[c0] = y0;
        d[c1] = y1;
      }
    } else if (s != d) {
      const int c = rd + (item - rot) * per;
      if constexpr (VEC) *reinterpret_cast<uint4*>(d + c) = *reinterpret_cast<const uint4*>(s + c);
      else d[c] = s[c];
    }
  }
}

// items of a row, and whether the vector form applies (rotated part a whole
// number of chunks on both sides)
__device__ __host__ __forceinline__ bool rope_vec(int rd, bool inter) {
  return inter ? rd % 8 == 0 : rd % 16 == 0;
}
__device__ __forceinline__ int rope_items(int rd, bool inter, int D, bool vec) {
  return vec ? (inter ? rd / 8 : rd / 16) + (D - rd) / 8 : (rd >> 1) + (D - rd);
}

// Grid: x = groups of `tokens` tokens, y = slices of the rows of a token.
template <bool VEC>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p, int tokens) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ __align__(16) Turn turns[];
  __shared__ Token toks[kMaxTokens];
  const long long total = (long long)p.batch * p.num_new;
  const long long first = (long long)blockIdx.x * tokens;
  const int count = (int)min((long long)tokens, total - first);
  fill_turns(p, first, count, turns, toks);
  const int pairs = p.rope.rotary_dim >> 1;
  const int items = rope_items(p.rope.rotary_dim, p.rope.interleaved != 0, p.D, VEC);
  const int rows = kThreads / items;  // rows per pass
  const int r = threadIdx.x / items;
  if (r >= rows) return;
  const int item = threadIdx.x - r * items;
  for (int k = 0; k < count; ++k) {
    if (!toks[k].live) continue;
    const long long at = first + k;
    if (p.Hq)
      rotate_rows<VEC>(p, turns + k * pairs, p.q + at * p.Hq * p.D, p.q_out + at * p.Hq * p.D, p.Hq,
                       item, items, r + rows * blockIdx.y, rows * gridDim.y);
    if (p.Hk)
      rotate_rows<VEC>(p, turns + k * pairs, p.k + at * p.Hk * p.D, p.k_out + at * p.Hk * p.D, p.Hk,
                       item, items, r + rows * blockIdx.y, rows * gridDim.y);
  }
}

// The 8 channels of chunk `ch` of a rotated row.
template <bool VEC>
__device__ __forceinline__ uint4 rotated_chunk(const RopeParams& p, const CacheGeom& c,
                                               const Turn* turns, const __half* row, int ch) {
  const int rd = p.rope.rotary_dim, pairs = rd >> 1;
  const bool inter = p.rope.interleaved != 0;
  uint4 v[2];
  v[0] = make_uint4(0u, 0u, 0u, 0u);
  v[1] = v[0];
  const uint4* own = reinterpret_cast<const uint4*>(row) + ch;
  if (KVQ_IN(c, KVQ_ARRAY_K_NEW, own, 16)) v[0] = __ldg(own);
  if (ch * 8 >= rd) return v[0];
  uint4 o;
  __half* y = reinterpret_cast<__half*>(&o);
  const __half* x = reinterpret_cast<const __half*>(v);
  __half skip;
  if constexpr (VEC) {
    if (inter) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        rope::rotate_exact(turns[ch * 4 + e], x[2 * e], x[2 * e + 1], y[2 * e], y[2 * e + 1]);
    } else {
      const bool upper = ch * 8 >= pairs;
      const uint4* oth = reinterpret_cast<const uint4*>(row + ch * 8 + (upper ? -pairs : pairs));
      if (KVQ_IN(c, KVQ_ARRAY_K_NEW, oth, 16)) v[1] = __ldg(oth);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (upper) rope::rotate_exact(turns[ch * 8 - pairs + e], x[8 + e], x[e], skip, y[e]);
        else rope::rotate_exact(turns[ch * 8 + e], x[e], x[8 + e], y[e], skip);
      }
    }
  } else {
    for (int e = 0; e < 8; ++e) {
      const int d = ch * 8 + e;
      y[e] = x[e];
      if (d >= rd) continue;
      const bool second = inter ? (d & 1) : d >= pairs;
      const int i = inter ? d >> 1 : (second ? d - pairs : d);
      const __half* op = row + (inter ? (d ^ 1) : (second ? i : d + pairs));
      const __half other = KVQ_IN(c, KVQ_ARRAY_K_NEW, op, 2) ? *op : __ushort_as_half(0);
      if (second) rope::rotate_exact(turns[i], other, x[e], skip, y[e]);
      else rope::rotate_exact(turns[i], x[e], other, y[e], skip);
    }
  }
  return o;
}

// Grid as rope_kernel.  K rows are rotated and quantized, V rows quantized
// (quantize8, as in append_kernel: a thread per 8 channels, a group's lanes
// adjacent), q rows rotated.  KIND: 0 asymmetric, 1 symmetric, 2 NF4.
template <int BITS, int KIND, bool VEC>
__global__ void __launch_bounds__(kThreads)
    rope_append_kernel(const __grid_constant__ RopeAppendParams pp, int tokens) {
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
  fill_turns(p, first, count, turns, toks);
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
        v = rotated_chunk<VEC>(p, c, turns + k * pairs, src, ch);
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
    const int items = rope_items(p.rope.rotary_dim, p.rope.interleaved != 0, p.D, VEC);
    const int qrows = kThreads / items, r = threadIdx.x / items;
    if (r >= qrows) return;
    for (int k = 0; k < count; ++k)
      if (toks[k].live)
        rotate_rows<VEC>(p, turns + k * pairs, p.q + (first + k) * p.Hq * p.D,
                         p.q_out + (first + k) * p.Hq * p.D, p.Hq, threadIdx.x - r * items, items,
                         r + qrows * blockIdx.y, qrows * gridDim.y);
  }
}

// Tokens per CTA and slices of a token's rows: up to kMaxTokens tokens share
// a CTA once the grid fills the device several times over (fewer CTAs repeat
// the launch overhead); with few tokens their rows are spread over CTAs.
void rope_grid(long long total, int rows_per_token, int rows_per_pass, int* tokens, dim3* grid) {
  int n = 1;
  while (n < kMaxTokens && total / (2 * n) >= 1216) n *= 2;
  long long slices = 1;
  const long long passes = ((long long)n * rows_per_token + rows_per_pass - 1) / rows_per_pass;
  while (slices * 2 <= passes && total / n * slices * 2 <= 608) slices *= 2;
  *tokens = n;
  *grid = dim3((unsigned)((total + n - 1) / n), (unsigned)slices);
}

template <typename Params>
cudaError_t launch2(void (*kernel)(Params, int), dim3 grid, size_t smem, cudaStream_t stream,
                    const Params& p, int tokens) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, tokens);
}

size_t turn_bytes(const kvq_rope& r, int tokens) {
  return (size_t)tokens * (r.rotary_dim / 2) * sizeof(Turn);  // at most 16 KB
}

template <int BITS, int KIND>
cudaError_t launch_append_bits(const RopeAppendParams& p, cudaStream_t s, dim3 grid, int tokens) {
  const size_t smem = turn_bytes(p.r.rope, tokens);
  return rope_vec(p.r.rope.rotary_dim, p.r.rope.interleaved != 0)
             ? launch2(rope_append_kernel<BITS, KIND, true>, grid, smem, s, p, tokens)
             : launch2(rope_append_kernel<BITS, KIND, false>, grid, smem, s, p, tokens);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
  const long long total = (long long)p.batch * p.num_new;
  if (total == 0 || p.Hq + p.Hk == 0) return cudaSuccess;
  const bool vec = rope_vec(p.rope.rotary_dim, p.rope.interleaved != 0) && p.D % 8 == 0;
  int tokens;
  dim3 grid;
  rope_grid(total, p.Hq + p.Hk, 32, &tokens, &grid);
  const size_t smem = turn_bytes(p.rope, tokens);
  return vec ? launch2(rope_kernel<true>, grid, smem, stream, p, tokens)
             : launch2(rope_kernel<false>, grid, smem, stream, p, tokens);
}

cudaError_t launch_rope_append(const RopeAppendParams& p, cudaStream_t stream) {
  const CacheGeom& c = p.a.geom;
  const long long total = (long long)p.a.batch * p.a.num_new;
  if (total == 0) return cudaSuccess;
  int tokens;
  dim3 grid;
  rope_grid(total, p.r.Hq + 2 * c.Hkv, 16, &tokens, &grid);
  switch (c.bits * 4 + (c.nf4 ? 2 : (c.sym ? 1 : 0))) {
    case 8:  return launch_append_bits<2, 0>(p, stream, grid, tokens);
    case 9:  return launch_append_bits<2, 1>(p, stream, grid, tokens);
    case 16: return launch_append_bits<4, 0>(p, stream, grid, tokens);
    case 17: return launch_append_bits<4, 1>(p, stream, grid, tokens);
    case 18: return launch_append_bits<4, 2>(p, stream, grid, tokens);
    case 32: return launch_append_bits<8, 0>(p, stream, grid, tokens);
    case 33: return launch_append_bits<8, 1>(p, stream, grid, tokens);
    default: return launch_append_bits<16, 0>(p, stream, grid, tokens);
  }
}

}  // namespace kvq
