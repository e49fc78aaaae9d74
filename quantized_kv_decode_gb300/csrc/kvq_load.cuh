// Eight channels of a cached K or V row as fp16 values, for the kernels that
// work on whole fp16 rows (reading the cache back, attention of several new
// tokens): x_hat = (q - z) s in fp32 ("What actually happens when you
// quantize a KV cache", section 3 step 3), rounded once to fp16 and held at
// the largest finite fp16 (a group's last code can decode up to half a step
// beyond its maximum).
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

// The arrays of one cache, as a kernel reads them.
struct CacheView {
  CacheGeom geom;
  const uint8_t* codes[2];  // K, V
  const __half* scale[2];
  const __half* zero[2];
  const __half* window[2];
  float nf4_level[16];
};

// Largest number of positions a sequence of this cache holds.
__device__ __host__ __forceinline__ long long cache_capacity(const CacheGeom& c) {
  const long long paged = (long long)c.slots * c.max_blocks + (c.kch ? c.sink : 0);
  return c.layout == KVQ_DENSE ? (long long)c.slots : paged;
}

// Row of position pos of a sequence of L tokens: >= 0, or -1 when its page
// is unmapped.  (Axis-aware window positions have no row; 0 marks them live.)
__device__ __forceinline__ long long view_row(const CacheGeom& c, int b, int kvh, int L, int pos) {
  if (!c.kch) return token_row(c, b, kvh, pos);
  return window_slot(c, L, pos) >= 0 ? 0 : kch_row(c, b, kvh, pos);
}

__device__ __forceinline__ uint32_t pack_sat(float a, float b) {
  const __half2 h = __floats2half2_rn(fminf(fmaxf(a, -65504.f), 65504.f),
                                      fminf(fmaxf(b, -65504.f), 65504.f));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// What pack_sat's rounding of a and b left (0 where it held them).
__device__ __forceinline__ uint32_t pack_rest(float a, float b, uint32_t hi) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return pack_sat(fabsf(a) > 65504.f ? 0.f : a - v.x, fabsf(b) > 65504.f ? 0.f : b - v.y);
}

// Channels [8 ch, 8 ch + 8) of K (which = 0) or V (which = 1) at position
// pos, cache row `row` >= 0, of a sequence of L tokens.  lo (may be null):
// what the rounding to fp16 left, itself as fp16.
template <int BITS>
__device__ __forceinline__ uint4 load8(const CacheView& v, int which, int b, int kvh, int L,
                                       int pos, long long row, int ch, uint4* lo = nullptr) {
  const CacheGeom& c = v.geom;
  uint4 o = make_uint4(0u, 0u, 0u, 0u);
  if (lo) *lo = o;
  const int a_codes = which ? KVQ_ARRAY_V_CODES : KVQ_ARRAY_K_CODES;
  const uint8_t* src = v.codes[which] + row * c.row_bytes + ch * BITS;
  if constexpr (BITS == 16) {
    if (KVQ_IN(c, a_codes, src, 16)) o = __ldg(reinterpret_cast<const uint4*>(src));
    return o;
  } else {
    if (c.kch) {
      const int slot = window_slot(c, L, pos);
      if (slot >= 0) {
        const long long bh = (long long)b * c.Hkv + kvh;
        const uint4* w = reinterpret_cast<const uint4*>(
                             v.window[which] + (bh * (c.sink + c.g) + slot) * c.D) + ch;
        if (KVQ_IN(c, which ? KVQ_ARRAY_V_WINDOW : KVQ_ARRAY_K_WINDOW, w, 16)) o = __ldg(w);
        return o;
      }
    }
    uint32_t w0 = 0, w1 = 0;
    if (KVQ_IN(c, a_codes, src, BITS)) {
      if constexpr (BITS == 2) {
        w0 = __ldg(reinterpret_cast<const uint16_t*>(src));
      } else if constexpr (BITS == 4) {
        w0 = __ldg(reinterpret_cast<const uint32_t*>(src));
      } else {
        const uint2 t = __ldg(reinterpret_cast<const uint2*>(src));
        w0 = t.x;
        w1 = t.y;
      }
    }
    float x[8];  // the code as the last bits of 2^23 + code
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t q = BITS == 8 ? __byte_perm(e < 4 ? w0 : w1, 0u, 0x4440 + (e & 3))
                                   : ((w0 >> (BITS * e)) & ((1u << BITS) - 1u));
      x[e] = __uint_as_float(q | 0x4B000000u) - 8388608.f;
    }
    const int a_scale = which ? KVQ_ARRAY_V_SCALE : KVQ_ARRAY_K_SCALE;
    const int a_zero = which ? KVQ_ARRAY_V_ZERO : KVQ_ARRAY_K_ZERO;
    if (c.kch && which == 0) {  // a scale and zero per channel of the block
      const long long h = kch_hdr(c, b, kvh, (pos - c.sink) / c.g) * c.D + ch * 8;
      uint4 s8 = o, z8 = o;
      if (KVQ_IN(c, a_scale, v.scale[0] + h, 16)) s8 = __ldg(reinterpret_cast<const uint4*>(v.scale[0] + h));
      if (KVQ_IN(c, a_zero, v.zero[0] + h, 16)) z8 = __ldg(reinterpret_cast<const uint4*>(v.zero[0] + h));
      const __half* s = reinterpret_cast<const __half*>(&s8);
      const __half* z = reinterpret_cast<const __half*>(&z8);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = (x[e] - __half2float(z[e])) * __half2float(s[e]);
    } else {
      const long long h = row * c.ngroups + ch * 8 / c.g;
      const float s = KVQ_IN(c, a_scale, v.scale[which] + h, 2) ? __half2float(__ldg(v.scale[which] + h)) : 0.f;
      if (BITS == 4 && c.nf4) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = v.nf4_level[(int)x[e]] * s;
      } else {
        float z = (float)(1 << (BITS - 1));
        if (!c.sym)
          z = KVQ_IN(c, a_zero, v.zero[which] + h, 2) ? __half2float(__ldg(v.zero[which] + h)) : 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (x[e] - z) * s;
      }
    }
    o.x = pack_sat(x[0], x[1]);
    o.y = pack_sat(x[2], x[3]);
    o.z = pack_sat(x[4], x[5]);
    o.w = pack_sat(x[6], x[7]);
    if (lo) {
      *lo = make_uint4(pack_rest(x[0], x[1], o.x), pack_rest(x[2], x[3], o.y), pack_rest(x[4], x[5], o.z),
                       pack_rest(x[6], x[7], o.w));
    }
    return o;
  }
}

struct ReadParams {
  CacheView v;
  const int32_t* seq_lens;
  const int32_t* start;
  __half* out[2];  // K, V; either may be null
  uint32_t* status;
  int32_t batch, num_rows;
};

cudaError_t launch_read(const ReadParams& p, cudaStream_t stream);

struct ExtendParams {
  CacheView v;
  const __half* q;  // [batch][num_new][Hq][D]
  __half* out;
  const int32_t* lens_before;
  const int32_t* new_lens;
  float* ws_o;   // [batch * num_new * Hq][splits][D]  (splits > 1)
  float* ws_ml;  // [batch * num_new * Hq][splits][2]
  uint32_t* status;
  int32_t batch, num_new, Hq, G;
  int32_t splits, chunk;  // chunk: positions per split, a multiple of kChunkAlign
  int32_t len_limit;
  float scale_log2;
};

// Which kernel takes the call, the rows of a CTA's tile (query token x head
// of the KV head's group) and its CTAs per SM.
struct ExtendPlan {
  int tile_rows = 0;
  int occ = 0;
  int kind = 0;  // 0: mma.sync kernel, 1 / 2: tensor-core kernel with that many 128-row tiles a CTA
};
cudaError_t extend_plan(const CacheGeom& c, int num_new, int G, ExtendPlan* plan);
cudaError_t launch_extend(const ExtendParams& p, const ExtendPlan& plan, cudaStream_t stream);

}  // namespace kvq
