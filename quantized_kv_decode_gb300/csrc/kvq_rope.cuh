// Rotary positions: the angle, its sine and cosine, and the rotated fp16 pair.
//
// Angle.  turns[i] is a pair's rotation per position in units of 2^-64 turns,
// so position * turns[i] in 64-bit wrap-around arithmetic is the angle modulo
// one turn without rounding, at any position.
//
// Sine and cosine.  The angle is cut to r in [-1/8, 1/8] turn and a quarter
// turn count.  With u = |r| / (1/8 turn) and w = u^2 (both in units of 2^-64),
//   sin = u * sum_k (-1)^k (pi/4)^(2k+1) / (2k+1)! w^k,
//   cos =     sum_k (-1)^k (pi/4)^(2k)   / (2k)!   w^k,
// the Taylor series, by Horner's rule: the first three coefficients in units
// of 2^-62 and 64-bit products, the rest, below 2^-11, in 32 bits (units of
// 2^-46 and 2^-53, of 2^-43 and 2^-49).  Eight terms each: the first one left
// out is below 2^-49, and with the 32-bit products' truncation the error seen
// over random angles is below 2^-43.
//
// Product.  c and s are split into two floats each (48 bits), the products
// with the fp16 values (11 bits) and their sum carry their rounding errors
// along, and the last rounding to fp16 sees the exact side of a tie.  So the
// result is the nearest fp16 to the formula's value, whatever order the
// multiplications are done in; keys quantized from it have the same codes as
// those of any other implementation that rounds correctly.  Almost always
// plain fp32 arithmetic settles that: with x lo added up first, the value is
// off by the roundings of the last two sums only, 2^-24 of |x1| a + |y|
// (y0's; a the amplitude) and terms below 2^-46, so where value - E and value
// + E round alike, E = 1.0625 2^-24 max(a, 1) (|x1| + |y|), the long way is
// not taken.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {
namespace rope {

// cos and sin of one pair, each hi + lo
struct Turn {
  float ch, cl, sh, sl;
};

// v in units of 2^-59, |v| < 2^61: the nearest multiple of 2^-23 and the rest
__device__ __forceinline__ void split_q59(long long v, float& hi, float& lo) {
  const long long top = (v + (1ll << 35)) >> 36;  // below 2^25
  hi = (float)(int)top * 0x1p-23f;
  lo = (float)(int)((v - (top << 36)) >> 5) * 0x1p-54f;
}

// amplitude (units of 2^-61, below 2^63) times cos and sin of `frac` turns
// (units of 2^-64)
__device__ __forceinline__ Turn turn_of(unsigned long long frac, unsigned long long amplitude) {
  const unsigned long long quarter = (frac + (1ull << 61)) >> 62;
  const long long r = (long long)(frac - (quarter << 62));
  unsigned long long a = (unsigned long long)(r < 0 ? -r : r);
  a = a < (1ull << 61) ? a : (1ull << 61) - 1;
  const unsigned long long u = a << 3;
  const unsigned long long w = __umul64hi(u, u);
  const uint32_t w32 = (uint32_t)(w >> 32);
  uint32_t t = 0xf47au - __umulhi(0xb8u, w32);
  t = 0xf183a8u - __umulhi(t, w32);
  t = 0xa83c1a44u - __umulhi(t, w32);
  t = 0x99696673u - (__umulhi(t, w32) >> 7);
  unsigned long long s = 0x28cd78ceeb55c4ull - ((unsigned long long)t * w32 >> 16);
  s = 0x52aef39896f94b0ull - __umul64hi(s, w);
  s = 0x3243f6a8885a308dull - __umul64hi(s, w);
  s = __umul64hi(s, u);
  t = 0xfceau - __umulhi(0xdbu, w32);
  t = 0xd368f9u - __umulhi(t, w32);
  t = 0x787d41a2u - __umulhi(t, w32);
  t = 0xaae9e3f2u - (__umulhi(t, w32) >> 6);
  unsigned long long c = 0x103c1f081b5ac3bull - ((unsigned long long)t * w32 >> 13);
  c = 0x13bd3cc9be45de5aull - __umul64hi(c, w);
  c = 0x4000000000000000ull - __umul64hi(c, w);
  // units of 2^-62 times units of 2^-61, high halves: units of 2^-59
  long long sv, cv;
  if (amplitude == 1ull << 61) {
    sv = (long long)(s >> 3);
    cv = (long long)(c >> 3);
  } else {
    sv = (long long)__umul64hi(s, amplitude);
    cv = (long long)__umul64hi(c, amplitude);
  }
  if (r < 0) sv = -sv;
  const long long x = (quarter & 1) ? -sv : cv;
  const long long y = (quarter & 1) ? cv : sv;
  Turn o;
  split_q59((quarter & 2) ? -x : x, o.ch, o.cl);
  split_q59((quarter & 2) ? -y : y, o.sh, o.sl);
  return o;
}

// fp16 nearest to a * (bh + bl) + c * (dh + dl), a and c fp16 values
__device__ __forceinline__ __half dot2_round(float a, float bh, float bl, float c, float dh,
                                             float dl) {
  const float p = __fmul_rn(a, bh), e = __fmaf_rn(a, bh, -p);
  const float q = __fmul_rn(c, dh), f = __fmaf_rn(c, dh, -q);
  const float h = __fadd_rn(p, q);
  const float z = __fadd_rn(h, -p);
  const float err = __fadd_rn(__fadd_rn(p, -__fadd_rn(h, -z)), __fadd_rn(q, -z));
  const float lo = __fadd_rn(__fadd_rn(err, __fadd_rn(e, f)), __fmaf_rn(a, bl, __fmul_rn(c, dl)));
  const float sum = __fadd_rn(h, lo);
  const float rem = __fadd_rn(lo, -__fadd_rn(sum, -h));
  // an even last bit with something left over moves one step towards it, so
  // that the value is on the right side of an fp16 tie (round to odd)
  int bits = __float_as_int(sum);
  if (rem != 0.f && (bits & 1) == 0 && sum != 0.f) bits += ((rem > 0.f) == (sum > 0.f)) ? 1 : -1;
  // an infinity or NaN among the inputs: the plain sum says which
  return __float2half_rn(isfinite(sum) ? __int_as_float(bits) : h);
}

// y0 = x0 c - x1 s, y1 = x1 c + x0 s
__device__ __forceinline__ void rotate_exact(const Turn& t, __half x0, __half x1, __half& y0,
                                             __half& y1) {
  const float a = __half2float(x0), b = __half2float(x1);
  y0 = dot2_round(a, t.ch, t.cl, -b, t.sh, t.sl);
  y1 = dot2_round(b, t.ch, t.cl, a, t.sh, t.sl);
}

// The same for a pair, plainly where that settles the rounding.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n"
      : "=l"(*reinterpret_cast<unsigned long long*>(&d))
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
        "l"(*reinterpret_cast<unsigned long long*>(&c)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;\n"
      : "=l"(*reinterpret_cast<unsigned long long*>(&d))
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return d;
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// y0 in the low half, y1 in the high one.  e: 1.0625 2^-24 max(amplitude, 1).
// sure: whether the rounding is settled; if not, rotate_long tells.
// (The bounds in two-wide arithmetic too take more moves than they save: 4 x 8191
// tokens 75.3 -> 78.4 us, appends of 4 x 8192 264 -> 276, of 256 x 1 9.4 -> 11.1; only
// where few tokens are live do they pay, 1684 of 8190 24.9 -> 22.4.)
__device__ __forceinline__ uint32_t rotate_pair(const Turn& t, float e, float x0, float x1, bool& sure) {
  const float2 x = make_float2(x0, x1), o = make_float2(-x1, x0);
  float2 r = mul2(x, make_float2(t.cl, t.cl));
  r = fma2(o, make_float2(t.sl, t.sl), r);
  r = fma2(o, make_float2(t.sh, t.sh), r);
  r = fma2(x, make_float2(t.ch, t.ch), r);
  const float d0 = __fmul_rn(fabsf(x1) + fabsf(r.x), e), d1 = __fmul_rn(fabsf(x0) + fabsf(r.y), e);
  const uint32_t up = half2_bits(r.x + d0, r.y + d1);
  // (an infinity among the inputs makes a NaN of x lo: the long way tells)
  const __half2 u = *reinterpret_cast<const __half2*>(&up);
  sure = up == half2_bits(r.x - d0, r.y - d1) && __hbeq2(u, u);
  return up;
}
__device__ __forceinline__ uint32_t rotate_long(const Turn& t, float x0, float x1) {
  const __half y0 = dot2_round(x0, t.ch, t.cl, -x1, t.sh, t.sl);
  const __half y1 = dot2_round(x1, t.ch, t.cl, x0, t.sh, t.sl);
  return (uint32_t)__half_as_ushort(y0) | (uint32_t)__half_as_ushort(y1) << 16;
}

__device__ __forceinline__ uint32_t pick(const uint4& v, int i) {
  const uint32_t a = (i & 1) ? v.y : v.x, b = (i & 1) ? v.w : v.z;
  return (i & 2) ? b : a;
}

// N pairs (x0 of pair i in x0[i/2], half i & 1, as fp16 pairs; INTER: pair i
// is x0[i]) turned by t[i * stride]: y0 and y1 laid out as x0 and x1.  The
// pairs that plain arithmetic leaves open are gone over one at a time, so
// that the long way is there once.
template <int N, bool INTER>
__device__ __forceinline__ void rotate_chunk(const Turn* t, int stride, float e, const uint4& x0v, const uint4& x1v,
                                             uint4& y0v, uint4& y1v) {
  const uint32_t x0[4] = {x0v.x, x0v.y, x0v.z, x0v.w}, x1[4] = {x1v.x, x1v.y, x1v.z, x1v.w};
  uint32_t y0[4], y1[4];
  uint32_t open = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t a = INTER ? x0[i] : x0[i >> 1], b = INTER ? 0u : x1[i >> 1];
    const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
    const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
    bool sure;
    const uint32_t r = rotate_pair(t[i * stride], e, (!INTER && (i & 1)) ? fa.y : fa.x,
                                   INTER ? fa.y : (i & 1) ? fb.y : fb.x, sure);
    if (!sure) open |= 1u << i;
    if (INTER) {
      y0[i] = r;
    } else if (i & 1) {
      const uint32_t q = y0[i >> 1];
      y0[i >> 1] = __byte_perm(q, r, 0x5410);
      y1[i >> 1] = __byte_perm(q, r, 0x7632);
    } else {
      y0[i >> 1] = r;
    }
  }
  while (open) {
    const int k = __ffs(open) - 1;
    open &= open - 1;
    const int w = INTER ? k : k >> 1;
    uint32_t a = pick(x0v, w), b = INTER ? 0u : pick(x1v, w);
    if (!INTER && (k & 1)) a >>= 16, b >>= 16;
    const float f0 = __half2float(__ushort_as_half((unsigned short)a));
    const float f1 = __half2float(__ushort_as_half((unsigned short)(INTER ? a >> 16 : b)));
    const uint32_t r = rotate_long(t[k * stride], f0, f1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool here = i == w;
      if (INTER) {
        y0[i] = here ? r : y0[i];
      } else {
        const uint32_t p0 = __byte_perm(y0[i], r, (k & 1) ? 0x5410 : 0x3254);
        const uint32_t p1 = __byte_perm(y1[i], r, (k & 1) ? 0x7610 : 0x3276);
        y0[i] = here ? p0 : y0[i];
        y1[i] = here ? p1 : y1[i];
      }
    }
  }
  y0v = make_uint4(y0[0], y0[1], y0[2], y0[3]);
  if (!INTER) y1v = make_uint4(y1[0], y1[1], y1[2], y1[3]);
}

}  // namespace rope

struct RopeParams {
  kvq_rope rope;
  const __half* q;
  __half* q_out;
  const __half* k;  // kvq_rope_apply only
  __half* k_out;
  const int32_t* positions;
  const int32_t* seq_lens_before;
  const int32_t* new_lens;
  uint32_t* status;
  int32_t D, batch, num_new, Hq, Hk;
};

struct RopeAppendParams {
  AppendParams a;
  RopeParams r;  // q (Hq = 0: none); k unused
};

// Several axes: pair i turns by at[token][axis[i]]; the cache rows of an
// append still follow r.seq_lens_before.
struct RopeAxesParams : RopeAppendParams {
  const int32_t* at;  // [batch][num_new][num_axes]
  int32_t num_axes;
  uint8_t axis[KVQ_ROPE_MAX_PAIRS];
};

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream);
cudaError_t launch_rope_append(const RopeAppendParams& p, cudaStream_t stream);
cudaError_t launch_rope_axes(const RopeAxesParams& p, cudaStream_t stream);
cudaError_t launch_rope_axes_append(const RopeAxesParams& p, cudaStream_t stream);

}  // namespace kvq
