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
// those of any other implementation that rounds correctly.  Almost always a
// plain fp32 product settles that: its error is below E = 2^-22 max(a, 1)
// (|x0| + |x1|) (two roundings of 2^-24 and the coefficients' 2^-24), so
// where value - E and value + E round alike the long way is not taken (one
// pair in about 500 takes it).
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

// The same for a pair, plainly where that settles the rounding.  hi: (c, s);
// lo is read only if need be.  e: 2^-22 max(amplitude, 1).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n"
      : "=l"(*reinterpret_cast<unsigned long long*>(&d))
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
        "l"(*reinterpret_cast<unsigned long long*>(&c)));
  return d;
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// y0 in the low half, y1 in the high one
__device__ __forceinline__ uint32_t rotate_pair(float2 hi, const float2* lo, float e, float x0, float x1) {
  const float2 r = fma2(make_float2(x0, x1), make_float2(hi.x, hi.x), make_float2(__fmul_rn(-x1, hi.y), __fmul_rn(x0, hi.y)));
  const float d = __fmul_rn(fabsf(x0) + fabsf(x1), e);
  const uint32_t up = half2_bits(r.x + d, r.y + d);
  if (up == half2_bits(r.x - d, r.y - d)) return up;
  const float2 l = *lo;
  const __half y0 = dot2_round(x0, hi.x, l.x, -x1, hi.y, l.y);
  const __half y1 = dot2_round(x1, hi.x, l.x, x0, hi.y, l.y);
  return (uint32_t)__half_as_ushort(y0) | (uint32_t)__half_as_ushort(y1) << 16;
}

}  // namespace rope

// Which rows of a padded batch sequence b has: new_lens[b], or num_new
// without the array; -1 for a value outside [0, num_new].
__device__ __forceinline__ int new_rows_of(const int32_t* new_lens, int b, int num_new) {
  if (!new_lens) return num_new;
  const int n = __ldg(new_lens + b);
  return (n < 0 || n > num_new) ? -1 : n;
}

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

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream);
cudaError_t launch_rope_append(const RopeAppendParams& p, cudaStream_t stream);

}  // namespace kvq
