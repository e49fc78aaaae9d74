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
// the Taylor series, by Horner's rule in units of 2^-62 (each term is smaller
// than the one before, so no intermediate leaves [0, 1]).  Eight and nine
// terms: the first term left out is below 2^-54, and so is the error seen
// over random angles.
//
// Product.  c and s are split into two floats each (48 bits), the products
// with the fp16 values (11 bits) and their sum carry their rounding errors
// along, and the last rounding to fp16 sees the exact side of a tie.  So the
// result is the nearest fp16 to the formula's value, whatever order the
// multiplications are done in; keys quantized from it have the same codes as
// those of any other implementation that rounds correctly.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {
namespace rope {

// cos and sin of one pair, each hi + lo
struct Turn {
  float ch, cl, sh, sl;
};

__device__ __forceinline__ void split_q59(long long v, float& hi, float& lo) {
  const float f = __ll2float_rn(v);
  const long long rest = v - (long long)f;  // |f| <= 2^61: the cast is exact
  hi = f * 0x1p-59f;
  lo = (float)rest * 0x1p-59f;
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
  unsigned long long s = 0x16faeull;
  s = 0x1e8f435ull - __umul64hi(s, w);
  s = 0x1e3074fdfull - __umul64hi(s, w);
  s = 0x150783487eeull - __umul64hi(s, w);
  s = 0x9969667315ecull - __umul64hi(s, w);
  s = 0x28cd78ceeb55c4ull - __umul64hi(s, w);
  s = 0x52aef39896f94b0ull - __umul64hi(s, w);
  s = 0x3243f6a8885a308dull - __umul64hi(s, w);
  s = __umul64hi(s, u);
  unsigned long long c = 0x120cull;
  c = 0x1b6e25ull - __umul64hi(c, w);
  c = 0x1f9d38a3ull - __umul64hi(c, w);
  c = 0x1a6d1f2a20ull - __umul64hi(c, w);
  c = 0xf0fa83448ddull - __umul64hi(c, w);
  c = 0x5574f1f8f2ffeull - __umul64hi(c, w);
  c = 0x103c1f081b5ac3bull - __umul64hi(c, w);
  c = 0x13bd3cc9be45de5aull - __umul64hi(c, w);
  c = 0x4000000000000000ull - __umul64hi(c, w);
  // units of 2^-62 times units of 2^-61, high halves: units of 2^-59
  long long sv = (long long)__umul64hi(s, amplitude);
  const long long cv = (long long)__umul64hi(c, amplitude);
  if (r < 0) sv = -sv;
  const long long x = (quarter & 1) ? -sv : cv;
  const long long y = (quarter & 1) ? cv : sv;
  Turn t;
  split_q59((quarter & 2) ? -x : x, t.ch, t.cl);
  split_q59((quarter & 2) ? -y : y, t.sh, t.sl);
  return t;
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
