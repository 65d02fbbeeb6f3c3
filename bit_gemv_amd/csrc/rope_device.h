// Rotary positions inside a kernel: the workgroup computes the cosines and
// sines of its token's angles once, into LDS, and every head is rotated with
// them.
//
// Pair i of a head turns by the angle pos * f_i.  In fp32 the angle of
// position 10^6 is off by 2^-24 * 10^6 = 0.06 radians, so it is formed in
// fp64 and reduced to a fraction of a turn there; the product and 1 / (2 pi)
// are held in two numbers each, since one rounding of the number of turns is
// 2^-53 of ALL turns: at position 2^31 a whole last place of fp32, at 10^6 still
// enough to round one value in a thousand the other way.  So the fraction is off by
// a few units of 2^-53 at any position.  Cosine, sine and the rotation itself stay in
// fp64 too and the rotated value is rounded to fp32 once.  That makes the value
// reproducible (it is the correctly rounded one but where the exact value lies
// within some 2^-50 of the pair's size of the border), which matters where it is
// quantized to int8 next: a last-bit difference would flip codes.  The fp64 work is one
// sincos per pair and token and four multiplications and additions per pair and
// head, under the time of the transfer: 4096 tokens of 40 heads of 128 values are
// rotated in 26 us, 6.4 TB/s read and written.
#pragma once

#include "rfp2_internal.h"

namespace rfp2 {

// mscale * (cos, sin) of pair i's angle at position pos.
__device__ __forceinline__ double2 rope_entry(const RopeView& r, int32_t pos, int i) {
#pragma clang fp contract(off)              // `turns` is the rounded product wherever it stands
  // 1 / (2 pi) = hi + lo
  constexpr double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  const double f = r.freqs[i], p = (double)pos;
  const double a = p * f, a_lo = __builtin_fma(p, f, -a);
  const double turns = a * hi;
  const double rest = __builtin_fma(a, hi, -turns) + __builtin_fma(a, lo, a_lo * hi);
  double s, c;
  sincospi(2.0 * ((turns - rint(turns)) + rest), &s, &c);
  return make_double2(r.mscale * c, r.mscale * s);
}

// One value of a pair, turned: x itself, o its partner; `first`: x is the pair's first
// value.  The product is rounded, then fused with the other, in every kernel alike.
__device__ __forceinline__ float rope_value(float x, float o, double2 cs, bool first) {
  const double p = (double)o * cs.y;
  return (float)__builtin_fma((double)x, cs.x, first ? -p : p);
}

// (x1, x2) turned by one pair's cosine and sine.
__device__ __forceinline__ float2 rope_turn(float x1, float x2, double2 cs) {
  return make_float2(rope_value(x1, x2, cs, true), rope_value(x2, x1, cs, false));
}

}  // namespace rfp2
