// Rows of fp32 values four to a lane, and their int8 form: what the kernels that write
// activations share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rfp2 {

template <bool NT = false>
__device__ __forceinline__ void load4(float (&x)[4], const float* p) {
  typedef float vec4 __attribute__((ext_vector_type(4)));
  vec4 v;
  if constexpr (NT) v = __builtin_nontemporal_load(reinterpret_cast<const vec4*>(p));
  else v = *reinterpret_cast<const vec4*>(p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}

// Sixteen bytes to memory that nobody reads soon: past the caches (NT), which a large
// output would only sweep.  Read-back of 20011 tokens of 8 heads of 128: 53.2 us with
// ordinary stores, 34.6 us so.
template <bool NT>
__device__ __forceinline__ void store4(float* p, float4 x) {
  typedef float vec4 __attribute__((ext_vector_type(4)));
  const vec4 v = {x.x, x.y, x.z, x.w};
  if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<vec4*>(p));
  else *reinterpret_cast<vec4*>(p) = v;
}

// 1 / d to the last bit: the chip's estimate (2^-24.4 off at most of 4 million), corrected twice
// (2^-53.0).
__device__ __forceinline__ double reciprocal(double d) {
  double r = __builtin_amdgcn_rcp(d);
  r = fma(r, fma(-d, r, 1.0), r);
  return fma(r, fma(-d, r, 1.0), r);
}

// 1 / sqrt(m) to the last bits, the same way (estimate 2^-24.2, corrected 2^-52.7; 0 for
// infinity): nine instructions one after
// another where the library's root and division are some sixty (one row of 4096 normed:
// 2.9 us with those, 2.6 so).
__device__ __forceinline__ double inverse_root(double m) {
  double r = __builtin_amdgcn_rsq(m);
  r = fma(0.5 * r, fma(-m * r, r, 1.0), r);
  r = fma(0.5 * r, fma(-m * r, r, 1.0), r);
  return m == INFINITY ? 0.0 : r;
}

// Code and scale as quantize_acts_kernel computes them, of N (4 or 8) values of
// each of the 32 / N neighbouring lanes of a block.  Magnitudes are compared as integers,
// where infinities and NaN are the largest.
//
// The two divisions are fp64 products with a reciprocal, rounded to fp32: the same bits as
// a division of fp32 numbers.  A quotient X 2^a / (D 2^b) of 24-bit whole numbers is no
// midpoint M 2^c of fp32 numbers (M odd of 25 bits would have to divide X), so X 2^s and
// M D, whole numbers below 2^49, differ by 1 or more: the quotient is 2^-49 of itself or
// further from a midpoint, and the product (two roundings, 2^-52) on the right side of it.
// (max / 127 may fall below the normal numbers, where midpoints are the odd multiples of
// 2^-150: 127 times one is none of max's multiples of 2^-149.)  A code is that quotient,
// at most 190 (127 but for a subnormal scale), plus the number before 1/2, cut off: the sum
// reaches the next whole number from the half on and from nowhere below.
template <int N>
__device__ __forceinline__ float quantize_block(const float (&x)[N], uint32_t (&codes)[N / 4]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  // over the lanes: neighbours, pairs, then the other four of eight in reverse
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, true));
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xF, 0xF, true));
  if (N == 4)
    top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x141, 0xF, 0xF, true));
  const bool finite = top < 0x7F800000u;
  const float scale =
      finite ? (float)((double)__uint_as_float(top) * (1.0 / 127.0)) : __builtin_nanf("");
#pragma unroll
  for (int i = 0; i < N / 4; ++i) codes[i] = 0;
  if (finite && scale != 0.0f) {
    const double inv = reciprocal((double)scale);
    uint32_t c[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float r = (float)((double)x[i] * inv);
      c[i] = (uint32_t)min(max((int)(r + copysignf(0x1.fffffep-2f, r)), -127), 127);
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      codes[i] = __builtin_amdgcn_perm(c[4 * i + 3], c[4 * i + 2], 0x04000C0Cu) |
                 __builtin_amdgcn_perm(c[4 * i + 1], c[4 * i], 0x0C0C0400u);
  }
  return scale;
}
__device__ __forceinline__ float quantize4(const float (&x)[4], uint32_t& codes) {
  uint32_t c[1];
  const float scale = quantize_block<4>(x, c);
  codes = c[0];
  return scale;
}

// The sum over every group of G neighbouring lanes, in all of them (G from 8 to 64; fp64:
// whatever the order, the rounding to fp32 afterwards does not see it).
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp_add(double s) {
  const uint64_t b = __builtin_bit_cast(uint64_t, s);
  const uint32_t lo =
      __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, ROWS == 0xF);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, ROWS, 0xF, ROWS == 0xF);
  return s + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
template <int G>
__device__ __forceinline__ double group_sum(double s) {
  s = dpp_add<0xB1>(s);                      // neighbours
  s = dpp_add<0x4E>(s);                      // pairs
  s = dpp_add<0x141>(s);                     // the other four of eight, in reverse
  if constexpr (G >= 16) s = dpp_add<0x140>(s);   // the other eight of sixteen, in reverse
  if constexpr (G >= 32) s += __shfl_xor(s, 16, 64);
  if constexpr (G >= 64) s += __shfl_xor(s, 32, 64);
  return s;
}
// The sum over the wave, in its last lane alone (no trip through the LDS).
__device__ __forceinline__ double sum_in_last_lane(double s) {
  s = group_sum<16>(s);
  s = dpp_add<0x142, 0xA>(s);                // rows 1 and 3: the row before
  return dpp_add<0x143, 0xC>(s);             // rows 2 and 3: the two before
}

}  // namespace rfp2
