// The logistic function and 2^t in fp64, to 2^-44 instead of the library's 2^-52: what is rounded
// to fp32 afterwards loses nothing that shows (one value in 2^18 at most may go to its other
// neighbour), and choices among scores that differ by less than that are nobody's.  On
// this chip an fp64 operation, conversion or rounding takes the four clocks of an fp32 one
// (a reciprocal sixteen), so what counts is how many there are.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rfp2 {

constexpr double kLog2E = 1.4426950408889634074;
constexpr double kRound = 6755399441055744.0;   // 1.5 * 2^52: a sum with it ends at the units

// 2^(n + f) for whole n, |n| <= 1000, handed over as m = n + kRound (its low word is n), and
// |f| <= 1/2 or little more, within 2^-45 of it: 2^f by the polynomial of degree 9 that
// meets it at the ten Chebyshev points of [-1/2, 1/2], n added to the exponent.
__device__ __forceinline__ double exp2_parts(double m, double f) {
  double p = 1.0205905413765595e-07;
  p = fma(p, f, 1.325964524488711e-06);
  p = fma(p, f, 1.5252672924850737e-05);
  p = fma(p, f, 0.0001540343375125101);
  p = fma(p, f, 0.0013333558200794592);
  p = fma(p, f, 0.009618129193934313);
  p = fma(p, f, 0.05550410866465167);
  p = fma(p, f, 0.2402265069564034);
  p = fma(p, f, 0.6931471805599462);
  p = fma(p, f, 1.0000000000000135);
  const uint64_t b = __builtin_bit_cast(uint64_t, p);
  const uint32_t n = (uint32_t)__builtin_bit_cast(uint64_t, m);
  return __builtin_bit_cast(double, b + ((uint64_t)(n << 20) << 32));
}

// 1 / (1 + 2^(n + f)) within 2^-44 of it.
__device__ __forceinline__ double logistic_parts(double m, double f) {
  const double d = 1.0 + exp2_parts(m, f);
  const double r = __builtin_amdgcn_rcp(d);
  return fma(r, fma(-d, r, 1.0), r);
}

// exp(x) for x in [-690, 690], within 2^-44 of it (2^-45.0 the farthest of 4 million).
__device__ __forceinline__ double exp_f64(double x) {
  const double m = fma(x, kLog2E, kRound);
  return exp2_parts(m, fma(x, kLog2E, kRound - m));
}

// 1 / (1 + exp(-x)) for x in [-690, 690], within 2^-44 of it (2^-45.0 the farthest seen).
__device__ __forceinline__ double logistic(double x) {
  const double m = fma(x, -kLog2E, kRound);
  return logistic_parts(m, fma(x, -kLog2E, kRound - m));
}

}  // namespace rfp2
