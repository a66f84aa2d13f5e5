// exp64.hpp -- an exponential and a reciprocal in binary64, exact enough to be
// rounded to binary32 afterwards (off by at most 2^-46.6 of the value; a
// rounding to binary32 is then that of the exact value but for one case in
// 2^21.6 where the error is largest, and goes to the other neighbour there),
// in about half the instructions of the math library's.
#pragma once

#include <hip/hip_runtime.h>

namespace coli {

// exp(x): x = n ln 2 + r with |r| <= ln 2 / 2, and the Taylor series of e^r
// up to r^11 (the rest, r^12 / 12! and smaller terms, is below 2^-46.6 of the
// result: most at r = -ln 2 / 2, where it is 2^-46.7).  Past +-1100 it is 0 or
// infinity, whatever x.
__device__ __forceinline__ double exp_64(double x) {
  x = __builtin_fmin(__builtin_fmax(x, -1100.0), 1100.0);
  const double n = __builtin_rint(x * 1.4426950408889634);
  double r = __builtin_fma(n, -0x1.62e42fefa39efp-1, x);
  r = __builtin_fma(n, -0x1.abc9e3b39803fp-56, r);
  double p = 1.0 / 39916800;
  p = __builtin_fma(p, r, 1.0 / 3628800);
  p = __builtin_fma(p, r, 1.0 / 362880);
  p = __builtin_fma(p, r, 1.0 / 40320);
  p = __builtin_fma(p, r, 1.0 / 5040);
  p = __builtin_fma(p, r, 1.0 / 720);
  p = __builtin_fma(p, r, 1.0 / 120);
  p = __builtin_fma(p, r, 1.0 / 24);
  p = __builtin_fma(p, r, 1.0 / 6);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)n);
}

// 1 / x for x >= 1: the hardware's estimate and two Newton steps; 0 for an
// infinity.
__device__ __forceinline__ double inverse_64(double x) {
  double y = __builtin_amdgcn_rcp(x);
  if (x > 1e300) return y;
  y = __builtin_fma(__builtin_fma(-x, y, 1.0), y, y);
  return __builtin_fma(__builtin_fma(-x, y, 1.0), y, y);
}

}  // namespace coli
