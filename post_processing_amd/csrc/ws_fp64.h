// ws_fp64.h -- the exponential a teacher's few listed tokens need in FP64.
// Internal to the library; plain arithmetic, so that a host compiler can test
// the same code.
#pragma once

#include <cmath>

#ifdef __HIPCC__
#define WS_FP64_FN __device__ __forceinline__
#else
#define WS_FP64_FN inline
#endif

namespace ws {

// e^x in FP64 to 3e-16 relative; 0 below -200.  Argument reduction after Cody
// and Waite, x = n log 2 + r with |r| <= 0.3466 and log 2 in two parts (their
// products exact in a fused multiply-add, so r is off by 6e-17), then the
// exponential's series to r^13 / 13!, whose next term is 5e-18.  Near 0 the
// error is half a step of the result, which 1 minus a sum of such needs: squaring
// e^(x / 1024) ten times instead was off by 2e-14 there and by 8e-11 at -88.
// Written out, as a library routine's constants would crowd the registers of a
// held row.
WS_FP64_FN double small_exp(double x) {
    if (x < -200.0) return 0.0;
    if (x > 710.0) x = 710.0;   // infinite from 709.8 on; NaN stays
    const double n = rint(x * 1.4426950408889634);
    double r = fma(n, -0.6931471805599453, x);
    r = fma(n, -2.3190468138462996e-17, r);
    double e = 1.0 / 6227020800.0;
    e = fma(e, r, 1.0 / 479001600.0);
    e = fma(e, r, 1.0 / 39916800.0);
    e = fma(e, r, 1.0 / 3628800.0);
    e = fma(e, r, 1.0 / 362880.0);
    e = fma(e, r, 1.0 / 40320.0);
    e = fma(e, r, 1.0 / 5040.0);
    e = fma(e, r, 1.0 / 720.0);
    e = fma(e, r, 1.0 / 120.0);
    e = fma(e, r, 1.0 / 24.0);
    e = fma(e, r, 1.0 / 6.0);
    e = fma(e, r, 0.5);
    e = fma(e, r, 1.0);
    e = fma(e, r, 1.0);
    return ldexp(e, n == n ? (int)n : 0);
}

}  // namespace ws
