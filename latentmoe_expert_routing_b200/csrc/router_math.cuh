// The router's fp64 exponential and sigmoid, shared by the layer's router and
// the stand-alone routing calls so that both give the same bits.
#pragma once
#include <cuda_runtime.h>

namespace lmoe {

// ---------------------------------------------------------------------------
// exp in fp64 from IEEE +, *, rint and an exact power-of-two multiply: a = n ln2 + r with a
// two-part (Cody-Waite) ln 2 whose high part has 32 significant bits, then the
// degree-13 Taylor polynomial of exp(r) by Horner.  The explicit _rn
// intrinsics keep the compiler from contracting a*b+c into an FMA, so the
// result is the same bit pattern on any IEEE machine that does the same steps.
// ---------------------------------------------------------------------------
__device__ __forceinline__ double exp_fixed(double a) {
  const double kInvLn2 = 0x1.71547652b82fep+0;
  const double kLn2Hi = 0x1.62e42fee00000p-1;
  const double kLn2Lo = 0x1.a39ef35793c76p-33;
  const double c[14] = {0x1.0000000000000p+0, 0x1.0000000000000p+0, 0x1.0000000000000p-1,
                        0x1.5555555555555p-3, 0x1.5555555555555p-5, 0x1.1111111111111p-7,
                        0x1.6c16c16c16c17p-10, 0x1.a01a01a01a01ap-13, 0x1.a01a01a01a01ap-16,
                        0x1.71de3a556c734p-19, 0x1.27e4fb7789f5cp-22, 0x1.ae64567f544e4p-26,
                        0x1.1eed8eff8d898p-29, 0x1.6124613a86d09p-33};
  double n = rint(__dmul_rn(a, kInvLn2));
  double r = __dsub_rn(__dsub_rn(a, __dmul_rn(n, kLn2Hi)), __dmul_rn(n, kLn2Lo));
  double p = c[13];
#pragma unroll
  for (int i = 12; i >= 0; --i) p = __dadd_rn(__dmul_rn(p, r), c[i]);
  // p * 2^n with 2^n built from its exponent bits: |n| <= 116 keeps both 2^n and
  // the product normal, so the multiply is exact (the same value scalbn gives)
  return __dmul_rn(p, __longlong_as_double((long long)((int)n + 1023) << 52));
}

__device__ __forceinline__ float sigmoid_fixed(float l) {
  double a = -fmin(fmax((double)l, -80.0), 80.0);
  return __double2float_rn(__ddiv_rn(1.0, __dadd_rn(1.0, exp_fixed(a))));
}

}  // namespace lmoe
