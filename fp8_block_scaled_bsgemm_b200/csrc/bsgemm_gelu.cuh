// GELU in its erf form by one exponential, for the activation kernels, whose
// arithmetic would otherwise outlast their memory traffic. (The GEMM's epilogue
// evaluates 1 + erff, with a residual and without, in every plan.)
#pragma once
#include "ptx.cuh"

namespace bsgg {

__device__ __forceinline__ float2 both2(float v) { return make_float2(v, v); }

// GELU and its slope, eight values (a run) at a time.
//
// With u = |z| and the lower tail of the normal distribution T = Phi(-u),
//   z Phi(z)          = max(z, 0) - u T,
//   Phi(z) + z phi(z) = 1/2 + sign(z) (1/2 - T + u phi(u)).
// log2 T is smooth and nearly quadratic in u, so T = 2^P(u) with a polynomial P
// of degree 6: one exponential and no division or case distinction. P is an
// iteratively reweighted least-squares fit (Lawson's method, 6000 Chebyshev
// nodes of [0, 6.5]) that weights the error by T, so T is off by 1.1e-7 at most,
// and falls below 2^-126 before u = 14, where u is clamped. That is coarser than
// 1 + erf in FP32, and a choice: the values go on to 3 or 4 significant bits.
// Largest errors in FP32 (2 million points of each interval), fitted / 1 + erf:
//     z        GELU               GELU / |z|         slope
//   -6..-5   3.0e-8 / 1.6e-7    6.0e-9 / 3.0e-8    5.0e-8 / 3.0e-8
//   -5..-4   3.1e-7 / 8.0e-8    7.7e-8 / 1.6e-8    1.2e-7 / 1.7e-8
//   -4..-3   3.9e-7 / 6.5e-8    1.1e-7 / 1.7e-8    1.5e-7 / 2.0e-8
//   -3..-2   2.8e-7 / 5.1e-8    1.1e-7 / 2.3e-8    1.6e-7 / 4.2e-8
//   -2..0    2.3e-7 / 4.7e-8    1.7e-7 / 5.1e-8    1.9e-7 / 6.2e-8
//    0..2    2.8e-7 / 1.6e-7    1.9e-7 / 1.1e-7    2.4e-7 / 1.4e-7
//    2..14   5.5e-7 / 4.4e-7    1.6e-7 / 1.1e-7    2.2e-7 / 1.2e-7
// Arithmetic, not memory, bounded these kernels at first. On 8192 x 14336 BF16:
// erff alone 30 instructions a value; exp(-u^2/2) times a polynomial of 1 / (1 +
// p u) 110 us (two special-function results a value are 53 us by themselves);
// exp(-u^2/2) times a polynomial of degree 10 in u 94 us.
// The steps of the polynomial run over the run's four pairs side by side: a
// packed instruction takes its constant from a register pair, which is then
// built once per step rather than once per pair and step.
constexpr float kUMax = 14.0f;

__device__ __forceinline__ float exp2_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float2 exp2_approx(float2 v) { return make_float2(exp2_approx(v.x), exp2_approx(v.y)); }

// n = -min(|z|, 14) and T = Phi(n)
__device__ __forceinline__ void normal_tail(const float2 (&z)[4], float2 (&n)[4], float2 (&t)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    n[i] = make_float2(fmaxf(-fabsf(z[i].x), -kUMax), fmaxf(-fabsf(z[i].y), -kUMax));
    t[i] = both2(1.91764611e-5f);
  }
  const float coef[6] = {6.58616424e-4f, 7.75443763e-3f, 5.2965425e-2f, -0.459060252f, 1.15112209f, -0.999999702f};
#pragma unroll
  for (int k = 0; k < 6; ++k) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = bsg::ffma2(t[i], n[i], both2(coef[k]));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = exp2_approx(t[i]);
}

}  // namespace bsgg
