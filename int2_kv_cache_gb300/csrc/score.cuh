// What kvq_score asks of attention scores, in the base-2 units that the softmaxes work in:
//   a <- cap tanh(a / cap);  a <- a - slope |t - s|;  s is seen by t if (s <= t and s > t - window) or s < prefix
#pragma once
#include "quant_common.cuh"

namespace kvq {

// A slope in base 2, held to where a bias of 2^31 tokens and the scores beside it stay finite.
__device__ __forceinline__ float score_slope(float slope) {
  return fminf(fmaxf(slope * 1.4426950408889634f, -0x1p90f), 0x1p90f);
}

// (tanh(y) / y - 1) / z, z = y^2 <= 0.64, fitted in Chebyshev points (degree 5): tanh off by 1.7e-8 of itself.
constexpr float CAP_FIT = 0.64f;
__host__ __device__ constexpr float tanh_fit_at(int i) {
  return i == 0   ? -0.3333333106652866f
         : i == 1 ? 0.13333072637251825f
         : i == 2 ? -0.05391922212202322f
         : i == 3 ? 0.021526681279575167f
         : i == 4 ? -0.007743903749123501f
                  : 0.001768743788556605f;
}
__device__ __forceinline__ float tanh_fit(float z) {
  float p = tanh_fit_at(5);
#pragma unroll
  for (int i = 4; i >= 0; --i) p = fmaf(z, p, tanh_fit_at(i));
  return p;
}
__device__ __forceinline__ uint64_t tanh_fit2(uint64_t z) {  // two at once
  uint64_t p = f2pk(tanh_fit_at(5), tanh_fit_at(5));
#pragma unroll
  for (int i = 4; i >= 0; --i) p = f2fma(z, p, f2pk(tanh_fit_at(i), tanh_fit_at(i)));
  return p;
}
// tanh y = 1 - 2 / (1 + e^(2 |y|)) with the sign of y beyond the fit.  Within it the same operations as where a whole warp
// stays within: a score's bits do not depend on its neighbours'.
__device__ __forceinline__ float tanh_any(float y) {
  const float z = y * y;
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fabsf(y) * 2.8853900817779268f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return z <= CAP_FIT ? fmaf(y * z, tanh_fit(z), y) : copysignf(fmaf(-2.f, r, 1.f), y);
}

}  // namespace kvq
