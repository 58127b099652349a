// mx_ortho.cuh -- what the two forms of the Newton-Schulz orthogonalisation share.
#pragma once
#include <cuda_runtime.h>
#include <cmath>

namespace mxk {

constexpr int kNsMaxSteps = 16;
constexpr int kNsLogSA = 12;  // A and B are held times 2^12

// How small X may be before a step.  Its singular values start at most at
// rho = |G|_F / (|G|_F + eps), and a step multiplies s by |a + b s^2 + c s^4|; the
// call has checked that they stay below 3.9.  Where this bound is small (eps much
// larger than G, or coefficients that shrink) X as it is would fall out of FP16's
// range, and a X is nearly all of the step.
__host__ __device__ inline float ns_next_bound(float u, const float* coeffs) {
  const float t = u * u;
  const float v = u * (fabsf(coeffs[0]) + fabsf(coeffs[1]) * t + fabsf(coeffs[2]) * t * t);
  return v < 3.9f ? v : 3.9f;
}
constexpr float kNsSmall = 0.0625f;

}  // namespace mxk
