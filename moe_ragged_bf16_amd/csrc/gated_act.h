// The activation of the gated feed-forward's kernels.  Included by .hip files only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mdg {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// s(q), q = a (q0 + q1 a^2).  The hardware's exponential and reciprocal: s is off by
// at most 2^-23 (|q| + 3) relative, far below the bf16 rounding that follows, for the
// |q| < 87 where it is not 0 or 1 (a reciprocal below 2^-126 is 0).  (The clamp keeps 0 * inf out of SiLU's q1 = 0.)
struct Act {
  float q0, q1;
  __device__ __forceinline__ float square(float a) const { return fminf(a * a, 1e30f); }
  __device__ __forceinline__ float logistic(float a, float a2) const {
    const float q = a * __builtin_fmaf(q1, a2, q0);
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(q * -kLog2e));
  }
  __device__ __forceinline__ float hidden(float a, float b) const { return a * logistic(a, square(a)) * b; }
  // d(hidden)/da and d(hidden)/db, times dh
  __device__ __forceinline__ void grads(float a, float b, float dh, float* da, float* db) const {
    const float a2 = square(a), s = logistic(a, a2);
    const float slope = __builtin_fmaf(a * (s * (1.0f - s)), __builtin_fmaf(3.0f * q1, a2, q0), s);
    *da = dh * b * slope;
    *db = dh * (a * s);
  }
};

__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

}  // namespace
}  // namespace mdg
