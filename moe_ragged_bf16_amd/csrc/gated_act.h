// The activation of the gated feed-forward's kernels.  Included by .hip files only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gated.h"

namespace mdg {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// act(a) = a s(q(a)), s the logistic function: SiLU, q(a) = a, and GELU in its tanh form,
// q(a) = 2 sqrt(2/pi) (a + 0.044715 a^3).  The hardware's exponential and reciprocal: s is
// off by at most 2^-23 (|q| + 3) relative, far below the bf16 rounding that follows, for the
// |q| < 87 where it is not 0 or 1 (a reciprocal below 2^-126 is 0).  In an epilogue every
// instruction here counts: a wave has its SIMD to itself and no products to run beside
// them (dgrad's, with one formula for both activations, took 108 cycles a value of a
// wave, SiLU's own 76).
__device__ __forceinline__ float logistic(float q_log2e) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-q_log2e));
}

template <int ACT>
struct Act;

template <>
struct Act<kActSilu> {
  static __device__ __forceinline__ float hidden(float a, float b) { return a * logistic(a * kLog2e) * b; }
  // d(hidden)/da and d(hidden)/db, times dh: the slope s + a s (1 - s) is s + s (a - a s)
  static __device__ __forceinline__ void grads(float a, float b, float dh, float* da, float* db) {
    const float s = logistic(a * kLog2e), as = a * s;
    *da = dh * b * __builtin_fmaf(s, a - as, s);
    *db = dh * as;
  }
};

template <>
struct Act<kActGeluTanh> {
  static constexpr float kQ0 = 1.59576912160573071f, kQ1 = kQ0 * 0.044715f;  // q = a (kQ0 + kQ1 a^2)
  // (clamped: past 2^30 the polynomial's derivative would overflow where s (1 - s) is 0)
  static __device__ __forceinline__ float square(float a) { return fminf(a * a, 1152921504606846976.0f); }
  static __device__ __forceinline__ float hidden(float a, float b) {
    return a * logistic(a * __builtin_fmaf(kQ1 * kLog2e, square(a), kQ0 * kLog2e)) * b;
  }
  static __device__ __forceinline__ void grads(float a, float b, float dh, float* da, float* db) {
    const float a2 = square(a), s = logistic(a * __builtin_fmaf(kQ1 * kLog2e, a2, kQ0 * kLog2e)), as = a * s;
    *da = dh * b * __builtin_fmaf(a * (s * (1.0f - s)), __builtin_fmaf(3.0f * kQ1, a2, kQ0), s);
    *db = dh * as;
  }
};

__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

}  // namespace
}  // namespace mdg
