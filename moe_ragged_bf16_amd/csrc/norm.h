// Internal interface between the C ABI (capi_norm.cpp) and the gfx950 kernels of
// the norms around a block (norm_kernels.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mdg {

constexpr int kNormMaxHidden = 16384;
// Blocks of a gradient call, each of which leaves a row of partial sums: up to the first
// number, or for long calls of some widths up to the second (bwd_blocks of capi_norm.cpp).
constexpr int kNormBlocks = 512, kNormManyBlocks = 1024;

struct NormParams {
  const void* residual;     // [tokens, hidden]
  const void* y;            // [tokens, hidden]; nullptr: out is the residual
  const void* weight;       // [hidden]; nullptr: no norm of out
  const void* post_weight;  // [hidden]; nullptr: no norm of y
  const float* gate;        // [tokens]; nullptr: ones
  void* out;                // [tokens, hidden]; not written without y
  void* normed;             // [tokens, hidden]
  float* rstd;              // [tokens]
  float* post_rstd;         // [tokens]
  int64_t tokens;
  int32_t hidden, fp32, weight_fp32;
  float scale, eps;
};

struct NormBwdParams {
  const void* dout;         // nullptr: zeros
  const void* dnormed;      // nullptr: zeros
  const void* out;
  const void* y;
  const void* weight;
  const void* post_weight;
  const float* gate;
  const float* rstd;
  const float* post_rstd;
  void* dresidual;          // outputs: each may be nullptr (not wanted)
  void* dy;
  void* dweight;            // [hidden] of the weights' type
  void* dpost_weight;
  float* dgate;             // [tokens]
  float* part;              // [blocks, 2, hidden] workspace: the blocks' sums for the two weights
  int64_t tokens;
  int32_t hidden, fp32, weight_fp32, blocks;
  float scale;
};

// Waves that share a row, 16 values a lane (8 for the narrowest rows).
constexpr int norm_waves(int hidden) {
  int w = 1;
  while (w * 64 * 16 < hidden) w *= 2;
  return w;
}
constexpr int norm_rows_per_block(int hidden) { return norm_waves(hidden) == 1 ? 4 : 1; }

hipError_t launch_norm_fwd(const NormParams& p, int blocks, hipStream_t s);
hipError_t launch_norm_bwd(const NormBwdParams& p, hipStream_t s);

}  // namespace mdg
