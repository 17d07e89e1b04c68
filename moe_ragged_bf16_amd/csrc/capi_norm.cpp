// C ABI of the norms around a block (include/moe_ragged_bf16.h): argument checks
// before anything is enqueued, launch sizes, launches.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "grouped_gemm.h"
#include "host_common.h"
#include "moe_ragged_bf16.h"
#include "norm.h"

namespace mdg {
namespace {

size_t align256(size_t b) { return (b + 255) / 256 * 256; }
bool real_dtype(int dtype) { return dtype == MDG_BF16 || dtype == MDG_FP32; }
int64_t dtype_bytes(int dtype) { return dtype == MDG_FP32 ? 4 : 2; }

int check_sizes(int64_t tokens, int64_t hidden) {
  if (tokens < 0 || hidden <= 0) return MDG_EINVAL;
  if (tokens > kMaxRows || hidden > kNormMaxHidden || hidden % 8 != 0) return MDG_EUNSUPPORTED;
  return MDG_OK;
}

// Every output apart from every input and from every other output.
template <size_t O, size_t I>
bool apart(const Range (&outs)[O], const Range (&ins)[I]) {
  for (size_t o = 0; o < O; ++o) {
    for (const Range& i : ins)
      if (overlaps(outs[o], i)) return false;
    for (size_t q = 0; q < o; ++q)
      if (overlaps(outs[o], outs[q])) return false;
  }
  return true;
}

Range optional(const void* p, int64_t bytes) { return range_of(p, p ? bytes : 0); }

// Blocks of a gradient call.  More of them keep more rows on their way and leave more
// sums to write and add: 512, and 1024 for long calls of bf16 rows of two waves, which
// leave a SIMD one wave and half of fp32's bytes (512 / 1024 blocks in us, 16384 rows: bf16 of
// 2048 104 / 89, of 1024 39 / 42, fp32 of 2048 151 / 163; 8192 bf16 rows of 4096 84 / 91; bf16 rows
// of 2048: 4096 of them 30.5 / 27.4, 1024 15.4 / 19.0).
int64_t bwd_blocks(int64_t tokens, int64_t hidden, int dtype) {
  const int rows = norm_rows_per_block((int)hidden);
  const bool more = dtype == MDG_BF16 && norm_waves((int)hidden) == 2 && tokens >= 8 * kNormBlocks;
  return std::min<int64_t>((tokens + rows - 1) / rows, more ? kNormManyBlocks : kNormBlocks);
}

size_t part_bytes(int64_t tokens, int64_t hidden) {  // (bf16 has the most)
  return align256((size_t)bwd_blocks(tokens, hidden, MDG_BF16) * 2 * (size_t)hidden * sizeof(float));
}

}  // namespace
}  // namespace mdg

using namespace mdg;

extern "C" {

MDG_API mdg_status block_norm_fwd(const void* residual, const void* y, const void* weight, const void* post_weight,
                                  const float* gate, void* out, void* normed, float* rstd, float* post_rstd,
                                  int64_t tokens, int64_t hidden, int dtype, int weight_dtype, float scale, float eps,
                                  void* stream) {
  int st = check_sizes(tokens, hidden);
  if (st != MDG_OK) return status(st);
  if (!real_dtype(dtype) || !real_dtype(weight_dtype)) return status(MDG_EINVAL);
  if (!isfinite(scale) || !isfinite(eps) || eps < 0.0f) return status(MDG_EINVAL);
  const bool some = tokens > 0;
  if (some && !y && (!weight || post_weight || gate || out)) return status(MDG_EINVAL);
  if (some && (!residual || (y && !out) || !weight != !normed || !weight != !rstd || !post_weight != !post_rstd))
    return status(MDG_EINVAL);
  if (!aligned16(residual) || !aligned16(y) || !aligned16(weight) || !aligned16(post_weight) || !aligned4(gate) ||
      !aligned16(out) || !aligned16(normed) || !aligned4(rstd) || !aligned4(post_rstd))
    return status(MDG_EINVAL);
  const int64_t rows = tokens * hidden * dtype_bytes(dtype), row = hidden * dtype_bytes(weight_dtype);
  const Range ins[5] = {range_of(residual, rows), optional(y, rows), optional(weight, row), optional(post_weight, row),
                        optional(gate, tokens * 4)};
  const Range outs[4] = {optional(out, rows), optional(normed, rows), optional(rstd, tokens * 4),
                         optional(post_rstd, tokens * 4)};
  if (!apart(outs, ins)) return status(MDG_EOVERLAP);
  if (!some) return status(MDG_OK);
  DeviceInfo dev;
  if ((st = check_device(&dev)) != MDG_OK) return status(st);
  NormParams p{};
  p.residual = residual;
  p.y = y;
  p.weight = weight;
  p.post_weight = post_weight;
  p.gate = gate;
  p.out = out;
  p.normed = normed;
  p.rstd = rstd;
  p.post_rstd = post_rstd;
  p.tokens = tokens;
  p.hidden = (int32_t)hidden;
  p.fp32 = dtype == MDG_FP32;
  p.weight_fp32 = weight_dtype == MDG_FP32;
  p.scale = scale;
  p.eps = eps;
  const int waves = norm_waves((int)hidden), per_block = norm_rows_per_block((int)hidden);
  const int64_t cus = dev.cus > 0 ? dev.cus : 256, most = cus * (32 / std::max(waves, 4));
  const int64_t blocks = std::min<int64_t>((tokens + per_block - 1) / per_block, most);
  return status(launch_norm_fwd(p, (int)blocks, static_cast<hipStream_t>(stream)) == hipSuccess ? MDG_OK : MDG_EHIP);
}

MDG_API size_t block_norm_bwd_workspace_bytes(int64_t tokens, int64_t hidden) {
  return check_sizes(tokens, hidden) == MDG_OK ? part_bytes(tokens, hidden) : 0;
}

MDG_API mdg_status block_norm_bwd(const void* dout, const void* dnormed, const void* out, const void* y,
                                  const void* weight, const void* post_weight, const float* gate, const float* rstd,
                                  const float* post_rstd, void* dresidual, void* dy, void* dweight, void* dpost_weight,
                                  float* dgate, int64_t tokens, int64_t hidden, int dtype, int weight_dtype,
                                  float scale, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_sizes(tokens, hidden);
  if (st != MDG_OK) return status(st);
  if (!real_dtype(dtype) || !real_dtype(weight_dtype) || !isfinite(scale)) return status(MDG_EINVAL);
  const bool some = tokens > 0;
  if (!weight && (dnormed || dweight)) return status(MDG_EINVAL);
  if ((!post_weight && dpost_weight) || (!gate && dgate)) return status(MDG_EINVAL);
  if (some && ((!dout && !dnormed) || (dnormed && (!out || !rstd)) || (post_weight && !post_rstd) ||
               ((post_weight || gate) && !y)))
    return status(MDG_EINVAL);
  if (!aligned16(dout) || !aligned16(dnormed) || !aligned16(out) || !aligned16(y) || !aligned16(weight) ||
      !aligned16(post_weight) || !aligned4(gate) || !aligned4(rstd) || !aligned4(post_rstd) || !aligned16(dresidual) ||
      !aligned16(dy) || !aligned16(dweight) || !aligned16(dpost_weight) || !aligned4(dgate))
    return status(MDG_EINVAL);
  const bool sums = dweight || dpost_weight;
  const size_t need = sums ? part_bytes(tokens, hidden) : 0;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MDG_OK) return status(st);
  const int64_t rows = tokens * hidden * dtype_bytes(dtype), row = hidden * dtype_bytes(weight_dtype);
  const Range ins[9] = {optional(dout, rows),       optional(dnormed, rows),    optional(out, rows),
                        optional(y, rows),          optional(weight, row),      optional(post_weight, row),
                        optional(gate, tokens * 4), optional(rstd, tokens * 4), optional(post_rstd, tokens * 4)};
  const Range outs[6] = {optional(dresidual, rows),   optional(dy, rows),         optional(dweight, row),
                         optional(dpost_weight, row), optional(dgate, tokens * 4), range_of(workspace, (int64_t)need)};
  if (!apart(outs, ins)) return status(MDG_EOVERLAP);
  if (!some && !sums) return status(MDG_OK);
  DeviceInfo dev;
  if ((st = check_device(&dev)) != MDG_OK) return status(st);
  NormBwdParams p{};
  p.dout = dout;
  p.dnormed = dnormed;
  p.out = out;
  p.y = y;
  p.weight = weight;
  p.post_weight = post_weight;
  p.gate = gate;
  p.rstd = rstd;
  p.post_rstd = post_rstd;
  p.dresidual = dresidual;
  p.dy = dy;
  p.dweight = dweight;
  p.dpost_weight = dpost_weight;
  p.dgate = dgate;
  p.part = sums ? static_cast<float*>(workspace) : nullptr;
  p.tokens = tokens;
  p.hidden = (int32_t)hidden;
  p.fp32 = dtype == MDG_FP32;
  p.weight_fp32 = weight_dtype == MDG_FP32;
  p.blocks = (int32_t)bwd_blocks(tokens, hidden, dtype);
  p.scale = scale;
  return status(launch_norm_bwd(p, static_cast<hipStream_t>(stream)) == hipSuccess ? MDG_OK : MDG_EHIP);
}

}  // extern "C"
