// gfx950 (CDNA4) kernels of the norm of many gradients and their clipping.
//
//   norm = sqrt(sum over all tensors of g^2),  g' = g min(1, max_norm / (norm + eps))
//
// A launch takes up to 128 tensors by value in its arguments, so nothing is copied to
// the device and a captured launch keeps its tensors.  Each tensor is cut into units
// of 32 KiB; a workgroup walks units b, b + grid, ..., so the sums' order is a function of
// the sizes.  Squares and sums are in 64 bits: no square of an fp32 value overflows or
// vanishes there, and the fp64 units keep up with memory many times over.  Without
// atomics: results are bitwise reproducible.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "clip.h"
#include "kernel_common.h"

namespace mdg {
namespace {

constexpr int kClipThreads = 256;
constexpr int kSteps = kClipUnitBytes / (kClipThreads * 16);  // 16-byte pieces a thread has of a unit

// 16 bytes that start on an element (tensors may start anywhere in a flat buffer).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// Units of the table's tensors before each one, in LDS; returns their number.
__device__ int clip_units(const ClipTable& t, int* before, int* scratch) {
  int units = 0;
  if ((int)threadIdx.x < t.count) {
    const int64_t n = t.elements[threadIdx.x];
    units = (int)(((n >> 1) * ((n & 1) ? 4 : 2) + kClipUnitBytes - 1) / kClipUnitBytes);
  }
  int total;
  const int b = block_excl_sum(units, scratch, &total);
  if ((int)threadIdx.x < t.count) before[threadIdx.x] = b;
  if (threadIdx.x == 0) before[t.count] = total;
  __syncthreads();
  return total;
}

// One unit: where it starts in its tensor and how many bytes it has.
struct ClipUnit {
  int tensor;
  bool fp32;
  int64_t at;
  int bytes;
};
__device__ __forceinline__ ClipUnit clip_unit(const ClipTable& t, const int* before, int u) {
  ClipUnit x;
  x.tensor = uniform(find_group(before, t.count, u));
  const int64_t n = t.elements[x.tensor];
  x.fp32 = n & 1;
  x.at = (int64_t)(u - uniform(before[x.tensor])) * kClipUnitBytes;
  const int64_t left = (n >> 1) * (x.fp32 ? 4 : 2) - x.at;
  x.bytes = (int)(left < kClipUnitBytes ? left : kClipUnitBytes);
  return x;
}

__device__ __forceinline__ u32x4 load_any(const uint8_t* p) { return *reinterpret_cast<const u32x4_any*>(p); }
// The first `bytes` (below 16) of a piece, zeros behind.
__device__ __forceinline__ u32x4 load_tail(const uint8_t* p, int bytes) {
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (2 * i < bytes) v[i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
  return v;
}
__device__ __forceinline__ void store_tail(uint8_t* p, const u32x4& v, int bytes) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (2 * i < bytes) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
}

// A thread's pieces of a unit: piece i at byte 16 (thread + 256 i).
__device__ __forceinline__ void load_unit(u32x4 (&v)[kSteps], const uint8_t* src, int bytes) {
  if (bytes == kClipUnitBytes) {  // (all but a tensor's last unit)
#pragma unroll
    for (int i = 0; i < kSteps; ++i) v[i] = load_any(src + 16 * (threadIdx.x + kClipThreads * i));
    return;
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int at = 16 * (threadIdx.x + kClipThreads * i);
    if (at + 16 <= bytes) v[i] = load_any(src + at);
    else if (at < bytes) v[i] = load_tail(src + at, bytes - at);
    else v[i] = u32x4{0u, 0u, 0u, 0u};
  }
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}
// The sum over the workgroup, the same bits in every thread.
__device__ __forceinline__ double block_sum(double v, double* scratch) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
  __syncthreads();
  return (scratch[0] + scratch[1]) + (scratch[2] + scratch[3]);
}

__device__ __forceinline__ double square(float f) { return (double)f * (double)f; }

__global__ __launch_bounds__(kClipThreads) void clip_norm_kernel(ClipTable t) {
  __shared__ int s_before[kClipTensors + 1];
  __shared__ int s_scratch[4];
  __shared__ double s_sum[4];
  const int total = clip_units(t, s_before, s_scratch);
  double sum[4] = {0.0, 0.0, 0.0, 0.0};
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    const ClipUnit x = clip_unit(t, s_before, u);
    u32x4 v[kSteps];
    load_unit(v, static_cast<const uint8_t*>(t.src[x.tensor]) + x.at, x.bytes);
    if (x.fp32) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) sum[c] += square(__uint_as_float(v[i][c]));
    } else {
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          sum[c] += square(__uint_as_float(v[i][c] << 16)) + square(__uint_as_float(v[i][c] & 0xffff0000u));
    }
  }
  const double s = block_sum((sum[0] + sum[1]) + (sum[2] + sum[3]), s_sum);
  if (threadIdx.x == 0) t.partial[t.first + blockIdx.x] = s;
}

// The norm from the launches' partial sums, in every thread of a workgroup.
__device__ __forceinline__ double clip_norm(const ClipTable& t, double* scratch) {
  double s = 0.0;
  for (int i = threadIdx.x; i < t.partials; i += kClipThreads) s += t.partial[i];
  return sqrt(block_sum(s, scratch));
}

__global__ __launch_bounds__(kClipThreads) void clip_finish_kernel(ClipTable t) {
  __shared__ double s_sum[4];
  const double norm = clip_norm(t, s_sum);
  if (threadIdx.x == 0) *t.norm_out = (float)norm;
}

// Walks the units from the last one back: what the norm kernel read last is what the
// caches still hold.  In place nothing is written where nothing changes.
__global__ __launch_bounds__(kClipThreads) void clip_scale_kernel(ClipTable t) {
  __shared__ int s_before[kClipTensors + 1];
  __shared__ int s_scratch[4];
  __shared__ double s_sum[4];
  const double norm = t.norm_in ? (double)*t.norm_in : clip_norm(t, s_sum);
  if (t.norm_out && blockIdx.x == 0 && threadIdx.x == 0) *t.norm_out = (float)norm;
  // a norm that is not finite leaves the gradients as they are
  const bool finite = fabsf((float)norm) < __builtin_inff();
  const double by = (double)t.max_norm / (norm + (double)t.eps);
  const float scale = finite && by < 1.0 ? (float)by : 1.0f;
  const int total = clip_units(t, s_before, s_scratch);
  for (int u = total - 1 - (int)blockIdx.x; u >= 0; u -= gridDim.x) {
    const ClipUnit x = clip_unit(t, s_before, u);
    const uint8_t* src = static_cast<const uint8_t*>(t.src[x.tensor]) + x.at;
    uint8_t* dst = static_cast<uint8_t*>(t.dst[x.tensor]) + x.at;
    if (scale == 1.0f && src == dst) continue;
    u32x4 v[kSteps];
    load_unit(v, src, x.bytes);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (scale != 1.0f) {  // (a copy keeps every bit, NaN's too)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (x.fp32) v[i][c] = __float_as_uint(__uint_as_float(v[i][c]) * scale);
          else v[i][c] = pack_bf16x2(__uint_as_float(v[i][c] << 16) * scale,
                                     __uint_as_float(v[i][c] & 0xffff0000u) * scale);
        }
      }
      const int at = 16 * (threadIdx.x + kClipThreads * i);
      if (at + 16 <= x.bytes) *reinterpret_cast<u32x4_any*>(dst + at) = v[i];
      else if (at < x.bytes) store_tail(dst + at, v[i], x.bytes - at);
    }
  }
}

}  // namespace

hipError_t launch_clip_norm(const ClipTable& t, hipStream_t s) {
  hipLaunchKernelGGL(clip_norm_kernel, dim3(t.blocks), dim3(kClipThreads), 0, s, t);
  return hipGetLastError();
}

hipError_t launch_clip_finish(const ClipTable& t, hipStream_t s) {
  hipLaunchKernelGGL(clip_finish_kernel, dim3(1), dim3(kClipThreads), 0, s, t);
  return hipGetLastError();
}

hipError_t launch_clip_scale(const ClipTable& t, int blocks, hipStream_t s) {
  hipLaunchKernelGGL(clip_scale_kernel, dim3(blocks), dim3(kClipThreads), 0, s, t);
  return hipGetLastError();
}

}  // namespace mdg
