// gfx950 (CDNA4) kernels of the norm of many gradients and their clipping.
//
//   norm = sqrt(sum over all tensors of g^2),  g' = g min(1, max_norm / (norm + eps))
//
// A launch takes up to 336 tensors by value in its arguments, so nothing is copied to
// the device and a captured launch keeps its tensors.  Each tensor is cut into units
// of 32 KiB; a workgroup walks units b, b + grid, ..., so the sums' order is a function of
// the sizes.  Squares and sums are in 64 bits: no square of an fp32 value overflows or
// vanishes there, and the fp64 units keep up with memory many times over.  Without
// atomics: results are bitwise reproducible.
//
// Memory bounds both kernels: 604 million fp32 values in two tensors (403 and 201 million; 2.4 GB
// read twice, written once) take 422 us for the norm (5.7 TB/s) and 907 to scale (5.3 TB/s read and
// written); 301 tensors of 60 million values in all 133 (139 in two launches of each).  Nine tensors of
// 0.3 million take 10.8: two launches, one waiting for the other's sums, 4.8 and 7.0.

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

// Addresses come from a table: their memory is said here, or accesses would be flat ones.
typedef __attribute__((address_space(1))) uint8_t gbyte;
typedef __attribute__((address_space(1))) uint16_t ghalf;
typedef __attribute__((address_space(1))) float gfloat;
typedef __attribute__((address_space(1))) u32x4_any gpiece;

// The table in LDS: addresses, sizes (2 elements + (1: fp32)) and the units of the
// tensors before each one.
struct ClipLds {
  uint64_t src[clip_tensors(false)], dst[clip_tensors(false)], elements[clip_tensors(false)];
  int before[clip_tensors(false) + 1];
  int scratch[4];
};
static_assert(clip_tensors(false) <= 2 * kClipThreads, "two tensors to a thread");
static_assert(kClipPartials == 4 * kClipThreads, "four partial sums to a thread");

// Fills it; returns the number of units.
__device__ __forceinline__ int clip_units(const ClipTable& t, ClipLds& s) {
  const int capacity = clip_tensors(t.apart);
  int units[2] = {0, 0};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = 2 * threadIdx.x + q;
    if (i >= t.count) continue;
    const uint32_t mid = t.words[capacity + i];
    const uint64_t src = (uint64_t)(mid & 0xffffu) << 32 | t.words[i];
    const uint64_t n = (uint64_t)(mid >> 16) << 32 | t.words[2 * capacity + i];
    s.src[i] = src;
    s.elements[i] = n;
    s.dst[i] = t.apart ? (uint64_t)t.words[4 * capacity + i] << 32 | t.words[3 * capacity + i] : src;
    units[q] = (int)(((int64_t)(n >> 1) * ((n & 1) ? 4 : 2) + kClipUnitBytes - 1) / kClipUnitBytes);
  }
  int total;
  const int b = block_excl_sum(units[0] + units[1], s.scratch, &total), i = 2 * threadIdx.x;
  if (i < t.count) s.before[i] = b;
  if (i + 1 < t.count) s.before[i + 1] = b + units[0];
  if (i == 0) s.before[t.count] = total;
  __syncthreads();
  return total;
}

// One unit: its tensor, where it starts and how many bytes it has.
struct ClipUnit {
  const gbyte* src;
  gbyte* dst;
  bool fp32;
  int bytes;
};
__device__ __forceinline__ ClipUnit clip_unit(const ClipTable& t, const ClipLds& s, int u) {
  ClipUnit x;
  const int i = uniform(find_group(s.before, t.count, u));
  const uint64_t n = s.elements[i];
  x.fp32 = uniform((int)(n & 1));
  const int64_t at = (int64_t)(u - s.before[i]) * kClipUnitBytes;
  const int64_t left = (int64_t)(n >> 1) * (x.fp32 ? 4 : 2) - at;
  x.bytes = uniform((int)(left < kClipUnitBytes ? left : kClipUnitBytes));
  x.src = reinterpret_cast<const gbyte*>(s.src[i]) + at;
  x.dst = reinterpret_cast<gbyte*>(s.dst[i]) + at;
  return x;
}

__device__ __forceinline__ u32x4 load_any(const gbyte* p) { return *reinterpret_cast<const gpiece*>(p); }

// A thread's pieces of a unit: piece i at byte 16 (thread + 256 i), zeros where the unit
// has no whole piece.
__device__ __forceinline__ void load_unit(u32x4 (&v)[kSteps], const gbyte* src, int bytes) {
  if (bytes == kClipUnitBytes) {  // (all but a tensor's last unit)
#pragma unroll
    for (int i = 0; i < kSteps; ++i) v[i] = load_any(src + 16 * (threadIdx.x + kClipThreads * i));
    return;
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int at = 16 * (threadIdx.x + kClipThreads * i);
    v[i] = u32x4{0u, 0u, 0u, 0u};
    if (at + 16 <= bytes) v[i] = load_any(src + at);
  }
}

// The elements behind a unit's whole pieces (fewer than 16 bytes), one to a thread: this
// thread's, at byte *at; false where it has none.
__device__ __forceinline__ bool rest_of(const ClipUnit& x, int* at) {
  *at = (x.bytes & ~15) + (int)threadIdx.x * (x.fp32 ? 4 : 2);
  return *at < x.bytes;
}
__device__ __forceinline__ float load_one(const ClipUnit& x, int at) {
  if (x.fp32) return *reinterpret_cast<const gfloat*>(x.src + at);
  return __uint_as_float((uint32_t)*reinterpret_cast<const ghalf*>(x.src + at) << 16);
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
  __shared__ ClipLds s_table;
  __shared__ double s_sum[4];
  const int total = clip_units(t, s_table);
  double sum[4] = {0.0, 0.0, 0.0, 0.0};
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    const ClipUnit x = clip_unit(t, s_table, u);
    u32x4 v[kSteps];
    load_unit(v, x.src, x.bytes);
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
    int at;
    if (rest_of(x, &at)) sum[0] += square(load_one(x, at));
  }
  const double s = block_sum((sum[0] + sum[1]) + (sum[2] + sum[3]), s_sum);
  if (threadIdx.x == 0) t.partial[t.first + blockIdx.x] = s;
}

// This thread's share of the launches' partial sums, its first loads apart from their use;
// ALL: any number of them, otherwise up to kClipPartials.
struct Partials {
  double first[4];
  __device__ __forceinline__ void load(const ClipTable& t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = threadIdx.x + kClipThreads * i;
      first[i] = at < t.partials ? t.partial[at] : 0.0;
    }
  }
  template <bool ALL>
  __device__ __forceinline__ double sum(const ClipTable& t) const {
    double s = (first[0] + first[1]) + (first[2] + first[3]);
    if constexpr (ALL)
      for (int i = threadIdx.x + kClipPartials; i < t.partials; i += kClipThreads) s += t.partial[i];
    return s;
  }
};

__global__ __launch_bounds__(kClipThreads) void clip_finish_kernel(ClipTable t) {
  __shared__ double s_sum[4];
  Partials mine;
  mine.load(t);
  const double norm = sqrt(block_sum(mine.sum<true>(t), s_sum));
  if (threadIdx.x != 0) return;
  if (t.norm_out) *t.norm_out = (float)norm;
  else t.partial[0] = norm;  // (every thread has its sums: a barrier lies between)
}

// Walks the units from the last one back: what the norm kernel read last is what the
// caches still hold.  In place nothing is written where nothing changes.  A workgroup's
// first unit loads while the norm is added up.
__global__ __launch_bounds__(kClipThreads, 6) void clip_scale_kernel(ClipTable t) {
  __shared__ ClipLds s_table;
  __shared__ double s_sum[4];
  Partials mine;
  mine.load(t);  // (none with a norm given or finished)
  const int total = clip_units(t, s_table);
  int u = total - 1 - (int)blockIdx.x;
  ClipUnit x{};
  u32x4 v[kSteps];
  if (u >= 0) {
    x = clip_unit(t, s_table, u);
    load_unit(v, x.src, x.bytes);
  }
  const double norm = t.norm_in    ? (double)*t.norm_in
                      : t.finished ? t.partial[0]
                                   : sqrt(block_sum(mine.sum<false>(t), s_sum));
  if (t.norm_out && blockIdx.x == 0 && threadIdx.x == 0) *t.norm_out = (float)norm;
  // a norm that is not finite leaves the gradients as they are
  const bool finite = fabsf((float)norm) < __builtin_inff();
  const double by = (double)t.max_norm / (norm + (double)t.eps);
  const float scale = finite && by < 1.0 ? (float)by : 1.0f;
  if (scale == 1.0f && !t.apart) return;
  while (u >= 0) {
    if (scale != 1.0f || x.src != x.dst) {
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
        if (at + 16 <= x.bytes) *reinterpret_cast<gpiece*>(x.dst + at) = v[i];
      }
      int at;
      if (rest_of(x, &at)) {
        const float f = load_one(x, at);
        const uint32_t bits = scale != 1.0f ? __float_as_uint(f * scale) : __float_as_uint(f);
        if (x.fp32) *reinterpret_cast<gfloat*>(x.dst + at) = __uint_as_float(bits);
        else *reinterpret_cast<ghalf*>(x.dst + at) =
            scale != 1.0f ? (uint16_t)pack_bf16x2(__uint_as_float(bits), 0.0f) : (uint16_t)(bits >> 16);
      }
    }
    u -= gridDim.x;
    if (u >= 0) {
      x = clip_unit(t, s_table, u);
      load_unit(v, x.src, x.bytes);
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
