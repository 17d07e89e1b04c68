// gfx950 (CDNA4) kernels of the norms before and after a block, fused with the block's
// gate and the scaled residual, and their gradients.
//
//   z = y, or y rstd_y w_post (rstd = 1 / sqrt(mean of squares + eps))
//   out = residual + scale gate[t] z          stored in the rows' type
//   normed = out rstd w                        of out as stored
//
// One pass over the rows: a row lies in the registers of 1 to 16 waves, 16 values a
// lane, and each sum over a row is DPP moves in a wave and one LDS exchange of the waves.
// Sums run in fp32 in one fixed order without atomics: results are bitwise
// reproducible.  The rows' bytes bound it: 16383 bf16 rows of 7168 with both norms 198 us, 4.75
// TB/s read and written; 16384 of 2048 44 us, 6.1, where the caches hold some; one token 3.5 us, a
// launch's own time.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kernel_common.h"
#include "norm.h"

namespace mdg {
namespace {

constexpr int kPieces = 2;  // of 8 values, of a row a lane holds

// 8 consecutive values in fp32, from or to memory in bf16 or fp32.
struct Eight {
  float v[8];
};

template <bool FP32>
struct Packed {
  u32x4 w[FP32 ? 2 : 1];
};

template <bool FP32>
__device__ __forceinline__ Packed<FP32> load8(const void* base, int64_t at) {
  Packed<FP32> p;
  const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(base) + at * (FP32 ? 4 : 2));
#pragma unroll
  for (int i = 0; i < (FP32 ? 2 : 1); ++i) p.w[i] = q[i];
  return p;
}
template <bool FP32>
__device__ __forceinline__ float value(const Packed<FP32>& p, int c) {
  if constexpr (FP32) return __uint_as_float(p.w[c >> 2][c & 3]);
  else return __uint_as_float((c & 1) ? p.w[0][c >> 1] & 0xffff0000u : p.w[0][c >> 1] << 16);
}
template <bool FP32>
__device__ __forceinline__ Packed<FP32> pack(const Eight& e) {
  Packed<FP32> p;
  if constexpr (FP32) {
#pragma unroll
    for (int c = 0; c < 8; ++c) p.w[c >> 2][c & 3] = __float_as_uint(e.v[c]);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) p.w[0][c] = pack_bf16x2(e.v[2 * c], e.v[2 * c + 1]);
  }
  return p;
}
template <bool FP32>
__device__ __forceinline__ void store8(void* base, int64_t at, const Packed<FP32>& p) {
  u32x4* q = reinterpret_cast<u32x4*>(static_cast<uint8_t*>(base) + at * (FP32 ? 4 : 2));
#pragma unroll
  for (int i = 0; i < (FP32 ? 2 : 1); ++i) q[i] = p.w[i];
}

// Weights of a piece in fp32.
__device__ __forceinline__ Eight weights8(const void* base, bool fp32, int at) {
  Eight e;
  if (fp32) {
    const Packed<true> p = load8<true>(base, at);
#pragma unroll
    for (int c = 0; c < 8; ++c) e.v[c] = value<true>(p, c);
  } else {
    const Packed<false> p = load8<false>(base, at);
#pragma unroll
    for (int c = 0; c < 8; ++c) e.v[c] = value<false>(p, c);
  }
  return e;
}

// Sums of N values over the waves of a row, the same bits in every lane.  `turn`
// alternates between two LDS buffers, so that one barrier a call is enough: a buffer is
// written again only past the barrier of the call in between.
template <int WAVES, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* s_red, int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = group_sum<64>(v[i]);
  if constexpr (WAVES > 1) {
    const int w = threadIdx.x >> 6;
    float* s = s_red + turn * (3 * 16);
    turn ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) s[i * WAVES + w] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float t = s[i * WAVES];
#pragma unroll
      for (int q = 1; q < WAVES; ++q) t += s[i * WAVES + q];
      v[i] = t;
    }
  }
}

template <int WAVES, bool FP32>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void norm_fwd_kernel(NormParams p) {
  constexpr int kRows = WAVES == 1 ? 4 : 1, kLanes = 64 * WAVES;
  __shared__ float s_red[2 * 3 * 16];
  const int H = p.hidden;
  const int lane = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  bool in[kPieces];
  Eight w[kPieces], wp[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c0 = (lane + i * kLanes) * 8;
    in[i] = c0 < H;
    if (in[i] && p.weight) w[i] = weights8(p.weight, p.weight_fp32, c0);
    if (in[i] && p.post_weight) wp[i] = weights8(p.post_weight, p.weight_fp32, c0);
  }
  int turn = 0;
  for (int64_t t = (int64_t)blockIdx.x * kRows + (WAVES == 1 ? threadIdx.x >> 6 : 0); t < p.tokens;
       t += (int64_t)gridDim.x * kRows) {
    const int64_t row = t * H + lane * 8;
    Packed<FP32> r[kPieces], y[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (in[i]) {
        r[i] = load8<FP32>(p.residual, row + i * kLanes * 8);
        if (p.y) y[i] = load8<FP32>(p.y, row + i * kLanes * 8);
      }
    if (p.y) {
      const float g = p.gate ? p.scale * p.gate[t] : p.scale;
      float ry = 1.0f;
      if (p.post_weight) {
        float ss[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          if (in[i])
#pragma unroll
            for (int c = 0; c < 8; ++c) ss[0] = __builtin_fmaf(value<FP32>(y[i], c), value<FP32>(y[i], c), ss[0]);
        row_sums<WAVES>(ss, s_red, turn);
        ry = 1.0f / sqrtf(ss[0] / (float)H + p.eps);
        if (lane == 0) p.post_rstd[t] = ry;
      }
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (in[i]) {
          Eight o;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            float z = value<FP32>(y[i], c);
            if (p.post_weight) z = z * ry * wp[i].v[c];
            o.v[c] = __builtin_fmaf(g, z, value<FP32>(r[i], c));
          }
          r[i] = pack<FP32>(o);
          store8<FP32>(p.out, row + i * kLanes * 8, r[i]);
        }
    }
    if (p.weight) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (in[i])
#pragma unroll
          for (int c = 0; c < 8; ++c) ss[0] = __builtin_fmaf(value<FP32>(r[i], c), value<FP32>(r[i], c), ss[0]);
      row_sums<WAVES>(ss, s_red, turn);
      const float ro = 1.0f / sqrtf(ss[0] / (float)H + p.eps);
      if (lane == 0) p.rstd[t] = ro;
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (in[i]) {
          Eight o;
#pragma unroll
          for (int c = 0; c < 8; ++c) o.v[c] = value<FP32>(r[i], c) * ro * w[i].v[c];
          store8<FP32>(p.normed, row + i * kLanes * 8, pack<FP32>(o));
        }
    }
  }
}

// With x = out rstd, g = dnormed w, z as above and h = hidden:
//   do = dout + rstd (g - x mean(g x)),  dresidual = do,  dz = scale gate do
//   dgate = scale A, A = sum do z = sum (dout + rstd g) z - rstd mean(g x) sum x z
//   dy = rstd_y (dz w_post - y rstd_y scale gate A / h), or dz without the norm of y
//   dweight = sum_t dnormed x,  dpost_weight = sum_t dz y rstd_y
// so one exchange of three sums a row is enough.  The weights' gradients add up in the
// lanes' registers over a block's rows; norm_finish_kernel adds the blocks.
// Memory bounds it: 16383 bf16 rows of 7168 with everything (six rows read or written for
// each) 287 us, 4.9 TB/s; 16384 fp32 rows of 2048 151 us, 5.3; one row of 16 waves at a time and
// their barrier hold 4096 fp32 rows of 16384 at 4.1.  bf16 rows: at most 128 registers, so that 16
// waves fit a CU (327 us with one block of 8).
// kLean: fp32 rows of 16 waves, which have 128 registers a lane: rows of dout and y and
// the weights are read again, from the caches, where they are used (held as for narrower
// rows 72 registers spilled: 4096 rows of 16384 835 us, here 385).
template <int WAVES, bool FP32>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES, FP32 || WAVES == 1 ? 1 : 4) void norm_bwd_kernel(NormBwdParams p) {
  constexpr int kRows = WAVES == 1 ? 4 : 1, kLanes = 64 * WAVES;
  __shared__ float s_red[2 * 3 * 16];
  __shared__ float s_part[WAVES == 1 ? 4 * 1024 : 1];
  const int H = p.hidden;
  const int lane = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  const bool pre = p.weight != nullptr && p.dnormed != nullptr, post = p.post_weight != nullptr;
  const bool with_z = post || p.gate != nullptr;
  constexpr bool kLean = FP32 && WAVES == 16;
  bool in[kPieces];
  Eight w[kPieces], wp[kPieces], aw[kPieces], ap[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c0 = (lane + i * kLanes) * 8;
    in[i] = c0 < H;
    if (!kLean && in[i] && pre) w[i] = weights8(p.weight, p.weight_fp32, c0);
    if (!kLean && in[i] && post) wp[i] = weights8(p.post_weight, p.weight_fp32, c0);
#pragma unroll
    for (int c = 0; c < 8; ++c) aw[i].v[c] = ap[i].v[c] = 0.0f;
  }
  // A piece's weights: held, or read again (through an address that the compiler cannot
  // know, or the loads would move out of the loop over rows).
  const auto weights = [&](const Eight& held, const void* base, bool some,
                           int i) -> std::conditional_t<kLean, Eight, const Eight&> {
    if constexpr (kLean) {
      int at = (lane + i * kLanes) * 8;
      opaque(at);
      return some ? weights8(base, p.weight_fp32, at) : Eight{};
    } else {
      return held;
    }
  };
  const float inv_h = 1.0f / (float)H;
  int turn = 0;
  for (int64_t t = (int64_t)blockIdx.x * kRows + (WAVES == 1 ? threadIdx.x >> 6 : 0); t < p.tokens;
       t += (int64_t)gridDim.x * kRows) {
    const int64_t row = t * H + lane * 8;
    Packed<FP32> d[kPieces], n[kPieces], o[kPieces], y[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (in[i]) {
        const int64_t at = row + i * kLanes * 8;
        if (!kLean && p.dout) d[i] = load8<FP32>(p.dout, at);
        if (pre) n[i] = load8<FP32>(p.dnormed, at), o[i] = load8<FP32>(p.out, at);
        if (!kLean && with_z) y[i] = load8<FP32>(p.y, at);
      }
    const auto again = [&](int i) {  // kLean: dout and y of a piece
      if constexpr (kLean) {
        __builtin_amdgcn_sched_barrier(0);
        int at = i * kLanes * 8;
        opaque(at);
        if (p.dout) d[i] = load8<FP32>(p.dout, row + at);
        if (with_z) y[i] = load8<FP32>(p.y, row + at);
      }
    };
    const float ro = pre ? p.rstd[t] : 0.0f, ry = post ? p.post_rstd[t] : 1.0f;
    const float gate = p.gate ? p.scale * p.gate[t] : p.scale;
    float s[3] = {0.0f, 0.0f, 0.0f};
    if (pre || with_z) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (in[i]) {
          if (with_z) again(i);
          const Eight& wi = weights(w[i], p.weight, pre, i);
          const Eight& wpi = weights(wp[i], p.post_weight, post, i);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float x = pre ? value<FP32>(o[i], c) * ro : 0.0f;
            const float g = pre ? value<FP32>(n[i], c) * wi.v[c] : 0.0f;
            s[0] = __builtin_fmaf(g, x, s[0]);
            if (with_z) {
              float z = value<FP32>(y[i], c) * ry;
              if (post) z *= wpi.v[c];
              const float dv = p.dout ? value<FP32>(d[i], c) : 0.0f;
              s[1] = __builtin_fmaf(__builtin_fmaf(ro, g, dv), z, s[1]);
              s[2] = __builtin_fmaf(x, z, s[2]);
            }
          }
        }
      row_sums<WAVES>(s, s_red, turn);
    }
    const float m = s[0] * inv_h;
    const float a = __builtin_fmaf(-ro * m, s[2], s[1]);
    const float back = gate * a * inv_h;
    if (p.dgate && lane == 0) p.dgate[t] = p.scale * a;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (in[i]) {
        const int64_t at = row + i * kLanes * 8;
        again(i);
        const Eight& wi = weights(w[i], p.weight, pre, i);
        const Eight& wpi = weights(wp[i], p.post_weight, post, i);
        Eight dr, dv;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float e = p.dout ? value<FP32>(d[i], c) : 0.0f;
          if (pre) {
            const float x = value<FP32>(o[i], c) * ro, nv = value<FP32>(n[i], c);
            e = __builtin_fmaf(ro, __builtin_fmaf(-x, m, nv * wi.v[c]), e);
            aw[i].v[c] = __builtin_fmaf(nv, x, aw[i].v[c]);
          }
          dr.v[c] = e;
          const float dz = gate * e;
          dv.v[c] = dz;
          if (post) {
            const float yh = value<FP32>(y[i], c) * ry;
            dv.v[c] = ry * __builtin_fmaf(-yh, back, dz * wpi.v[c]);
            ap[i].v[c] = __builtin_fmaf(dz, yh, ap[i].v[c]);
          }
        }
        if (p.dresidual) store8<FP32>(p.dresidual, at, pack<FP32>(dr));
        if (p.dy) store8<FP32>(p.dy, at, pack<FP32>(dv));
      }
  }
  if (p.part == nullptr) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if ((which ? p.dpost_weight : p.dweight) == nullptr) continue;
    float* part = p.part + ((int64_t)blockIdx.x * 2 + which) * H;
    if constexpr (WAVES == 1) {  // the block's four rows of sums, in wave order
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (in[i])
#pragma unroll
          for (int c = 0; c < 8; ++c)
            s_part[(threadIdx.x >> 6) * 1024 + (lane + i * 64) * 8 + c] = which ? ap[i].v[c] : aw[i].v[c];
      __syncthreads();
      for (int c = threadIdx.x; c < H; c += 256)
        part[c] = ((s_part[c] + s_part[1024 + c]) + s_part[2 * 1024 + c]) + s_part[3 * 1024 + c];
    } else {
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (in[i]) store8<true>(part, (lane + i * kLanes) * 8, pack<true>(which ? ap[i] : aw[i]));
    }
  }
}

// Adds the blocks' sums of a weight (blockIdx.y) over 32 columns (whole cache lines): row
// group g of 32 adds blocks g, g + 32, ..., then the two groups of a wave by a shuffle and
// the 16 waves in order.
constexpr int kFinishCols = 32, kFinishRows = 1024 / kFinishCols;

__global__ __launch_bounds__(1024) void norm_finish_kernel(NormBwdParams p) {
  __shared__ float s_sum[16][kFinishCols];
  void* out = blockIdx.y ? p.dpost_weight : p.dweight;
  if (out == nullptr) return;
  const int col = threadIdx.x % kFinishCols, g = threadIdx.x / kFinishCols, c = blockIdx.x * kFinishCols + col;
  float s = 0.0f;
  if (c < p.hidden)
#pragma unroll 8
    for (int b = g; b < p.blocks; b += kFinishRows) s += p.part[((int64_t)b * 2 + blockIdx.y) * p.hidden + c];
  for (int d = kFinishCols; d < 64; d <<= 1) s += __shfl_xor(s, d, 64);
  if ((threadIdx.x & 63) < kFinishCols) s_sum[threadIdx.x >> 6][col] = s;
  __syncthreads();
  if (threadIdx.x >= kFinishCols || c >= p.hidden) return;
  s = s_sum[0][col];
#pragma unroll
  for (int i = 1; i < 16; ++i) s += s_sum[i][col];
  if (p.weight_fp32) static_cast<float*>(out)[c] = s;
  else static_cast<uint16_t*>(out)[c] = (uint16_t)pack_bf16x2(s, 0.0f);
}

template <bool FP32>
void norm_fwd(const NormParams& p, int blocks, hipStream_t s) {
  const int waves = norm_waves(p.hidden);
  const dim3 g(blocks), b(waves == 1 ? 256 : 64 * waves);
  switch (waves) {
    case 1: hipLaunchKernelGGL((norm_fwd_kernel<1, FP32>), g, b, 0, s, p); break;
    case 2: hipLaunchKernelGGL((norm_fwd_kernel<2, FP32>), g, b, 0, s, p); break;
    case 4: hipLaunchKernelGGL((norm_fwd_kernel<4, FP32>), g, b, 0, s, p); break;
    case 8: hipLaunchKernelGGL((norm_fwd_kernel<8, FP32>), g, b, 0, s, p); break;
    default: hipLaunchKernelGGL((norm_fwd_kernel<16, FP32>), g, b, 0, s, p); break;
  }
}

template <bool FP32>
void norm_bwd(const NormBwdParams& p, hipStream_t s) {
  const int waves = norm_waves(p.hidden);
  const dim3 g(p.blocks), b(waves == 1 ? 256 : 64 * waves);
  switch (waves) {
    case 1: hipLaunchKernelGGL((norm_bwd_kernel<1, FP32>), g, b, 0, s, p); break;
    case 2: hipLaunchKernelGGL((norm_bwd_kernel<2, FP32>), g, b, 0, s, p); break;
    case 4: hipLaunchKernelGGL((norm_bwd_kernel<4, FP32>), g, b, 0, s, p); break;
    case 8: hipLaunchKernelGGL((norm_bwd_kernel<8, FP32>), g, b, 0, s, p); break;
    default: hipLaunchKernelGGL((norm_bwd_kernel<16, FP32>), g, b, 0, s, p); break;
  }
}

}  // namespace

hipError_t launch_norm_fwd(const NormParams& p, int blocks, hipStream_t s) {
  if (p.fp32) norm_fwd<true>(p, blocks, s);
  else norm_fwd<false>(p, blocks, s);
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormBwdParams& p, hipStream_t s) {
  if (p.blocks > 0) {
    if (p.fp32) norm_bwd<true>(p, s);
    else norm_bwd<false>(p, s);
  }
  if (p.dweight || p.dpost_weight)
    hipLaunchKernelGGL(norm_finish_kernel, dim3((p.hidden + kFinishCols - 1) / kFinishCols, 2), dim3(1024), 0, s, p);
  return hipGetLastError();
}

}  // namespace mdg
