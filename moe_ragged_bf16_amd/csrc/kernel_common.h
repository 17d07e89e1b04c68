// Device helpers shared by the gfx950 kernels of this library: vector types,
// wave and block scans, the walk over work units, waits, rounding.
// Included by .hip files only, inside their translation unit.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mdg {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

typedef __attribute__((address_space(3))) void lds_void;

// ---------------------------------------------------------------------------
// block-wide scans (256 threads = 4 waves of 64)
// ---------------------------------------------------------------------------
__device__ __forceinline__ int wave_incl_sum(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    int u = __shfl_up(v, d, 64);
    if (lane >= d) v += u;
  }
  return v;
}

__device__ __forceinline__ int wave_incl_max(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    int u = __shfl_up(v, d, 64);
    if (lane >= d) v = max(v, u);
  }
  return v;
}

// Exclusive scans across the block; `scratch` holds 4 ints of LDS.
__device__ __forceinline__ int block_excl_sum(int v, int* scratch, int* total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int incl = wave_incl_sum(v);
  if (lane == 63) scratch[w] = incl;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < w; ++i) before += scratch[i];
  *total = scratch[0] + scratch[1] + scratch[2] + scratch[3];
  __syncthreads();
  return before + incl - v;
}

__device__ __forceinline__ int block_excl_max(int v, int* scratch) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int incl = wave_incl_max(v);
  int excl = __shfl_up(incl, 1, 64);
  if (lane == 0) excl = 0;
  if (lane == 63) scratch[w] = incl;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < w; ++i) before = max(before, scratch[i]);
  __syncthreads();
  return max(before, excl);
}

// ---------------------------------------------------------------------------
// reductions over the L lanes that share a row (L a power of two, 1..64)
// ---------------------------------------------------------------------------
// Steps of 1, 2, 4 and 8 lanes are DPP moves within a row of 16 lanes (quad
// permutes, then the half-row and row mirrors: once groups of 4 (8) agree, the
// mirror image of a lane holds the other group's value); steps of 16 and 32
// swap rows with the gfx950 permlane swaps.  No step touches LDS.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

template <int STEP>
__device__ __forceinline__ void partner(uint32_t v, uint32_t* a, uint32_t* b) {
  if constexpr (STEP == 1) {
    *a = v, *b = dpp<0xB1>(v);   // quad_perm [1, 0, 3, 2]
  } else if constexpr (STEP == 2) {
    *a = v, *b = dpp<0x4E>(v);   // quad_perm [2, 3, 0, 1]
  } else if constexpr (STEP == 4) {
    *a = v, *b = dpp<0x141>(v);  // row_half_mirror
  } else if constexpr (STEP == 8) {
    *a = v, *b = dpp<0x140>(v);  // row_mirror
  } else if constexpr (STEP == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    *a = r[0], *b = r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    *a = r[0], *b = r[1];
  }
}

template <int L, int STEP = 1>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  if constexpr (STEP < L) {
    uint32_t a, b;
    partner<STEP>(v, &a, &b);
    return group_max<L, STEP * 2>(max(a, b));
  } else {
    return v;
  }
}

// (The two addends of a step are the same pair on both sides, so every lane of
// the group ends with the same bits.)
template <int L, int STEP = 1>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr (STEP < L) {
    uint32_t a, b;
    partner<STEP>(__float_as_uint(v), &a, &b);
    return group_sum<L, STEP * 2>(__uint_as_float(a) + __uint_as_float(b));
  } else {
    return v;
  }
}

template <int L, int STEP = 1>
__device__ __forceinline__ float group_fmax(float v) {
  if constexpr (STEP < L) {
    uint32_t a, b;
    partner<STEP>(__float_as_uint(v), &a, &b);
    return group_fmax<L, STEP * 2>(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  } else {
    return v;
  }
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Smallest e with uprefix[e + 1] > u (the group that owns unit u).
__device__ __forceinline__ int find_group(const int* uprefix, int E, int u) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (uprefix[mid + 1] > u) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Row-major walk of a rows x cols tile grid in panels of `gm` rows, so that
// consecutive units share column panels and row panels.
__device__ __forceinline__ void panel_order(int u, int rows, int cols, int gm, int* r, int* c) {
  const int per_panel = gm * cols;
  const int panel = u / per_panel;
  const int r0 = panel * gm;
  const int h = min(gm, rows - r0);
  const int rem = u - panel * per_panel;
  *c = rem / h;
  *r = r0 + rem % h;
}

// Byte offset that the buffer range check rejects: a load returns 0 and a store
// is dropped.  Masked lanes use it, so every wave issues the same instructions.
constexpr uint32_t kOutOfRange = 0x80000000u;

// Waits until at most `kVm` of this wave's vector memory operations are
// outstanding and all its LDS reads have returned.
template <int kVm>
__device__ __forceinline__ void wait_vm_lgkm() {
  static_assert(kVm >= 0 && kVm < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((kVm & 15) | ((kVm >> 4) << 14) | (7 << 4) | (0 << 8));
}

// Workgroup barrier for the stage ring.  __syncthreads() would also make the
// compiler drain every outstanding load (its workgroup fence waits for all
// vector memory operations), which would serialise the LDS-DMA prefetch; the
// stage waits are explicit instead (wait_vm_lgkm before each barrier), and the
// empty asm statements keep the compiler from moving LDS accesses across it.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// fp32 -> bf16 with round to nearest, ties to even (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __bf16 a = static_cast<__bf16>(lo);
  __bf16 b = static_cast<__bf16>(hi);
  return (uint32_t)__builtin_bit_cast(uint16_t, a) | ((uint32_t)__builtin_bit_cast(uint16_t, b) << 16);
}

// Keeps a per-lane value opaque to the compiler at this point, so that the
// addresses derived from it are formed where they are used instead of being
// hoisted out of the unit loop (where they would only occupy registers).
__device__ __forceinline__ void opaque(int& v) { asm volatile("" : "+v"(v)); }

// This lane's index, computed where it is used (a volatile statement the
// compiler cannot hoist): the epilogue's lane-dependent addresses are then
// formed in the epilogue rather than kept in registers across the main loop.
__device__ __forceinline__ int lane_here() {
  int l;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
  return l;
}
__device__ __forceinline__ void opaque(uint32_t& v) { asm volatile("" : "+v"(v)); }

// Reads one accumulator out of its AGPR where the epilogue uses it.  Left to
// itself the compiler copies the whole 256-register tile into VGPRs when the
// main loop ends, which leaves no room for anything else and makes it spill.
// (The epilogue starts long after the last MFMA: a wait for all memory
// operations and a workgroup barrier lie between them.)
__device__ __forceinline__ float acc_read(float a) {
  float v;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
  return v;
}

}  // namespace
}  // namespace mdg
