// gfx950 (CDNA4) kernels around the expert products of a Mixture-of-Experts
// layer: routing with counts and balance loss, the plan that sorts slots by
// expert, rows dispatched by the plan and combined back, and the gradients.
//
// All sums run in fp32 (integers where they count; the loss's last sum in 64 bits) in
// one fixed order and no floating-point atomics are used, so every output is bitwise
// reproducible.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernel_common.h"
#include "moe.h"

namespace mdg {
namespace {

__device__ __forceinline__ uint16_t narrow(float f) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}

constexpr float kNegInf = -__builtin_inff();

// Sum over a wave's groups of L lanes, lane by lane of a group: rotations within
// rows of 16 lanes, then the permlane swaps.
template <int L, int STEP = 8>
__device__ __forceinline__ float sum_over_groups(float v) {
  if constexpr (STEP >= L && STEP > 0) {
    return sum_over_groups<L, STEP / 2>(v + __uint_as_float(dpp<0x120 + STEP>(__float_as_uint(v))));  // row_ror
  } else {
    uint32_t a, b;
    if constexpr (L <= 16) {
      partner<16>(__float_as_uint(v), &a, &b);
      v = __uint_as_float(a) + __uint_as_float(b);
    }
    if constexpr (L <= 32) {
      partner<32>(__float_as_uint(v), &a, &b);
      v = __uint_as_float(a) + __uint_as_float(b);
    }
    return v;
  }
}

// V consecutive logits of a row from column c0, in their bits (bf16: two to a word).
// With `vec` (rows start on 16 bytes and experts are a multiple of V) in 16-byte
// pieces; else element by element, and the gradient's stores likewise.  65536 rows, top-4,
// forward with its second launch / gradient in us: 128 experts fp32 22.3 / 15.4, 127
// 27.6 / 43.8, 100 24.9 / 34.6; bf16 20.6 / 13.1, 24.6 / 31.1, 23.9 / 26.3; 64 experts
// fp32 14.9 / 9.4, 60 17.0 / 18.6; bf16 14.4 / 8.0, 16.2 / 11.5.
template <int V, bool FP32>
struct LogitBits {
  static constexpr int kWords = FP32 ? V : V / 2;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const void* base, int64_t row, int c0, int experts, bool vec) {
    const int64_t at = row * experts + c0;
    if (vec) {  // a lane's V columns are all there or all not
      if (c0 < experts) {
        const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(base) + at * (FP32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
          const u32x4 x = q[i];
#pragma unroll
          for (int c = 0; c < 4; ++c) w[4 * i + c] = x[c];
        }
      } else {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = FP32 ? 0xff800000u : 0xff80ff80u;
      }
    } else {  // columns at or past `experts` read -inf
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        if constexpr (FP32) {
          w[i] = c0 + i < experts ? static_cast<const uint32_t*>(base)[at + i] : 0xff800000u;
        } else {
          const uint16_t* q = static_cast<const uint16_t*>(base) + at + 2 * i;
          const uint32_t lo = c0 + 2 * i < experts ? q[0] : 0xff80u, hi = c0 + 2 * i + 1 < experts ? q[1] : 0xff80u;
          w[i] = lo | (hi << 16);
        }
      }
    }
  }
  __device__ __forceinline__ float value(int v) const {
    if constexpr (FP32) return __uint_as_float(w[v]);
    else return __uint_as_float((v & 1) ? w[v / 2] & 0xffff0000u : w[v / 2] << 16);
  }
};

// ---------------------------------------------------------------------------
// routing
// ---------------------------------------------------------------------------
// An order-preserving integer of a logit: -0 and +0 are equal, NaN is above
// everything.  -inf, an expert that cannot be chosen, is kKeyNone or (bf16) a little
// below; a chosen expert's key becomes its slot's number + 1, far below.
constexpr uint32_t kKeyNone = 0x007fffffu;

__device__ __forceinline__ uint32_t key_of(float f) {
  if (f != f) return 0xffffffffu;
  const uint32_t u = __float_as_uint(f + 0.0f);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

// The key of a column of a row.  A bf16 key leaves the lower 16 bits free for the
// expert's complement, so keys differ and the largest is the choice, the lowest
// expert among equal logits.
template <bool FP32>
__device__ __forceinline__ uint32_t choice_key(float f, int column) {
  const uint32_t k = key_of(f);
  return FP32 ? k : (k & 0xffff0000u) | (0xffffu - (uint32_t)column);
}
// A key's logit.
template <bool FP32>
__device__ __forceinline__ float choice_value(uint32_t key) {
  if constexpr (FP32) return value_of(key);
  else return (key & 0xffff0000u) == 0xffff0000u ? __uint_as_float(0x7fc00000u)
                                                 : value_of((key & 0x80000000u) ? key & 0xffff0000u : key | 0xffffu);
}

// One round of the top-k over the V keys a lane of the group: the largest key becomes
// slot + 1.  fp32 keys may be equal: where a wave has more hits than groups, the
// lowest column of each group's is taken.  Returns the key (<= kKeyNone: the group has
// nothing left, and no key was changed).
template <int L, int V, bool FP32>
__device__ __forceinline__ uint32_t choose(uint32_t (&key)[V], int c0, uint32_t slot) {
  uint32_t best = key[0];
#pragma unroll
  for (int v = 1; v < V; ++v) best = max(best, key[v]);
  const uint32_t top = group_max<L>(best);
  const bool some = top > kKeyNone;
  const uint32_t want = some ? top : 0xffffffffu;  // (no key of a group without a choice equals it)
  if constexpr (FP32) {
    int hits = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) hits += __popcll(__ballot(key[v] == want));
    if (hits * L != __popcll(__ballot(some))) {
      uint32_t col = 0xffffu;
#pragma unroll
      for (int v = V - 1; v >= 0; --v)
        if (key[v] == want) col = c0 + v;
      col = 0xffffu - group_max<L>(0xffffu - col);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (key[v] == want && c0 + v == (int)col) key[v] = slot + 1;
      return top;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) key[v] = key[v] == want ? slot + 1 : key[v];
  return top;
}

// e^x for x <= 0, to about 1.5 units in the last place: 2^t with t = x log2(e) in two
// parts (t rounded, and what rounding left, which enters by its first-order term).
// Results below the smallest normal number (x < -87.3) are 0, so a chosen expert that
// unlikely gets weight 0; the clamp keeps -inf - (-inf) out (and loses NaN).  The gradient
// takes the library's exponential, so its softmax may differ from the forward's in
// the last place.
__device__ __forceinline__ float exp_nonpositive(float x) {
  constexpr float kLog2e = 1.44269502162933349609375f;    // log2(e) rounded to fp32
  constexpr float kLog2eLow = 1.925963033500011079e-08f;  // log2(e) - kLog2e
  constexpr float kLn2 = 0.693147180559945309f;
  x = fmaxf(x, -200.0f);
  const float t = x * kLog2e;
  const float rest = __builtin_fmaf(x, kLog2eLow, __builtin_fmaf(x, kLog2e, -t));
  const float r = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(r, rest * kLn2, r);
}

// The balance loss from the sums of one expert: a = E c / (k Tr^2) is the
// derivative of the loss by the expert's probability sum, a * sum its share.
__device__ __forceinline__ double balance_of(const RouteParams& p, int count, int routed) {
  return routed > 0 ? (double)p.experts * count / ((double)p.top_k * routed * routed) : 0.0;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Slots j = i * L + (lane in group) that a lane keeps of its row's top-k.
template <int L, int V>
constexpr int own_slots() {
  constexpr int most = kRouteMaxTopK < L * V ? kRouteMaxTopK : L * V;
  return most > L ? most / L : 1;
}

// L lanes hold a row, V consecutive logits each.  The top-k is k rounds of choose(),
// in registers and DPP moves; the first round's value is the softmax maximum; lanes
// that hold a chosen expert write its slot.  Each lane adds the probabilities of its
// columns over all rows of its block in registers; the next row's logits load while
// a row is worked on.  Latency bounds it, one row in flight per lane group and 16 waves to
// a CU: 65536 rows of 128 fp32 logits, top-4, take 17 to 20 us, 1.8 TB/s (12.3 us with
// one round in place of four); the library exponential and passing each round's choice
// to the slot's lane made it 1.4 us longer.
template <int L, int V, bool FP32>
__global__ __launch_bounds__(kRouteThreads) void route_fwd_kernel(RouteParams p) {
  extern __shared__ uint8_t smem[];
  const int E = p.experts, k = p.top_k;
  const int waves = blockDim.x >> 6;
  float* s_sum = reinterpret_cast<float*>(smem);             // [waves][E]
  int* s_cnt = reinterpret_cast<int*>(s_sum + waves * E);    // [E]
  int* s_routed = s_cnt + E;                                 // [1]
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int lig = lane & (L - 1), grp = tid / L, c0 = lig * V;
  for (int e = tid; e < E; e += blockDim.x) s_cnt[e] = 0;
  if (tid == 0) *s_routed = 0;

  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
  int routed = 0;
  const int64_t row_end = min(p.tokens, (int64_t)(blockIdx.x + 1) * p.rows_per_block);
  int64_t r = (int64_t)blockIdx.x * p.rows_per_block + grp;
  LogitBits<V, FP32> bits;
  bool keep = true;
  if (r < row_end) {
    bits.load(p.logits, r, c0, E, p.vec != 0);
    keep = p.mask == nullptr || p.mask[r] != 0;
  }
  __syncthreads();
  while (r < row_end) {
    float l[V];
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {  // (columns past the last are -inf)
      l[v] = keep ? bits.value(v) : kNegInf;
      key[v] = choice_key<FP32>(l[v], c0 + v);
    }
    const int64_t row = r;
    r += blockDim.x / L;
    if (r < row_end) {
      bits.load(p.logits, r, c0, E, p.vec != 0);
      keep = p.mask == nullptr || p.mask[r] != 0;
    }
    uint32_t first = 0;
    int found = 0;
    for (int j = 0; j < k; ++j) {
      const uint32_t top = choose<L, V, FP32>(key, c0, (uint32_t)j);
      if (j == 0) first = top;
      found += top > kKeyNone;
    }
    const bool live = first > kKeyNone;
    const float big = live ? choice_value<FP32>(first) : 0.0f;
    const float poison = big < __builtin_inff() ? 0.0f : __uint_as_float(0x7fc00000u);  // NaN for a row with NaN or +inf
    float ex[V], total = poison, chosen = poison;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      ex[v] = exp_nonpositive(l[v] - big);
      total += ex[v];
      chosen += key[v] - 1u < (uint32_t)kRouteMaxTopK ? ex[v] : 0.0f;
    }
    total = group_sum<L>(total);
    if (p.normalize) chosen = group_sum<L>(chosen);
    const float scale = 1.0f / (p.normalize ? chosen : total);
    const int64_t slots = row * k;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t j = key[v] - 1u;
      if (j < (uint32_t)kRouteMaxTopK) {
        p.weight[slots + j] = ex[v] * scale;
        p.idx[slots + j] = c0 + v;
        atomicAdd(&s_cnt[c0 + v], 1);
      }
    }
    for (int j = found + lig; j < k; j += L) {  // slots no expert is left for
      p.weight[slots + j] = 0.0f;
      p.idx[slots + j] = -1;
    }
    if (live) {
      const float inv = 1.0f / total;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = __builtin_fmaf(ex[v], inv, acc[v]);
      if (lig == 0) ++routed;
    }
  }

  // the block's sums: over the wave's groups, then over the waves in order
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float s = sum_over_groups<L>(acc[v]);
    if (lane < L && lane * V + v < E) s_sum[w * E + lane * V + v] = s;
  }
  if (routed) atomicAdd(s_routed, routed);
  __syncthreads();
  if (gridDim.x > 1) {
    for (int e = tid; e < E; e += blockDim.x) {
      float s = s_sum[e];
      for (int i = 1; i < waves; ++i) s += s_sum[i * E + e];
      p.part_sum[(int64_t)blockIdx.x * E + e] = s;
      p.part_cnt[(int64_t)blockIdx.x * E + e] = s_cnt[e];
    }
    if (tid == 0) p.part_routed[blockIdx.x] = *s_routed;
    if (tid == 0 && blockIdx.x == 0) *p.part_done = 0;  // for the finishing kernel, next on the stream
    return;
  }
  // one block: finish here
  const int tr = *s_routed;
  double share = 0.0;
  for (int e = tid; e < E; e += blockDim.x) {
    float s = s_sum[e];
    for (int i = 1; i < waves; ++i) s += s_sum[i * E + e];
    const double a = balance_of(p, s_cnt[e], tr);
    p.counts[e] = s_cnt[e];
    p.balance[e] = (float)a;
    share += a * s;
  }
  share = wave_sum(share);
  __syncthreads();
  double* s_share = reinterpret_cast<double*>(smem);
  if (lane == 0) s_share[w] = share;
  __syncthreads();
  if (tid == 0) {
    double sum = 0.0;
    for (int i = 0; i < waves; ++i) sum += s_share[i];
    *p.loss = (float)sum;
  }
}

// Adds the route blocks' partial sums and writes counts, balance and loss.  A
// workgroup takes kFinishCols experts, its threads as columns x row groups, so
// that all of the table's loads are in flight at once (one workgroup walking
// [256 blocks, 256 experts] alone took 60 us, these 4.4 us).  The order of an expert's
// sum is fixed: row group g of 64 adds blocks g, g + 64, ..., a wave's 4 groups are added by
// shuffles, then the 16 waves.  The last workgroup to finish adds the workgroups'
// shares of the loss.
constexpr int kFinishCols = 16;
constexpr int kFinishRows = kRouteThreads / kFinishCols;  // row groups
static_assert(kRouteMaxExperts <= 64 * kFinishCols, "a lane for every workgroup's share");

__global__ __launch_bounds__(kRouteThreads) void route_finish_kernel(RouteParams p) {
  __shared__ int s_tr[kRouteThreads / 64];
  __shared__ float s_sum[kRouteThreads / 64][kFinishCols];
  __shared__ int s_cnt[kRouteThreads / 64][kFinishCols];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int E = p.experts;
  const int col = tid % kFinishCols, rg = tid / kFinishCols, e = blockIdx.x * kFinishCols + col;
  int tr = tid < p.blocks ? p.part_routed[tid] : 0;
  float s = 0.0f;
  int c = 0;
  if (e < E)
    for (int b = rg; b < p.blocks; b += kFinishRows) {
      s += p.part_sum[(int64_t)b * E + e];
      c += p.part_cnt[(int64_t)b * E + e];
    }
  // a wave's 4 row groups, then the 16 waves' sums, in this order on every run
  for (int d = kFinishCols; d < 64; d <<= 1) {
    s += __shfl_xor(s, d, 64);
    c += __shfl_xor(c, d, 64);
  }
  if (lane < kFinishCols) {
    s_sum[w][lane] = s;
    s_cnt[w][lane] = c;
  }
  tr = wave_incl_sum(tr);
  if (lane == 63) s_tr[w] = tr;
  __syncthreads();
  if (w != 0) return;
  constexpr int kWaves = kRouteThreads / 64, kEach = kWaves * kFinishCols / 64;
  s = 0.0f;
  c = tr = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    s += s_sum[rg * kEach + i][col];
    c += s_cnt[rg * kEach + i][col];
  }
  for (int d = kFinishCols; d < 64; d <<= 1) {
    s += __shfl_xor(s, d, 64);
    c += __shfl_xor(c, d, 64);
  }
#pragma unroll
  for (int i = 0; i < kWaves; ++i) tr += s_tr[i];
  double share = 0.0;
  if (lane < kFinishCols && e < E) {
    const double a = balance_of(p, c, tr);
    p.counts[e] = c;
    p.balance[e] = (float)a;
    share = a * s;
  }
  share = wave_sum(share);
  int done = 0;
  if (lane == 0) {
    __hip_atomic_store(&p.part_share[blockIdx.x], share, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    done = __hip_atomic_fetch_add(p.part_done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (__shfl(done, 0, 64) != (int)gridDim.x - 1) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  share = lane < (int)gridDim.x
              ? __hip_atomic_load(&p.part_share[lane], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
              : 0.0;
  share = wave_sum(share);
  if (lane == 0) *p.loss = (float)share;
}

// d logits of a row, with p its softmax, w its weights, a = balance, g = dloss:
//   D = g sum_e p a (+ sum_j w dw without normalisation)
//   dl_e = p_e (g a_e - D) + [e chosen in slot j] (w_j (dw_j - sum_j w dw) with
//   normalisation, else w_j dw_j).
// The softmax is computed anew from the logits (cheaper than reading it back).
// Memory bounds it: 65536 rows of 128 fp32 logits take 15.6 us, 4.3 TB/s (a large
// copy: 4.9).
template <int L, int V, bool FP32>
__global__ __launch_bounds__(256) void route_bwd_kernel(RouteBwdParams p) {
  constexpr int kOwn = own_slots<L, V>();
  const int E = p.experts, k = p.top_k;
  const int lane = threadIdx.x & 63, lig = lane & (L - 1), c0 = lig * V;
  const int64_t r = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  if (r >= p.tokens) return;
  LogitBits<V, FP32> bits;
  bits.load(p.logits, r, c0, E, p.vec != 0);
  // this lane's slots of the row
  int own_e[kOwn];
  float own_w[kOwn], own_d[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int j = i * L + lig;
    own_e[i] = j < k ? p.idx[r * k + j] : -1;
    own_w[i] = j < k ? p.weight[r * k + j] : 0.0f;
    own_d[i] = j < k && p.dweight ? p.dweight[r * k + j] : 0.0f;
  }
  const float g = p.dloss ? *p.dloss : 0.0f;
  float a[V];
  if (p.vec && c0 < E) {
#pragma unroll
    for (int v = 0; v < V; ++v) a[v] = p.balance[c0 + v];
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) a[v] = c0 + v < E ? p.balance[c0 + v] : 0.0f;
  }
  float inner = 0.0f;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    own_d[i] = own_e[i] >= 0 ? own_d[i] : 0.0f;
    inner += own_w[i] * own_d[i];
  }
  inner = group_sum<L>(inner);
  const bool live = __shfl(own_e[0], lane & ~(L - 1), 64) >= 0;
  float l[V], dl[V], big = kNegInf, total = 0.0f, pa = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    l[v] = bits.value(v);
    big = fmaxf(big, l[v]);
  }
  big = group_fmax<L>(big);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    a[v] *= g;
    l[v] = c0 + v < E ? expf(l[v] - big) : 0.0f;
    total += l[v];
    pa += l[v] * a[v];
  }
  total = group_sum<L>(total);
  pa = group_sum<L>(pa);
  const float inv = 1.0f / total;
  const float d = pa * inv + (p.normalize ? 0.0f : inner);
#pragma unroll
  for (int v = 0; v < V; ++v) dl[v] = l[v] * inv * (a[v] - d);
  if (p.dweight) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const float own_add = own_w[i] * (own_d[i] - (p.normalize ? inner : 0.0f));
      for (int jl = 0; jl < L && i * L + jl < k; ++jl) {  // slot by slot to the lane that holds its expert
        const int from = (lane & ~(L - 1)) + jl;
        const float add = L == 1 ? own_add : __shfl(own_add, from, 64);
        const int at = (L == 1 ? own_e[i] : __shfl(own_e[i], from, 64)) - c0;
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (at == v) dl[v] += add;
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) dl[v] = live ? dl[v] : 0.0f;
  const int64_t at = r * E + c0;
  if (p.vec) {
    if (c0 >= E) return;
    if constexpr (FP32) {
      f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(p.dlogits) + at);
#pragma unroll
      for (int i = 0; i < V / 4; ++i) q[i] = f32x4{dl[4 * i], dl[4 * i + 1], dl[4 * i + 2], dl[4 * i + 3]};
    } else {
      u32x4* q = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.dlogits) + at);
#pragma unroll
      for (int i = 0; i < V / 8; ++i) {
        u32x4 x;
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = pack_bf16x2(dl[8 * i + 2 * c], dl[8 * i + 2 * c + 1]);
        q[i] = x;
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (c0 + v < E) {
        if constexpr (FP32) static_cast<float*>(p.dlogits)[at + v] = dl[v];
        else static_cast<uint16_t*>(p.dlogits)[at + v] = narrow(dl[v]);
      }
  }
}

// ---------------------------------------------------------------------------
// the plan: a stable counting sort of the slots by expert
// ---------------------------------------------------------------------------
// Slots (t, j) in order t * top_k + j.  A block sorts p.chunk consecutive
// slots, each wave a run of consecutive ones: a slot's row is offs of its
// expert + the expert's slots in earlier blocks + in earlier waves + earlier in
// its wave's run (lanes that hold the same expert, found with ballots over the
// bits of the expert number).  Latency bounds it (a chain of loads, LDS sums and
// barriers): 32768 slots of 64 experts take 4 + 6.4 us, 6 slots 2.9 us in one launch.
__device__ __forceinline__ int slot_expert(const PlanParams& p, int64_t s, int64_t end) {
  if (s >= end) return -1;
  const int e = p.idx[s];
  return (unsigned)e < (unsigned)p.experts ? e : -1;
}

// Orders the LDS accesses of one wave's lanes (the hardware runs them in order;
// this keeps the compiler from moving them).
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Adds the experts of slots [begin, end), taken by one wave, to hist.
__device__ __forceinline__ void plan_count(const PlanParams& p, int* hist, int64_t begin, int64_t end) {
  const int lane = threadIdx.x & 63;
  for (int64_t s = begin; s < end; s += 64) {
    const int e = slot_expert(p, s + lane, end);
    if (e >= 0) atomicAdd(&hist[e], 1);
  }
}

__global__ __launch_bounds__(kPlanThreads) void plan_count_kernel(PlanParams p) {
  extern __shared__ int s_plan[];  // [E]
  const int tid = threadIdx.x;
  for (int e = tid; e < p.experts; e += kPlanThreads) s_plan[e] = 0;
  __syncthreads();
  const int64_t begin = (int64_t)blockIdx.x * p.chunk, end = min(p.slots, begin + p.chunk);
  for (int64_t s = begin + tid; s < end; s += kPlanThreads) {
    const int e = slot_expert(p, s, end);
    if (e >= 0) atomicAdd(&s_plan[e], 1);
  }
  __syncthreads();
  for (int e = tid; e < p.experts; e += kPlanThreads) p.hist[(int64_t)blockIdx.x * p.experts + e] = s_plan[e];
}

__global__ __launch_bounds__(kPlanThreads) void plan_rank_kernel(PlanParams p) {
  extern __shared__ int s_plan[];  // [runs][E] next row of each wave's slots by expert
  __shared__ int s_scan[kPlanThreads / 64];
  const int runs = p.runs;  // the first `runs` waves take slots
  const int E = p.experts, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  for (int i = tid; i < runs * E; i += kPlanThreads) s_plan[i] = 0;
  __syncthreads();
  const int64_t begin = (int64_t)blockIdx.x * p.chunk, end = min(p.slots, begin + p.chunk);
  const int64_t run = ((end - begin + runs - 1) / runs + 63) / 64 * 64;
  const int64_t wb = min(end, begin + w * run), we = min(end, wb + run);
  // thread e (E <= kPlanThreads): the expert's slots in all blocks and in the blocks before
  int all = 0, before = 0;
  if (tid < E && gridDim.x > 1) {
#pragma unroll 8
    for (int b = 0; b < p.blocks; ++b) {
      const int c = p.hist[(int64_t)b * E + tid];
      all += c;
      if (b < (int)blockIdx.x) before += c;
    }
  }
  if (w < runs) plan_count(p, s_plan + w * E, wb, we);
  __syncthreads();
  if (tid < E && gridDim.x == 1)
    for (int i = 0; i < runs; ++i) all += s_plan[i * E + tid];
  const int incl = wave_incl_sum(all);
  if (lane == 63) s_scan[w] = incl;
  __syncthreads();
  int start = incl - all;
  for (int i = 0; i < w; ++i) start += s_scan[i];
  if (tid < E) {
    if (blockIdx.x == 0) p.offs[tid] = start + all;
    int at = start + before;
    for (int i = 0; i < runs; ++i) {
      const int c = s_plan[i * E + tid];
      s_plan[i * E + tid] = at;
      at += c;
    }
  }
  __syncthreads();
  if (w >= runs) return;
  int* next = s_plan + w * E;
  for (int64_t s = wb; s < we; s += 64) {
    const int e = slot_expert(p, s + lane, we);
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; (E - 1) >> b; ++b) {
      const uint64_t one = __ballot((e >> b) & 1);
      same &= ((e >> b) & 1) ? one : ~one;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    const int base = e >= 0 ? next[e] : 0;
    if (s + lane < we) p.dest[s + lane] = e >= 0 ? base + rank : -1;
    wave_lds_order();
    if (e >= 0 && rank == 0) next[e] = base + __popcll(same);
    wave_lds_order();
  }
}

// ---------------------------------------------------------------------------
// rows by the plan
// ---------------------------------------------------------------------------
// A team of TEAM threads (64 or 256) takes one token and walks its row in
// 16-byte pieces.  Bytes bound all of these: each row is read once and written
// once, wherever the plan puts it.  4095 tokens x 8 rows of 7168 bf16 (0.53 GB moved a
// pass, 1 GB by the gradient): dispatch 93 us (5.7 TB/s, mostly writes), the weighted
// sum 123 us (4.3 TB/s, mostly reads: one 16-byte load in flight per thread, slot after
// slot; kernels here that load ahead read at 4.9), the gradient 179 us (5.6 TB/s).  A
// wave instead of four for short rows (TEAM 64).

// Rows from offs[E-1] on belong to no slot: zeros, shared out over the blocks.
__device__ __forceinline__ void zero_rest(const RowsParams& p) {
  const int64_t first = min(max((int64_t)p.offs[p.experts - 1], (int64_t)0), p.slots);
  u32x4* out = static_cast<u32x4*>(p.out);
  const u32x4 z = {0u, 0u, 0u, 0u};
  for (int64_t r = first + blockIdx.x; r < p.slots; r += gridDim.x)
    for (int c = threadIdx.x; c < p.pieces; c += blockDim.x) out[r * p.pieces + c] = z;
}

template <int TEAM>
__device__ __forceinline__ int64_t team_token() {
  const int t = (int)blockIdx.x * (256 / TEAM) + (TEAM == 256 ? 0 : uniform(threadIdx.x >> 6));
  return t;
}

// The row slot (t, j) has, or -1 (also for a dest that lies outside the rows).
__device__ __forceinline__ int slot_row(const RowsParams& p, int64_t t, int j) {
  const int d = p.dest[t * p.top_k + j];
  return (unsigned)d < (unsigned)p.slots ? d : -1;
}

template <int TEAM>
__global__ __launch_bounds__(256) void dispatch_kernel(RowsParams p) {
  const int64_t t = team_token<TEAM>();
  const u32x4* in = static_cast<const u32x4*>(p.in);
  u32x4* out = static_cast<u32x4*>(p.out);
  if (t < p.tokens)
    for (int c = threadIdx.x & (TEAM - 1); c < p.pieces; c += TEAM) {
      const u32x4 v = in[t * p.pieces + c];
      for (int j = 0; j < p.top_k; ++j) {
        const int d = slot_row(p, t, j);
        if (d >= 0) out[(int64_t)d * p.pieces + c] = v;
      }
    }
  zero_rest(p);
}

// 16 bytes as fp32 values and back.
template <bool FP32>
struct Piece {
  static constexpr int kN = FP32 ? 4 : 8;
  static __device__ __forceinline__ void get(float (&f)[kN], const u32x4& x) {
    if constexpr (FP32) {
#pragma unroll
      for (int c = 0; c < 4; ++c) f[c] = __uint_as_float(x[c]);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        f[2 * c] = __uint_as_float(x[c] << 16);
        f[2 * c + 1] = __uint_as_float(x[c] & 0xffff0000u);
      }
    }
  }
  static __device__ __forceinline__ u32x4 put(const float (&f)[kN]) {
    u32x4 x;
    if constexpr (FP32) {
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = __float_as_uint(f[c]);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = pack_bf16x2(f[2 * c], f[2 * c + 1]);
    }
    return x;
  }
};

// out[t] = sum_j w[t, j] in[dest[t, j]], in fp32 in the order of j, rounded once.
template <int TEAM, bool FP32>
__global__ __launch_bounds__(256) void gather_sum_kernel(RowsParams p) {
  using Pc = Piece<FP32>;
  const int64_t t = team_token<TEAM>();
  if (t >= p.tokens) return;
  const u32x4* in = static_cast<const u32x4*>(p.in);
  for (int c = threadIdx.x & (TEAM - 1); c < p.pieces; c += TEAM) {
    float acc[Pc::kN];
#pragma unroll
    for (int i = 0; i < Pc::kN; ++i) acc[i] = 0.0f;
    for (int j = 0; j < p.top_k; ++j) {
      const int d = slot_row(p, t, j);
      if (d < 0) continue;
      const float w = p.weight ? p.weight[t * p.top_k + j] : 1.0f;
      float f[Pc::kN];
      Pc::get(f, in[(int64_t)d * p.pieces + c]);
#pragma unroll
      for (int i = 0; i < Pc::kN; ++i) acc[i] = __builtin_fmaf(w, f[i], acc[i]);
    }
    static_cast<u32x4*>(p.out)[t * p.pieces + c] = Pc::put(acc);
  }
}

// dy[dest[t, j]] = w[t, j] dout[t]; dw[t, j] = <dout[t], y[dest[t, j]]>.
template <int TEAM, bool FP32>
__global__ __launch_bounds__(256) void combine_bwd_kernel(RowsParams p) {
  using Pc = Piece<FP32>;
  constexpr int kSlots = 8;  // slots whose dot products are summed in one walk of the row
  __shared__ float s_dot[4][kSlots];
  const int64_t t = team_token<TEAM>();
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const u32x4* y = static_cast<const u32x4*>(p.in);
  const u32x4* dout = static_cast<const u32x4*>(p.dout);
  u32x4* dy = static_cast<u32x4*>(p.out);
  for (int j0 = 0; j0 < p.top_k; j0 += kSlots) {
    float dot[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) dot[j] = 0.0f;
    if (t < p.tokens)
      for (int c = threadIdx.x & (TEAM - 1); c < p.pieces; c += TEAM) {
        float g[Pc::kN];
        Pc::get(g, dout[t * p.pieces + c]);
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
          if (j0 + j >= p.top_k) break;
          const int d = slot_row(p, t, j0 + j);
          if (d < 0) continue;
          const float wt = p.weight[t * p.top_k + j0 + j];
          float f[Pc::kN], h[Pc::kN];
          Pc::get(f, y[(int64_t)d * p.pieces + c]);
#pragma unroll
          for (int i = 0; i < Pc::kN; ++i) {
            dot[j] = __builtin_fmaf(g[i], f[i], dot[j]);
            h[i] = wt * g[i];
          }
          dy[(int64_t)d * p.pieces + c] = Pc::put(h);
        }
      }
#pragma unroll
    for (int j = 0; j < kSlots; ++j) dot[j] = group_sum<64>(dot[j]);
    if constexpr (TEAM == 64) {
      if (lane == 0 && t < p.tokens)
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
          if (j0 + j < p.top_k) p.dweight[t * p.top_k + j0 + j] = dot[j];
    } else {
      if (lane == 0)
#pragma unroll
        for (int j = 0; j < kSlots; ++j) s_dot[w][j] = dot[j];
      __syncthreads();
      if (threadIdx.x < kSlots && j0 + (int)threadIdx.x < p.top_k && t < p.tokens) {
        const int j = threadIdx.x;
        p.dweight[t * p.top_k + j0 + j] = ((s_dot[0][j] + s_dot[1][j]) + s_dot[2][j]) + s_dot[3][j];
      }
      __syncthreads();
    }
  }
  zero_rest(p);
}

// A row of at least 4 KiB gives each of 256 threads a piece; a shorter one goes
// to a wave, four tokens to a block.  Measured (us, 256 / 64 threads): 4096 tokens x 8
// of 2048 bf16: dispatch 25 / 30, sum 35 / 49, gradient 48 / 58; 16384 x 4 of 1024:
// 26 / 26, 27 / 25, 70 / 50; of 512: 14 / 14, 17 / 14, 35 / 24.
bool wide_team(const RowsParams& p) { return p.pieces >= 256; }

}  // namespace

hipError_t launch_route_fwd(const RouteParams& p, int threads, hipStream_t s) {
  const size_t waves = threads / 64;
  const size_t sums = (waves * p.experts + p.experts + 4) * 4, shares = waves * 8;
  const size_t lds = sums > shares ? sums : shares;
  const dim3 g(p.blocks), b(threads);
#define MDG_ROUTE(L, V)                                                             \
  if (p.fp32) hipLaunchKernelGGL((route_fwd_kernel<L, V, true>), g, b, lds, s, p); \
  else hipLaunchKernelGGL((route_fwd_kernel<L, V, false>), g, b, lds, s, p)
  if (route_values(p.experts) == 16) {
    MDG_ROUTE(64, 16);
  } else {
    switch (route_lanes(p.experts)) {
      case 1: MDG_ROUTE(1, 8); break;
      case 2: MDG_ROUTE(2, 8); break;
      case 4: MDG_ROUTE(4, 8); break;
      case 8: MDG_ROUTE(8, 8); break;
      case 16: MDG_ROUTE(16, 8); break;
      case 32: MDG_ROUTE(32, 8); break;
      default: MDG_ROUTE(64, 8); break;
    }
  }
#undef MDG_ROUTE
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || p.blocks == 1) return err;
  hipLaunchKernelGGL(route_finish_kernel, dim3((p.experts + kFinishCols - 1) / kFinishCols), dim3(kRouteThreads), 0, s,
                     p);
  return hipGetLastError();
}

hipError_t launch_route_bwd(const RouteBwdParams& p, hipStream_t s) {
  const int rows = 256 / route_lanes(p.experts);
  const dim3 g((unsigned)((p.tokens + rows - 1) / rows)), b(256);
#define MDG_ROUTE(L, V)                                                           \
  if (p.fp32) hipLaunchKernelGGL((route_bwd_kernel<L, V, true>), g, b, 0, s, p); \
  else hipLaunchKernelGGL((route_bwd_kernel<L, V, false>), g, b, 0, s, p)
  if (route_values(p.experts) == 16) {
    MDG_ROUTE(64, 16);
  } else {
    switch (route_lanes(p.experts)) {
      case 1: MDG_ROUTE(1, 8); break;
      case 2: MDG_ROUTE(2, 8); break;
      case 4: MDG_ROUTE(4, 8); break;
      case 8: MDG_ROUTE(8, 8); break;
      case 16: MDG_ROUTE(16, 8); break;
      case 32: MDG_ROUTE(32, 8); break;
      default: MDG_ROUTE(64, 8); break;
    }
  }
#undef MDG_ROUTE
  return hipGetLastError();
}

hipError_t launch_plan(const PlanParams& p, hipStream_t s) {
  if (p.blocks > 1) {
    hipLaunchKernelGGL(plan_count_kernel, dim3(p.blocks), dim3(kPlanThreads), (size_t)p.experts * 4, s, p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  hipLaunchKernelGGL(plan_rank_kernel, dim3(p.blocks), dim3(kPlanThreads),
                     (size_t)p.experts * 4 * p.runs, s, p);
  return hipGetLastError();
}

hipError_t launch_dispatch(const RowsParams& p, hipStream_t s) {
  if (wide_team(p)) hipLaunchKernelGGL((dispatch_kernel<256>), dim3((unsigned)p.tokens), dim3(256), 0, s, p);
  else hipLaunchKernelGGL((dispatch_kernel<64>), dim3((unsigned)((p.tokens + 3) / 4)), dim3(256), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_gather_sum(const RowsParams& p, hipStream_t s) {
  const bool wide = wide_team(p);
  const dim3 g((unsigned)(wide ? p.tokens : (p.tokens + 3) / 4)), b(256);
  if (wide && p.fp32) hipLaunchKernelGGL((gather_sum_kernel<256, true>), g, b, 0, s, p);
  else if (wide) hipLaunchKernelGGL((gather_sum_kernel<256, false>), g, b, 0, s, p);
  else if (p.fp32) hipLaunchKernelGGL((gather_sum_kernel<64, true>), g, b, 0, s, p);
  else hipLaunchKernelGGL((gather_sum_kernel<64, false>), g, b, 0, s, p);
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const RowsParams& p, hipStream_t s) {
  const bool wide = wide_team(p);
  const dim3 g((unsigned)(wide ? p.tokens : (p.tokens + 3) / 4)), b(256);
  if (wide && p.fp32) hipLaunchKernelGGL((combine_bwd_kernel<256, true>), g, b, 0, s, p);
  else if (wide) hipLaunchKernelGGL((combine_bwd_kernel<256, false>), g, b, 0, s, p);
  else if (p.fp32) hipLaunchKernelGGL((combine_bwd_kernel<64, true>), g, b, 0, s, p);
  else hipLaunchKernelGGL((combine_bwd_kernel<64, false>), g, b, 0, s, p);
  return hipGetLastError();
}

}  // namespace mdg
