// gfx950 (CDNA4) kernels of the experts' gated feed-forward for groups that do not fill
// 256-row tiles (gated_kernels.hip has the formulas): the small kernel for few rows,
// which streams weights to registers, and the middle kernel's tiles of 128 x 128 or 64 x 64.
//
// The order of every sum is fixed: results are bitwise reproducible.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gated.h"
#include "gated_act.h"
#include "grouped_gemm.h"
#include "kernel_common.h"

namespace mdg {
namespace {

// Row pieces of TILE rows, group by group, `per` units to a piece.  Finds unit `slot`:
// its group, the group's first row and rows, and the unit's number within the group;
// false where there is none (for the whole workgroup of 256 threads, 4 groups each, so
// that any number of groups takes one round of loads).  `spread`: slots are workgroups,
// which go round the XCDs, and each XCD takes consecutive units, an eighth of those
// there are (the grid is an upper bound: by its size the first XCDs would get more).
struct Rows {
  int e, start, rows, unit;
};
template <int TILE>
__device__ __forceinline__ bool find_rows(const GemmParams& p, int slot, int per, bool spread, Rows* out) {
  __shared__ int s_scratch[4];
  __shared__ Rows s_rows;
  const int E = p.num_groups, M = (int)p.m_rows, t = threadIdx.x;
  int end[4], run = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (4 * t + q < E) run = max(run, min(max(p.offs[4 * t + q], 0), M));
    end[q] = run;
  }
  const int before = block_excl_max(run, s_scratch);
  int units[4], sum = 0, start = before;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    end[q] = max(end[q], before);
    units[q] = (end[q] - start + TILE - 1) / TILE * per;
    sum += units[q];
    start = end[q];
  }
  int total;
  int u = block_excl_sum(sum, s_scratch, &total);
  int v = slot;
  if (spread) {
    const int share = (total + 7) / 8;
    v = (slot >> 3) < share ? (slot & 7) * share + (slot >> 3) : total;
  }
  if (v >= total) return false;
  start = before;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (v >= u && v < u + units[q]) s_rows = Rows{4 * t + q, start, end[q] - start, v - u};
    u += units[q];
    start = end[q];
  }
  __syncthreads();
  out->e = uniform(s_rows.e);
  out->start = uniform(s_rows.start);
  out->rows = uniform(s_rows.rows);
  out->unit = uniform(s_rows.unit);
  return true;
}

__device__ __forceinline__ u32x2 pack4(const f32x4& v) {
  u32x2 pk;
  pk[0] = pack_bf16x2(v[0], v[1]);
  pk[1] = pack_bf16x2(v[2], v[3]);
  return pk;
}

__device__ __forceinline__ f32x4 mfma(const bf16x8& b, const bf16x8& a, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
}

// Wait states between a matrix instruction and the first other access of its result,
// tied to the results (the build checks the generated code for them).
template <int I, int J>
__device__ __forceinline__ void settle(f32x4 (&acc)[I][J]) {
  asm volatile("s_nop 15");
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) asm volatile("" : "+v"(acc[i][j]));
}

// ---------------------------------------------------------------------------
// the small kernel (fwd)
// ---------------------------------------------------------------------------
// A workgroup computes up to 64 rows of 16 hidden columns: 16 rows of W_gate and 16 of
// W_up, straight from memory into matrix operands, and the rows of x through the
// caches.  Its four waves take pieces of 256 of K in turn and their sums are added in wave
// order.  The weights' bytes bound it: all of a piece's loads go out before the first
// product (16 of 16 bytes a lane, 12 waves to a CU).  2 rows in two groups of 2 x 14336 x 4096
// take 83 us, 5.6 TB/s; 100 rows over 8 groups of 2 x 512 x 1024 8 us, most of it latency.
constexpr int kSmallPiece = 256;

template <int MB, int ACT>
__device__ __forceinline__ void small_gated(const GatedParams& gp, int e, int row0, int rows, int f0, f32x4* s_acc) {
  const GemmParams& p = gp.g;
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const int K = p.k, f = gp.f, r = lane & 15, c = (lane >> 4) * 16;
  const int cols = min(kGatedSmallCols, f - f0);
  const uint16_t* wg = p.b + ((int64_t)e * 2 * f + f0) * K;
  __amdgpu_buffer_rsrc_t rw[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    rw[j] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(wg + (j ? (int64_t)f * K : 0)), 0,
                                              uniform(cols * K * 2), 0x00020000);
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(p.a) + (int64_t)row0 * K, 0, uniform(rows * K * 2), 0x00020000);
  f32x4 acc[MB][2];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = w * kSmallPiece; k0 < K; k0 += 4 * kSmallPiece) {
    // 16 bytes of step s (32 of K) of row `row`; those past the row's end read zeros
    const auto load = [&](const __amdgpu_buffer_rsrc_t& rs, int row, int s) {
      const int at = (k0 + s * 32) * 2 + c;
      return __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(
                                            rs, at < K * 2 ? (uint32_t)(row * K * 2 + at) : kOutOfRange, 0, 0));
    };
    bf16x8 wf[8][2], xf[MB == 1 ? 8 : 1];
#pragma unroll
    for (int s = 0; s < 8; ++s)
#pragma unroll
      for (int j = 0; j < 2; ++j) wf[s][j] = load(rw[j], r, s);
    if constexpr (MB == 1) {
#pragma unroll
      for (int s = 0; s < 8; ++s) xf[s] = load(rx, r, s);
    }
    __builtin_amdgcn_sched_barrier(0);  // (left to itself the compiler moves each load next to its use)
#pragma unroll
    for (int s = 0; s < 8; ++s)
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        bf16x8 x;
        if constexpr (MB == 1) x = xf[s];
        else x = load(rx, i * 16 + r, s);
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma(wf[s][j], x, acc[i][j]);
      }
  }
  settle(acc);
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) s_acc[((i * 2 + j) * 4 + w) * 64 + lane] = acc[i][j];
  __syncthreads();
  // row block w: lane l holds row l % 16, hidden columns 4 (l / 16) .. + 3
  const int row = w * 16 + r, col = f0 + (lane >> 4) * 4;
  if (w >= MB || row >= rows || col >= f) return;
  f32x4 a = s_acc[(w * 2) * 4 * 64 + lane], b = s_acc[(w * 2 + 1) * 4 * 64 + lane], h;
#pragma unroll
  for (int q = 1; q < 4; ++q) {
    a += s_acc[(w * 2 * 4 + q) * 64 + lane];
    b += s_acc[((w * 2 + 1) * 4 + q) * 64 + lane];
  }
#pragma unroll
  for (int x = 0; x < 4; ++x) h[x] = Act<ACT>::hidden(a[x], b[x]);
  const int64_t t = row0 + row;
  *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.out) + t * f + col) = pack4(h);
  if (gp.keep != nullptr) {
    *reinterpret_cast<u32x2*>(gp.keep + t * 2 * f + col) = pack4(a);
    *reinterpret_cast<u32x2*>(gp.keep + t * 2 * f + f + col) = pack4(b);
  }
}

template <int ACT>
__global__ __launch_bounds__(256, 3) void gated_small_kernel(GatedParams gp) {
  __shared__ f32x4 s_acc[kGatedSmallRows / 16 * 2 * 4 * 64];
  Rows u;
  if (!find_rows<kGatedSmallRows>(gp.g, blockIdx.y, 1, false, &u)) return;
  const int row0 = u.start + u.unit * kGatedSmallRows, rows = min(kGatedSmallRows, u.rows - u.unit * kGatedSmallRows);
  const int f0 = blockIdx.x * kGatedSmallCols;
  if (rows <= 16) small_gated<1, ACT>(gp, u.e, row0, rows, f0, s_acc);
  else if (rows <= 32) small_gated<2, ACT>(gp, u.e, row0, rows, f0, s_acc);
  else small_gated<4, ACT>(gp, u.e, row0, rows, f0, s_acc);
}

// ---------------------------------------------------------------------------
// the middle kernel
// ---------------------------------------------------------------------------
// Tiles of 128 rows x 128 columns (fwd: 64 hidden columns, gate and up in turns of 16;
// dgrad: 128 hidden columns), four waves of 64 x 64, stages of 64 reductions (16 KiB an
// operand), two buffers, two workgroups to a CU, one of which computes while the other
// waits (with 256 tiles, as dgrad has for 3001 rows over 16 groups of 2000 x 1000, a CU has
// one, and nothing runs beside its loads: 47 to 60 % of its wave cycles are waits for them and
// for barriers); and 64 x 64 (32 x 32 a wave) where those leave CUs idle (mid_tile of
// capi_gated.cpp): a workgroup reads, waits and multiplies in turn, so a smaller tile's
// stages are shorter (one group of 100 rows of 2 x 2048 x 2048 12.6 us, 20 in tiles of 128,
// also with four buffers in place of two).
// With tiles enough, what a CU takes in bounds it, 34 to 45 GB/s with all of them at it: 64
// groups of 128 rows on average of 2 x 1536 x 2048 take 200 us, 12 TB/s into LDS; rows that
// do not start on cache lines (k no multiple of 64) ask for two lines where one would do, and
// loads issue no faster than the L1 works those off (1.69 times the lines from L2; 57 % of the
// wave cycles wait to issue an instruction, 47 % on cache lines): 16 groups of 188 rows on
// average of 2 x 1000 x 2000 62 us, of 2 x 1024 x 2048 47.  With few rows the weights' bytes
// do: 488 rows over 64 groups of 2 x 1536 x 2048 139 us, 5.7 TB/s.
// (Tried and not kept: weights straight to registers and four buffers of rows, 192 KiB on
// their way to a CU, 0 to 12 % longer; 256 rows and eight waves, a quarter fewer bytes but
// one workgroup to a CU, 20 to 40 % longer; two stages' loads and fragments at a time, so that
// a line that both need is asked for at once: no faster for either k.)
// Buffer B of operand A (0) or B (1); each a static array of its own, so that the compiler
// can tell reads of one from loads still landing in another.
template <int OPERAND, int B, int TILE>
__device__ __forceinline__ uint8_t* mid_buffer() {
  __shared__ __attribute__((aligned(1024))) uint8_t s_buf[TILE * 128];
  return s_buf;
}

// An operand read along its rows: LDS rows of 64 reductions (128 bytes), 16-byte chunk c of
// row r at c ^ (r % 8).  A fragment is 16 rows x 32 reductions (half h).
__device__ __forceinline__ bf16x8 mid_frag(const uint8_t* st, int row0, int h, int lane) {
  const int r = row0 + (lane & 15);
  return *reinterpret_cast<const bf16x8*>(st + r * 128 + (((h * 4 + (lane >> 4)) ^ (r & 7)) << 4));
}
// An operand with its reduction strided: 64 reductions x TILE columns, LDS rows of 2 TILE
// bytes, chunk c of reduction r at c ^ swz(r), read by the transposing LDS read (as
// load_frag of tile_pipe.h, whose rows are 512 bytes): each 32-byte window then serves two
// of an instruction's 16 rows, the least for its 512 bytes.
template <int TILE>
__device__ __forceinline__ int mid_swz(int r) {
  return TILE == 128 ? 2 * ((r & 3) | (((r >> 3) & 1) << 2)) : (r & 2) | (((r >> 3) & 1) << 2);
}
template <int TILE>
__device__ __forceinline__ bf16x8 mid_frag_t(const uint8_t* st, int col0, int h, int lane) {
  const int g = lane >> 4, s = lane & 15, r = h * 32 + 8 * g + (s >> 2);
  const int chunk = ((col0 >> 3) + ((s >> 1) & 1)) ^ mid_swz<TILE>(r);
  const uint8_t* p0 = st + r * (2 * TILE) + chunk * 16 + (s & 1) * 8;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p0));
  const s16x4 hi =
      __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p0 + 4 * (2 * TILE)));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// bf16 rows of 128 bytes in LDS (chunk c of row r at c ^ (r / 2 % 8)) to columns
// f0 .. f0 + valid of rows row0 .. of a tensor with rows of `ld`: 8 rows an instruction.
template <int TILE>
__device__ __forceinline__ void mid_store_rows(const uint8_t* st, uint16_t* to, int64_t ld, int row0, int f0, int i_valid,
                                               int f_valid, int w, int lane) {
#pragma unroll
  for (int q = 0; q < TILE / 32; ++q) {
    const int r = (w * (TILE / 32) + q) * 8 + (lane >> 3), c = lane & 7;
    if (r < i_valid && c * 8 < f_valid)
      *reinterpret_cast<u32x4*>(to + (int64_t)(row0 + r) * ld + f0 + c * 8) =
          *reinterpret_cast<const u32x4*>(st + r * 128 + ((c ^ ((r >> 1) & 7)) << 4));
  }
}

template <int OP, int ACT, int TILE>
__global__ __launch_bounds__(256, TILE == 128 ? 2 : 4) void gated_mid_kernel(GatedParams gp) {
  const GemmParams& p = gp.g;
  constexpr int kCols = OP == kFwd ? TILE / 2 : TILE;  // hidden columns of a tile
  constexpr int kB = TILE / 32;                        // blocks of 16 each way of a wave's quarter; loads of an operand
  const int f = gp.f, n_j = (f + kCols - 1) / kCols;
  Rows u;
  if (!find_rows<TILE>(p, blockIdx.x, n_j, true, &u)) return;
  int rt, ct;
  panel_order(u.unit, (u.rows + TILE - 1) / TILE, n_j, 4, &rt, &ct);
  const int row0 = u.start + rt * TILE, i_valid = min(TILE, u.rows - rt * TILE);
  const int f0 = ct * kCols, f_valid = min(kCols, f - f0);
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6), wi = w >> 1, wj = w & 1;
  const int R = OP == kFwd ? p.k : p.n;  // the reduction, and A's row length
  const int nk = (R + 63) / 64;
  // A: segments 4 q + w of 8 rows; lane l loads chunk (l % 8) ^ (l / 8) of row l / 8 of it
  const uint16_t* xa = p.a + (int64_t)row0 * R;
  const uint32_t chunk = (uint32_t)(((lane & 7) ^ (lane >> 3)) * 16);
  const uint32_t off_a = (uint32_t)(w * 8 + (lane >> 3)) * (uint32_t)(R * 2) + chunk;
  // B, fwd: segment 4 q + w of 8 tile columns, in column block 2 q + w / 2: gate (w < 2) or up of
  // hidden column 16 q + 8 (w % 2) + l / 8.
  // B, dgrad: segments of kS = 512 / TILE reductions; lane l loads chunk (l % C) ^ swz of
  // reduction 4 kS q + kS w + l / C, C = TILE / 8 chunks a row (the swizzle does not depend on q)
  const uint16_t* xb = OP == kFwd ? p.b + ((int64_t)u.e * 2 * f + (w < 2 ? 0 : f) + f0) * R
                                  : p.b + (int64_t)u.e * R * f + f0;
  constexpr int kS = 512 / TILE, kC = TILE / 8;
  const int rb = kS * w + lane / kC;
  const uint32_t chunk_t = (uint32_t)(((lane % kC) ^ mid_swz<TILE>(rb)) * 16);
  const uint32_t off_b = OP == kFwd ? (uint32_t)((w & 1) * 8 + (lane >> 3)) * (uint32_t)(R * 2) + chunk
                                    : (uint32_t)rb * (uint32_t)(f * 2) + chunk_t;
  const bool in_b = OP == kFwd || (int)chunk_t < f_valid * 2;

  auto load_stage = [&](auto buffer, int kt) {
    constexpr int B = decltype(buffer)::value;
    const int left = (R - kt * 64) * 2;  // bytes of a row of A from here on
    const bool in = left > 0;
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(xa) + (in ? kt * 64 : 0), 0, uniform(in ? i_valid * R * 2 - kt * 128 : 0), 0x00020000);
    __amdgpu_buffer_rsrc_t rbs;
    if constexpr (OP == kFwd) {
      rbs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(xb) + (in ? kt * 64 : 0), 0,
                                              uniform(in ? f_valid * R * 2 - kt * 128 : 0), 0x00020000);
    } else {  // (reductions past R lie past the last row's end)
      const int rows = min(64, R - kt * 64);
      rbs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(xb) + (in ? (int64_t)kt * 64 * f : 0), 0,
                                              uniform(in ? (rows - 1) * f * 2 + f_valid * 2 : 0), 0x00020000);
    }
#pragma unroll
    for (int q = 0; q < kB; ++q) {
      const uint32_t at = (int)chunk < left ? off_a + (uint32_t)(q * 32) * (uint32_t)(R * 2) : kOutOfRange;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(mid_buffer<0, B, TILE>() + (q * 4 + w) * 1024), 16, at,
                                               0, 0, 0);
      uint32_t bt;
      if constexpr (OP == kFwd) bt = (int)chunk < left ? off_b + (uint32_t)(q * 16) * (uint32_t)(R * 2) : kOutOfRange;
      else bt = in_b ? off_b + (uint32_t)(q * 4 * kS) * (uint32_t)(f * 2) : kOutOfRange;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rbs, (lds_void*)(mid_buffer<1, B, TILE>() + (q * 4 + w) * 1024), 16, bt,
                                               0, 0, 0);
    }
  };
  f32x4 acc[kB][kB];
#pragma unroll
  for (int i = 0; i < kB; ++i)
#pragma unroll
    for (int j = 0; j < kB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // Stage kt, in buffer kt % 2: wait for its loads (the next stage's follow them) and
  // read its fragments; a second barrier after the reads frees its buffer for stage kt + 2.
  auto step = [&](auto buffer, int kt) {
    constexpr int B = decltype(buffer)::value;
    wait_vm_lgkm<2 * kB>();
    lds_barrier();
    bf16x8 a[2][kB], b[2][kB];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < kB; ++i) {
        a[h][i] = mid_frag(mid_buffer<0, B, TILE>(), wi * (TILE / 2) + i * 16, h, lane);
        if constexpr (OP == kFwd) b[h][i] = mid_frag(mid_buffer<1, B, TILE>(), wj * (TILE / 2) + i * 16, h, lane);
        else b[h][i] = mid_frag_t<TILE>(mid_buffer<1, B, TILE>(), wj * (TILE / 2) + i * 16, h, lane);
      }
    wait_vm_lgkm<2 * kB>();
    lds_barrier();  // every wave has its fragments
    load_stage(buffer, kt + 2);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < kB; ++i)
#pragma unroll
        for (int j = 0; j < kB; ++j) acc[i][j] = mfma(b[h][j], a[h][i], acc[i][j]);
  };
  load_stage(std::integral_constant<int, 0>{}, 0);
  load_stage(std::integral_constant<int, 1>{}, 1);
  int kt = 0;
  for (; kt + 2 <= nk; kt += 2) {
    step(std::integral_constant<int, 0>{}, kt);
    step(std::integral_constant<int, 1>{}, kt + 1);
  }
  if (kt < nk) step(std::integral_constant<int, 0>{}, kt);
  settle(acc);
  wait_vm_lgkm<0>();
  __syncthreads();  // no load in flight, every wave past its reads: the buffers are free

  uint8_t *const s0 = mid_buffer<0, 0, TILE>(), *const s1 = mid_buffer<0, 1, TILE>();
  const int r16 = lane & 15, q4 = lane >> 4;
  if constexpr (OP == kFwd) {
    // acc[i][2 j], [2 j + 1]: gate and up of hidden columns 8 kB wj + 16 j ..; lane l holds row l % 16,
    // columns 4 (l / 16) .. + 3 of a block.
    const auto place = [&](int i, int j) {
      const int r = wi * (TILE / 2) + i * 16 + r16;
      return r * 128 + (((wj * kB + j * 2 + (q4 >> 1)) ^ ((r >> 1) & 7)) << 4) + (q4 & 1) * 8;
    };
    uint16_t* const h = static_cast<uint16_t*>(p.out);
    if (gp.keep != nullptr) {
#pragma unroll
      for (int i = 0; i < kB; ++i)
#pragma unroll
        for (int j = 0; j < kB / 2; ++j) {
          *reinterpret_cast<u32x2*>(s0 + place(i, j)) = pack4(acc[i][2 * j]);
          *reinterpret_cast<u32x2*>(s1 + place(i, j)) = pack4(acc[i][2 * j + 1]);
        }
      __syncthreads();
      mid_store_rows<TILE>(s0, gp.keep, 2 * f, row0, f0, i_valid, f_valid, w, lane);
      mid_store_rows<TILE>(s1, gp.keep + f, 2 * f, row0, f0, i_valid, f_valid, w, lane);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kB; ++i)
#pragma unroll
      for (int j = 0; j < kB / 2; ++j) {
        f32x4 v;
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = Act<ACT>::hidden(acc[i][2 * j][x], acc[i][2 * j + 1][x]);
        *reinterpret_cast<u32x2*>(s0 + place(i, j)) = pack4(v);
      }
    __syncthreads();
    mid_store_rows<TILE>(s0, h, f, row0, f0, i_valid, f_valid, w, lane);
  } else {
    // 32 of a wave's TILE / 2 rows of dh at a time in fp32 in memory of its own, rows of 2 TILE bytes,
    // chunk c of row r at c ^ (r % kC); a lane then has 8 columns of rows kR q + l / kL.
    constexpr int kL = TILE / 16, kR = 64 / kL;  // lanes of a row, rows an instruction
    uint8_t* xo = (w < 2 ? s0 : s1) + (w & 1) * (TILE * 64);
    const int col = wj * (TILE / 2) + (lane % kL) * 8;
    u32x4 av[TILE / 2 / kR], bv[TILE / 2 / kR];
#pragma unroll
    for (int q = 0; q < TILE / 2 / kR; ++q) {
      const int r = wi * (TILE / 2) + q * kR + lane / kL;
      const bool in = r < i_valid && col < f_valid;
      const uint16_t* g = gp.gate_up + (in ? (int64_t)(row0 + r) * 2 * f + f0 + col : 0);
      av[q] = *reinterpret_cast<const u32x4*>(g);
      bv[q] = *reinterpret_cast<const u32x4*>(g + f);
    }
#pragma unroll
    for (int half = 0; half < kB / 2; ++half) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < kB; ++j)
          *reinterpret_cast<f32x4*>(xo + (i * 16 + r16) * (2 * TILE) + (((j * 4 + q4) ^ (r16 % kC)) << 4)) =
              acc[2 * half + i][j];
#pragma unroll
      for (int q = 0; q < 32 / kR; ++q) {
        const int rr = q * kR + lane / kL, c = (lane % kL) * 2;
        const f32x4 lo = *reinterpret_cast<const f32x4*>(xo + rr * (2 * TILE) + ((c ^ (rr % kC)) << 4));
        const f32x4 hi = *reinterpret_cast<const f32x4*>(xo + rr * (2 * TILE) + (((c + 1) ^ (rr % kC)) << 4));
        u32x4 da, db;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t a = av[32 / kR * half + q][x], b = bv[32 / kR * half + q][x];
          float p0, p1, g0, g1;
          Act<ACT>::grads(lo_f(a), lo_f(b), x < 2 ? lo[2 * x] : hi[2 * x - 4], &p0, &g0);
          Act<ACT>::grads(hi_f(a), hi_f(b), x < 2 ? lo[2 * x + 1] : hi[2 * x - 3], &p1, &g1);
          da[x] = pack_bf16x2(p0, p1);
          db[x] = pack_bf16x2(g0, g1);
        }
        const int r = wi * (TILE / 2) + half * 32 + rr;
        if (r < i_valid && col < f_valid) {
          uint16_t* d = static_cast<uint16_t*>(p.out) + (int64_t)(row0 + r) * 2 * f + f0 + col;
          *reinterpret_cast<u32x4*>(d) = da;
          *reinterpret_cast<u32x4*>(d + f) = db;
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_gated_small(const GatedParams& p, int pieces, hipStream_t s) {
  const dim3 g((p.f + kGatedSmallCols - 1) / kGatedSmallCols, pieces), b(256);
  if (p.act == kActSilu) hipLaunchKernelGGL((gated_small_kernel<kActSilu>), g, b, 0, s, p);
  else hipLaunchKernelGGL((gated_small_kernel<kActGeluTanh>), g, b, 0, s, p);
  return hipGetLastError();
}

template <int OP, int ACT>
static void launch_mid(const GatedParams& p, int tile, int grid, hipStream_t s) {
  const dim3 g(grid), b(256);
  if (tile == kGatedMidTile) hipLaunchKernelGGL((gated_mid_kernel<OP, ACT, kGatedMidTile>), g, b, 0, s, p);
  else hipLaunchKernelGGL((gated_mid_kernel<OP, ACT, kGatedMidTile / 2>), g, b, 0, s, p);
}

hipError_t launch_gated_mid(Op op, const GatedParams& p, int tile, int grid, hipStream_t s) {
  const bool silu = p.act == kActSilu;
  if (op == kFwd && silu) launch_mid<kFwd, kActSilu>(p, tile, grid, s);
  else if (op == kFwd) launch_mid<kFwd, kActGeluTanh>(p, tile, grid, s);
  else if (silu) launch_mid<kDgrad, kActSilu>(p, tile, grid, s);
  else launch_mid<kDgrad, kActGeluTanh>(p, tile, grid, s);
  return hipGetLastError();
}

}  // namespace mdg
