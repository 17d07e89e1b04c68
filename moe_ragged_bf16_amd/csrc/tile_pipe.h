// The tile products' pipeline, shared by the kernels that compute 256 x 256 output
// tiles of bf16 products in groups: the table of groups and their work units, the
// stages in LDS and the loads that fill them, the matrix products, and a unit's
// way through them.  The head of grouped_gemm_kernels.hip describes the whole.
// Included by .hip files only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "grouped_gemm.h"
#include "kernel_common.h"
#include "tile_epilogue.h"

namespace mdg {
namespace {

constexpr int kStageBytes = kTileI * kTileR * 2;  // one operand, one stage: 16 KiB
static_assert(kTileI == kTileJ, "square tiles assumed by the stage layout");
static_assert(kStageBytes == 16 * 1024, "a stage is 16 segments of 1 KiB (one wave load each)");
static_assert(kTileR == 32 && kStages == 4, "the pipeline below is written for 4 stages of 32");

// ---------------------------------------------------------------------------
// per-group work: one rule for the GEMM kernel and the reduce kernel
// ---------------------------------------------------------------------------
struct UnitShape {
  int n_i, n_j;  // tiles along i and j of one slice
};

template <int OP>
__device__ __forceinline__ UnitShape unit_shape(const GemmParams& p) {
  UnitShape s;
  if (OP == kFwd) {
    s.n_i = 1;
    s.n_j = (p.n + kTileJ - 1) / kTileJ;
  } else if (OP == kDgrad) {
    s.n_i = 1;
    s.n_j = (p.k + kTileJ - 1) / kTileJ;
  } else {
    s.n_i = (p.n + kTileI - 1) / kTileI;
    s.n_j = (p.k + kTileJ - 1) / kTileJ;
  }
  return s;
}

// Slices of a group: fwd/dgrad row tiles; wgrad row chunks (an empty expert
// still has one slice: its zero dW tiles).
template <int OP>
__device__ __forceinline__ int group_slices(int m, const GemmParams& p) {
  if (OP == kWgrad) return m == 0 ? 1 : (m + p.chunk_rows - 1) / p.chunk_rows;
  return (m + kTileI - 1) / kTileI;
}

// LDS table of the groups.  Thread t handles groups 4t .. 4t+3.
struct GroupTable {
  int* end;      // [E]     clamped, non-decreasing end row of each group
  int* uprefix;  // [E + 1] exclusive prefix of work units
  int* sprefix;  // [E]     wgrad: exclusive prefix of partial slots (split groups only)
  int* scratch;  // [4]
};

template <int OP>
__device__ int build_group_table(const GemmParams& p, GroupTable tb) {
  const int E = p.num_groups;
  const int M = (int)p.m_rows;
  const int t = threadIdx.x;
  const UnitShape us = unit_shape<OP>(p);
  const int tiles_per_slice = us.n_i * us.n_j;

  int endv[4];
  int run = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = 4 * t + q;
    int v = 0;
    if (e < E) v = min(max(p.offs[e], 0), M);
    run = max(run, v);
    endv[q] = run;
  }
  const int before = block_excl_max(run, tb.scratch);
  int units[4], slots[4];
  int usum = 0, ssum = 0;
  int start = before;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = 4 * t + q;
    const int end = max(before, endv[q]);
    const int m = end - start;
    units[q] = 0;
    slots[q] = 0;
    if (e < E) {
      const int sl = group_slices<OP>(m, p);
      units[q] = sl * tiles_per_slice;
      slots[q] = (OP == kWgrad && sl > 1) ? sl : 0;
      tb.end[e] = end;
    }
    usum += units[q];
    ssum += slots[q];
    start = end;
  }
  int utotal, stotal;
  int ub = block_excl_sum(usum, tb.scratch, &utotal);
  int sb = block_excl_sum(ssum, tb.scratch, &stotal);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = 4 * t + q;
    if (e < E) {
      tb.uprefix[e] = ub;
      tb.sprefix[e] = sb;
    }
    ub += units[q];
    sb += slots[q];
  }
  if (t == 0) tb.uprefix[E] = utotal;
  __syncthreads();
  return utotal;
}

// ---------------------------------------------------------------------------
// LDS stage layouts and the DMA that fills them
// ---------------------------------------------------------------------------
// "RC" operand (reduction contiguous in memory): 256 rows x 32 r, 64-byte LDS
// rows; 16-byte chunk c of row `row` lives at chunk c ^ swz_rc(row) with
// swz_rc(row) = (row / 2) % 4.  A fragment read (16 consecutive rows, lane group
// l / 16 reading chunk l / 16 of each) is then free of bank conflicts: measured
// with the LDS bank-conflict counter, where no swizzle, row % 4 or (row / 4) % 4
// cost about 4 extra cycles per ds_read_b128.
__device__ __forceinline__ int swz_rc(int row) { return (row >> 1) & 3; }
// "TC" operand (tile columns contiguous in memory): 32 r x 256 columns,
// 512-byte LDS rows; 16-byte chunk c of row r lives at chunk c ^ swz_tc(r) with
// swz_tc(r) = 2 * ((r % 4) + 4 * ((r / 8) % 2)).  A transposing fragment read
// touches 32 bytes of each of the 16 rows 8g + t (g, t = 0..3) or 8g + 4 + t;
// the swizzle spreads them so that each 32-byte bank window serves exactly two
// rows, the minimum for 512 bytes per instruction.
__device__ __forceinline__ int swz_tc(int r) { return 2 * ((r & 3) | (((r >> 3) & 1) << 2)); }

// Per-lane byte offsets (relative to the stage's first element in memory) of
// this wave's 4 DMA loads of one operand stage.  The 16 KiB stage is 16 segments
// of 1 KiB; wave w fills segments q*4 + w, q = 0..3; within a segment lane l
// writes LDS bytes [16 l, 16 l + 16).
template <bool TC>
__device__ __forceinline__ void dma_offsets(uint32_t (&off)[4], int ld_bytes, int w, int lane) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int seg = q * 4 + w;
    if (!TC) {
      const int row = seg * 16 + (lane >> 2);
      const int c = (lane & 3) ^ swz_rc(row);
      off[q] = (uint32_t)(row * ld_bytes + c * 16);
    } else {
      const int r = seg * 2 + (lane >> 5);
      const int c = (lane & 31) ^ swz_tc(r);
      off[q] = (uint32_t)(r * ld_bytes + c * 16);
    }
  }
}

// Byte offset, within the 64-byte stage row of an RC operand, of the 16-byte
// chunk that each of this wave's 4 loads fetches (used to mask a partial stage).
__device__ __forceinline__ void dma_chunks_rc(uint32_t (&cb)[4], int w, int lane) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int row = (q * 4 + w) * 16 + (lane >> 2);
    cb[q] = (uint32_t)(((lane & 3) ^ swz_rc(row)) * 16);
  }
}

// Operand of one unit: where its data starts and how much of it is real.  The
// byte ranges handed to the buffer loads never leave the operand's own valid
// rows, so no load can touch memory past a tensor.
struct Operand {
  const uint8_t* base;  // element (first row, first column) of the unit's panel
  int ld_bytes;         // row stride in memory
  int lim;              // RC: bytes of the valid rows (rows_valid * ld_bytes); TC: valid reduction rows
  int aux;              // RC: reduction extent in bytes; TC: valid bytes of a row (valid columns * 2)
};

// One operand stage's DMA: the buffer descriptor of stage `kt` and this wave's
// first LDS segment; load q (0..3) fills segment q * 4 + w.
struct DmaStage {
  __amdgpu_buffer_rsrc_t rs;
  uint8_t* lds;
};

template <bool TC>
__device__ __forceinline__ DmaStage dma_begin(const Operand& o, uint8_t* lds_w, int kt, bool live) {
  const int r0 = kt * kTileR;
  const uint8_t* base;
  int bytes;
  if (!TC) {
    base = o.base + r0 * 2;
    bytes = r0 * 2 < o.aux ? o.lim - r0 * 2 : 0;
  } else {
    base = o.base + (int64_t)r0 * o.ld_bytes;
    const int rows = min(max(o.lim - r0, 0), kTileR);
    bytes = rows > 0 ? (rows - 1) * o.ld_bytes + o.aux : 0;
  }
  if (!live) bytes = 0;
  bytes = uniform(bytes);  // (see dma_stage)
  DmaStage d;
  d.rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, bytes, 0x00020000);
  d.lds = lds_w;
  return d;
}

__device__ __forceinline__ void dma_one(const DmaStage& d, uint32_t off, int q) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(d.rs, (lds_void*)(d.lds + q * 4096), 16, off, 0, 0, 0);
}

// Valid bytes of each row of an RC operand's stage kt (64 for a whole stage,
// fewer in the last stage of a reduction that is not a multiple of 32).
__device__ __forceinline__ uint32_t stage_valid_bytes(const Operand& o, int kt) {
  return (uint32_t)min(max(o.aux - kt * kTileR * 2, 0), kTileR * 2);
}

// dma_one for a possibly partial RC stage: chunks at or past `kv` bytes of the
// row load zeros instead (the same instruction, with an offset out of range).
__device__ __forceinline__ void dma_one_masked(const DmaStage& d, uint32_t off, uint32_t cb, uint32_t kv, int q) {
  dma_one(d, cb < kv ? off : kOutOfRange, q);
}

// Issues this wave's DMA loads of reduction stage `kt` of one operand into the
// LDS stage at `lds` (a wave-uniform address: `lds_w` already includes this
// wave's first segment).  The buffer's range check zero-fills everything past
// the valid rows (and, for RC operands, stages past the reduction extent).
template <bool TC>
__device__ __forceinline__ void dma_stage(const Operand& o, const uint32_t (&off)[4], uint8_t* lds_w, int kt,
                                          bool live) {
  const int r0 = kt * kTileR;
  const uint8_t* base;
  int bytes;
  if (!TC) {
    base = o.base + r0 * 2;
    bytes = r0 * 2 < o.aux ? o.lim - r0 * 2 : 0;
  } else {
    base = o.base + (int64_t)r0 * o.ld_bytes;
    const int rows = min(max(o.lim - r0, 0), kTileR);
    bytes = rows > 0 ? (rows - 1) * o.ld_bytes + o.aux : 0;
  }
  if (!live) bytes = 0;  // a stage past the unit's last one: the loads only write zeros
  // The size is uniform but may be computed with vector instructions (there is
  // no scalar med3); reading it back as a scalar keeps the descriptor in SGPRs
  // instead of making the compiler wrap every load in a readfirstlane loop.
  bytes = uniform(bytes);
  const __amdgpu_buffer_rsrc_t rs =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, bytes, 0x00020000);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds_w + q * 4096), 16, off[q], 0, 0, 0);
}

// dma_stage of an RC operand whose stage may be partial (see dma_one_masked).
__device__ __forceinline__ void dma_stage_masked(const Operand& o, const uint32_t (&off)[4], const uint32_t (&cb)[4],
                                                 uint8_t* lds_w, int kt, bool live) {
  const DmaStage d = dma_begin<false>(o, lds_w, kt, live);
  const uint32_t kv = stage_valid_bytes(o, kt);
#pragma unroll
  for (int q = 0; q < 4; ++q) dma_one_masked(d, off[q], cb[q], kv, q);
}

// Waits until at most `n` vector memory operations of this wave are
// outstanding (and all its LDS reads have returned).  The immediate is the
// largest available one not above n, so the wait is never shorter than asked.
__device__ __forceinline__ void wait_vm(int n) {
  if (n >= 63) wait_vm_lgkm<63>();
  else if (n >= 56) wait_vm_lgkm<56>();
  else if (n >= 52) wait_vm_lgkm<52>();
  else if (n >= 48) wait_vm_lgkm<48>();
  else if (n >= 40) wait_vm_lgkm<40>();
  else if (n >= 32) wait_vm_lgkm<32>();
  else if (n >= 24) wait_vm_lgkm<24>();
  else if (n >= 20) wait_vm_lgkm<20>();
  else if (n >= 16) wait_vm_lgkm<16>();
  else if (n >= 8) wait_vm_lgkm<8>();
  else wait_vm_lgkm<0>();
}

// DMA loads per stage per wave (both operands).
constexpr int kDmaPerStage = 8;

// ---------------------------------------------------------------------------
// MFMA fragments from LDS
// ---------------------------------------------------------------------------
// v_mfma_f32_16x16x32_bf16 (operand layouts measured on gfx950): lane l holds
// A[m = l % 16][k = 8 (l / 16) + e] and B[k = 8 (l / 16) + e][n = l % 16],
// e = 0..7, and receives D[m = 4 (l / 16) + r][n = l % 16], r = 0..3.  Under the
// power limit this shape sustains 11-15 % more MFMA throughput on random operands
// than 32x32x16 (measured), for the same LDS traffic per FLOP.
//
// A fragment is a 16 x 32 block of one operand's stage: 16 tile rows from
// `row0`, all 32 reductions; lane l holds row row0 + l % 16, reductions
// 8 (l / 16) .. 8 (l / 16) + 7.
template <bool TC>
__device__ __forceinline__ bf16x8 load_frag(const uint8_t* st, int row0, int lane) {
  if (!TC) {
    const int row = row0 + (lane & 15);
    return *reinterpret_cast<const bf16x8*>(st + row * 64 + (((lane >> 4) ^ swz_rc(row)) << 4));
  } else {
    // ds_read_b64_tr_b16: within each 16-lane group g = l / 16, lane s addresses
    // T[r0 + s/4][m0 + 4 (s%4)] (4 columns) and receives T[r0 + q][m0 + s],
    // q = 0..3; with r0 = 8g and 8g + 4 the two reads give reductions
    // 8g .. 8g + 7 of column m0 + s.
    const int g = lane >> 4, s = lane & 15;
    const int r = 8 * g + (s >> 2);
    const int chunk = ((row0 >> 3) + ((s >> 1) & 1)) ^ swz_tc(r);  // swz_tc(r + 4) == swz_tc(r)
    const uint8_t* p0 = st + r * 512 + chunk * 16 + (s & 1) * 8;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p0));
    const s16x4 hi =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p0 + 4 * 512));
    const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, v);
  }
}

// LDS reads one fragment costs.
template <bool TC>
constexpr int frag_reads() { return TC ? 2 : 1; }

// The accumulators: 64 blocks of 16 x 16, each 4 registers kept in AGPRs.
// The MFMA is written as an asm statement whose accumulator operand must be an
// AGPR read and written in place: issued through the builtin, the register
// allocator placed part of the 64 accumulators in VGPRs and copied each one
// into and out of AGPRs around every MFMA.  The statement is volatile, so the
// LDS reads and DMA loads stay where the step places them between MFMAs.
// (Each accumulator's next MFMA is 32 MFMAs later, and the epilogue reads them
// after a barrier.)
__device__ __forceinline__ void mfma_block(f32x4& c, const bf16x8& b, const bf16x8& a) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(b), "v"(a));
}

// Wave w owns the 128 x 128 sub-tile (i: 128 (w/2), j: 128 (w%2)) as 8 x 8
// blocks of 16 x 16.  The MFMA is issued as D = Bfrag x Afrag, so D's rows are
// j: lane l then holds i = l % 16 and four consecutive j per block.  A stage is
// consumed in two halves of 32 MFMAs, row blocks 0..3 and 4..7, each walking
// the column blocks outermost so that a half needs fb[0] and its 4 A fragments
// first and one more B fragment every 4 MFMAs.
// The 4 MFMAs of column block jb in one half (row blocks ib0 .. ib0 + 3).
__device__ __forceinline__ void mma_col(Acc& acc, const bf16x8& fb, const bf16x8 (&fa)[4], int ib0, int jb) {
#pragma unroll
  for (int ib = 0; ib < 4; ++ib) mfma_block(acc[ib0 + ib][jb], fb, fa[ib]);
}

// Scheduling groups that pin the order of one half step: 32 MFMAs with `R` LDS
// reads and `V` DMA loads spread evenly between them.
template <int R, int V, int m = 0>
__device__ __forceinline__ void interleave_32() {
  if constexpr (m < 32) {
    constexpr int d = (m + 1) * R / 32 - m * R / 32;
    constexpr int v = (m + 1) * V / 32 - m * V / 32;
    if constexpr (d > 0) __builtin_amdgcn_sched_group_barrier(0x100, d, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (v > 0) __builtin_amdgcn_sched_group_barrier(0x020, v, 0);
    interleave_32<R, V, m + 1>();
  }
}

// ---------------------------------------------------------------------------
// one unit of work, decoded
// ---------------------------------------------------------------------------
struct Unit {
  int valid;
  int nk;        // reduction stages of 32, rounded up to a multiple of 4 (extra stages load zeros)
  int nkr;       // stages that hold data (nk - 3 <= nkr <= nk); the steps of the others are skipped
  Operand a, b;
  void* out;
  int64_t ldc;
  int i_valid, j_valid, mode;
};

template <int OP>
__device__ __forceinline__ Unit decode_unit(const GemmParams& p, const GroupTable& tb, const UnitShape& us,
                                            int total, int u) {
  Unit x;
  x.valid = u < total;
  if (!x.valid) return x;
  const int E = p.num_groups;
  const int N = p.n, K = p.k;
  const int e = uniform(find_group(tb.uprefix, E, u));
  const int gs = uniform(e == 0 ? 0 : tb.end[e - 1]);
  const int gm = uniform(tb.end[e]) - gs;
  const int ul = u - uniform(tb.uprefix[e]);
  const uint8_t* A = reinterpret_cast<const uint8_t*>(p.a);
  const uint8_t* B = reinterpret_cast<const uint8_t*>(p.b);
  x.mode = kStoreBf16;
  if (OP == kFwd || OP == kDgrad) {
    int rt, ct;
    panel_order(ul, (gm + kTileI - 1) / kTileI, us.n_j, 4, &rt, &ct);
    const int row0 = gs + rt * kTileI;
    x.i_valid = min(kTileI, gm - rt * kTileI);
    const int j0 = ct * kTileJ;
    x.nkr = ((OP == kFwd ? K : N) + kTileR - 1) / kTileR;
    x.nk = (x.nkr + 3) & ~3;
    if (OP == kFwd) {
      x.a = Operand{A + (int64_t)row0 * K * 2, K * 2, x.i_valid * K * 2, K * 2};        // X rows
      x.j_valid = min(kTileJ, N - j0);
      x.b = Operand{B + ((int64_t)e * N + j0) * K * 2, K * 2, x.j_valid * K * 2, K * 2};  // W[e] rows n
      x.out = static_cast<uint16_t*>(p.out) + (int64_t)row0 * N + j0;
      x.ldc = N;
    } else {
      x.a = Operand{A + (int64_t)row0 * N * 2, N * 2, x.i_valid * N * 2, N * 2};         // G rows
      x.b = Operand{B + ((int64_t)e * N * K + j0) * 2, K * 2, N, min(kTileJ, K - j0) * 2};  // W[e] columns k
      x.j_valid = min(kTileJ, K - j0);
      x.out = static_cast<uint16_t*>(p.out) + (int64_t)row0 * K + j0;
      x.ldc = K;
    }
  } else {
    const int tiles = us.n_i * us.n_j;
    const int c = ul / tiles;
    int ti, tj;
    panel_order(ul - c * tiles, us.n_i, us.n_j, 4, &ti, &tj);
    const int R = p.chunk_rows;
    int red = min(R, gm - c * R);
    red = red < 0 ? 0 : red;
    const int i0 = ti * kTileI, j0 = tj * kTileJ;
    const int64_t row0 = gs + (int64_t)c * R;  // first row of this chunk
    x.i_valid = min(kTileI, N - i0);
    x.j_valid = min(kTileJ, K - j0);
    // both operands in place, the reduction (rows) strided: rows past the chunk's
    // end load zeros (their stages are cut at `red` rows)
    x.a = Operand{A + (row0 * N + i0) * 2, N * 2, red, x.i_valid * 2};  // G rows, columns n
    x.b = Operand{B + (row0 * K + j0) * 2, K * 2, red, x.j_valid * 2};  // X rows, columns k
    x.nkr = (red + kTileR - 1) / kTileR;
    x.nk = (x.nkr + 3) & ~3;
    x.ldc = K;
    const int chunks = group_slices<kWgrad>(gm, p);
    if (chunks > 1) {
      const int slot = uniform(tb.sprefix[e]) + c;
      x.out = p.partial + (int64_t)slot * N * K + (int64_t)i0 * K + j0;
      x.mode = kStoreF32;
    } else if (p.out_fp32) {
      x.out = static_cast<float*>(p.out) + (int64_t)e * N * K + (int64_t)i0 * K + j0;
      x.mode = p.accumulate ? kStoreF32Acc : kStoreF32;
    } else {
      x.out = static_cast<uint16_t*>(p.out) + (int64_t)e * N * K + (int64_t)i0 * K + j0;
      x.mode = p.accumulate ? kStoreBf16Acc : kStoreBf16;
    }
  }
  return x;
}

// ---------------------------------------------------------------------------
// fwd/dgrad tail split
// ---------------------------------------------------------------------------
// With U units on a persistent grid, the U mod kBalanceSlots units left after
// whole rounds would run on a few CUs while the rest idle.  Those T tail units
// are instead cut into S consecutive ranges of their reduction (whole groups
// of 4 stages, S = min(kBalanceSlots / T, kMaxSplit, groups, slots / T)); each
// piece writes a dense fp32 partial tile and a second kernel adds the S
// partials in range order.  The plan is a function of the sizes and offs only.
// Each piece still sums its range in the one fixed order, so results stay
// bitwise reproducible.
struct Plan {
  int full;   // units processed whole (the first `full` work items)
  int tail;   // split tail units (0: no split)
  int split;  // pieces per tail unit
  int items;  // full + tail * split
};

template <int OP>
__device__ __forceinline__ Plan make_plan(const GemmParams& p, int total) {
  Plan pl{total, 0, 1, total};
  if (OP == kWgrad || p.tail_slots < 2) return pl;
  const int t = total % kBalanceSlots;
  if (t == 0) return pl;
  const int groups = (((OP == kFwd ? p.k : p.n) + kTileR - 1) / kTileR + 3) / 4;
  const int sp = min(min(kBalanceSlots / t, kMaxSplit), min(groups, p.tail_slots / t));
  if (sp < 2) return pl;
  pl.full = total - t;
  pl.tail = t;
  pl.split = sp;
  pl.items = pl.full + t * sp;
  return pl;
}

// Moves an operand's start k0 reductions further (the buffer ranges keep
// ending where the operand's valid data ends).
__device__ __forceinline__ void shift_rc(Operand& o, int k0) {
  o.base += 2 * k0;
  o.lim -= 2 * k0;
  o.aux -= 2 * k0;
}
__device__ __forceinline__ void shift_tc(Operand& o, int k0) {
  o.base += (int64_t)k0 * o.ld_bytes;
  o.lim -= k0;
}

__device__ __forceinline__ TailUnit* tail_table(const GemmParams& p) {
  return reinterpret_cast<TailUnit*>(reinterpret_cast<uint8_t*>(p.tail_head) + 256);
}

// Work item v: a whole unit, or piece s of tail unit t.
template <int OP>
__device__ __forceinline__ Unit decode_item(const GemmParams& p, const GroupTable& tb, const UnitShape& us,
                                            int total, const Plan& pl, int v) {
  if (OP == kWgrad || v < pl.full) return decode_unit<OP>(p, tb, us, total, v);
  Unit x;
  x.valid = v < pl.items;
  if (!x.valid) return x;
  const int q = v - pl.full;
  const int t = q / pl.split, sp = q - t * pl.split;
  x = decode_unit<OP>(p, tb, us, total, pl.full + t);
  if (sp == 0 && threadIdx.x == 0) {  // where the reduce kernel writes this tile
    TailUnit* tu = tail_table(p) + t;
    tu->out = static_cast<uint16_t*>(x.out);
    tu->ldc = (int)x.ldc;
    tu->i_valid = x.i_valid;
    tu->j_valid = x.j_valid;
    tu->pad = 0;
  }
  const int g = x.nk / 4;
  const int g0 = sp * g / pl.split, g1 = (sp + 1) * g / pl.split;
  const int k0 = 4 * g0 * kTileR;
  x.nk = 4 * (g1 - g0);
  x.nkr = min(x.nk, x.nkr - 4 * g0);
  shift_rc(x.a, k0);
  if (OP == kFwd) shift_rc(x.b, k0);
  else shift_tc(x.b, k0);
  x.out = p.partial + (int64_t)q * (kTileI * kTileJ);  // slot t * split + sp
  x.ldc = kTileJ;
  x.i_valid = kTileI;
  x.j_valid = kTileJ;
  x.mode = kStoreF32;
  return x;
}

// ---------------------------------------------------------------------------
// the GEMM kernel
// ---------------------------------------------------------------------------
// The LDS stage ring: one separate array per (stage buffer, operand).  Distinct
// objects let the compiler prove that reading one buffer does not depend on the
// loads still landing in the others, so it never waits for the whole load queue
// before an LDS read.
__shared__ __attribute__((aligned(1024))) uint8_t s_a0[kStageBytes];
__shared__ __attribute__((aligned(1024))) uint8_t s_a1[kStageBytes];
__shared__ __attribute__((aligned(1024))) uint8_t s_a2[kStageBytes];
__shared__ __attribute__((aligned(1024))) uint8_t s_a3[kStageBytes];
__shared__ __attribute__((aligned(1024))) uint8_t s_b0[kStageBytes];
__shared__ __attribute__((aligned(1024))) uint8_t s_b1[kStageBytes];
__shared__ __attribute__((aligned(1024))) uint8_t s_b2[kStageBytes];
__shared__ __attribute__((aligned(1024))) uint8_t s_b3[kStageBytes];

template <int S>
__device__ __forceinline__ uint8_t* stage_a() {
  if constexpr (S == 0) return s_a0;
  else if constexpr (S == 1) return s_a1;
  else if constexpr (S == 2) return s_a2;
  else return s_a3;
}
template <int S>
__device__ __forceinline__ uint8_t* stage_b() {
  if constexpr (S == 0) return s_b0;
  else if constexpr (S == 1) return s_b1;
  else if constexpr (S == 2) return s_b2;
  else return s_b3;
}

// MASK: the reduction extent is not a multiple of 32, so the last stage of an
// RC operand is partial and its loads mask the chunks past the extent.
// PAIRS: stages of the row-read operands are loaded in pairs (see kPairs).
template <int OP, bool MASK, bool PAIRS>
struct Pipe {
  // operands with the reduction strided: W in dgrad, G and X in wgrad
  static constexpr bool ATC = (OP == kWgrad);
  static constexpr bool BTC = (OP != kFwd);
  // Stages loaded in pairs (fwd, dgrad: an operand is read along its rows).  A
  // stage of such an operand holds 64 bytes of each row, half a 128-byte cache
  // line, and the next stage the other half: loaded a step apart, every line
  // would come from the L2 twice (the L1 no longer holds it); requested by
  // consecutive instructions, the L1 merges the two halves into one fetch.
  // (Transposed operands load 512-byte row segments, whole lines already, so
  // dgrad pairs only A; wgrad pairs nothing.)  The pairing shortens by one
  // step the lead of the first stage of each pair, which costs more than it
  // saves when a unit streams its weights from HBM (few rows per expert), so
  // for fwd it is a launch choice.
  static constexpr bool kPairs = PAIRS && !(ATC && BTC);
  static constexpr bool kPairB = kPairs && !BTC;
  uint32_t off_a[4], off_b[4];
  uint32_t cb_a[4], cb_b[4];  // MASK: chunk byte positions of the RC loads (dma_chunks_rc)
  int w, wi, wj, lane;

  // This wave's 4 DMA loads of operand A (resp. B) of stage kt into buffer S.
  template <int S>
  __device__ __forceinline__ void issue_a(const Unit& x, int kt) const {
    if constexpr (MASK && !ATC) dma_stage_masked(x.a, off_a, cb_a, stage_a<S>() + w * 1024, kt, kt < x.nk);
    else dma_stage<ATC>(x.a, off_a, stage_a<S>() + w * 1024, kt, kt < x.nk);
  }
  template <int S>
  __device__ __forceinline__ void issue_b(const Unit& x, int kt) const {
    if constexpr (MASK && !BTC) dma_stage_masked(x.b, off_b, cb_b, stage_b<S>() + w * 1024, kt, kt < x.nk);
    else dma_stage<BTC>(x.b, off_b, stage_b<S>() + w * 1024, kt, kt < x.nk);
  }

  // One load of stage kt's operand (masked when the stage may be partial).
  template <bool TC>
  __device__ __forceinline__ void dma_q(const DmaStage& d, uint32_t off, uint32_t cb, uint32_t kv, int q) const {
    if constexpr (MASK && !TC) dma_one_masked(d, off, cb, kv, q);
    else dma_one(d, off, q);
  }

  // This wave's loads of operand A (resp. B) of stages kt and kt+1 into buffers
  // S and S+1, the two halves of each row segment by consecutive instructions.
  template <int S>
  __device__ __forceinline__ void issue_a_pair(const Unit& x, int kt) const {
    const DmaStage d0 = dma_begin<ATC>(x.a, stage_a<S>() + w * 1024, kt, kt < x.nk);
    const DmaStage d1 = dma_begin<ATC>(x.a, stage_a<S + 1>() + w * 1024, kt + 1, kt + 1 < x.nk);
    const uint32_t k0 = MASK && !ATC ? stage_valid_bytes(x.a, kt) : 0;
    const uint32_t k1 = MASK && !ATC ? stage_valid_bytes(x.a, kt + 1) : 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      dma_q<ATC>(d0, off_a[q], cb_a[q], k0, q);
      dma_q<ATC>(d1, off_a[q], cb_a[q], k1, q);
    }
  }
  template <int S>
  __device__ __forceinline__ void issue_b_pair(const Unit& x, int kt) const {
    const DmaStage d0 = dma_begin<BTC>(x.b, stage_b<S>() + w * 1024, kt, kt < x.nk);
    const DmaStage d1 = dma_begin<BTC>(x.b, stage_b<S + 1>() + w * 1024, kt + 1, kt + 1 < x.nk);
    const uint32_t k0 = MASK && !BTC ? stage_valid_bytes(x.b, kt) : 0;
    const uint32_t k1 = MASK && !BTC ? stage_valid_bytes(x.b, kt + 1) : 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      dma_q<BTC>(d0, off_b[q], cb_b[q], k0, q);
      dma_q<BTC>(d1, off_b[q], cb_b[q], k1, q);
    }
  }

  // A short unit: a wgrad unit of fewer than 4 real stages (a group or row
  // chunk of at most 96 rows; most units of workloads with many small
  // experts).  Stages 0..2 are loaded ahead as for every unit (those past its
  // last real stage load zeros and move no memory), it issues no other load,
  // and it runs its real stages without the ring: the stages it leaves out
  // would only add products of zeros, which leave every accumulator bit as it
  // is.  fwd and dgrad reduce over K or N and have no short units.
  static __device__ __forceinline__ bool is_short(const Unit& x) { return OP == kWgrad && x.nkr < 4; }

  // Stage S of a short unit (landed in every wave): the same MFMAs, in the
  // same order per accumulator, as a step of the ring.
  template <int S>
  __device__ __forceinline__ void short_stage(Acc& acc) const {
    bf16x8 fa[2][4], fb[8];
#pragma unroll
    for (int b = 0; b < 8; ++b) fb[b] = load_frag<BTC>(stage_b<S>(), wj * 128 + 16 * b, lane);
#pragma unroll
    for (int b = 0; b < 8; ++b) fa[b >> 2][b & 3] = load_frag<ATC>(stage_a<S>(), wi * 128 + 16 * b, lane);
#pragma unroll
    for (int jb = 0; jb < 8; ++jb) mma_col(acc, fb[jb], fa[0], 0, jb);
#pragma unroll
    for (int jb = 0; jb < 8; ++jb) mma_col(acc, fb[jb], fa[1], 4, jb);
  }

  // A unit's first stages, loaded while the previous unit's epilogue runs (or
  // at the start): stages 0..2 (kPairs: stages 0 and 1 as a pair, then stage
  // 2).  Stage 3 (its operand A; fwd: all of it) follows once the epilogue,
  // which stages its results through stage 3's buffers, is done (issue_last,
  // at the top of a ring unit).
  __device__ __forceinline__ void prefetch_first(const Unit& x) const {
    if constexpr (kPairB) {
      issue_a_pair<0>(x, 0);
      issue_b_pair<0>(x, 0);
    } else if constexpr (kPairs) {
      issue_a_pair<0>(x, 0);
      issue_b<0>(x, 0);
      issue_b<1>(x, 1);
    } else {
      issue_a<0>(x, 0);
      issue_b<0>(x, 0);
      issue_a<1>(x, 1);
      issue_b<1>(x, 1);
    }
    issue_a<2>(x, 2);
    issue_b<2>(x, 2);
  }
  __device__ __forceinline__ void issue_last(const Unit& x) const {
    issue_a<3>(x, 3);
    if constexpr (kPairB) issue_b<3>(x, 3);  // (otherwise the first step issues it)
  }
  // Loads issued after the last one of what a unit's first step needs (fwd:
  // the pairs of stages 0, 1, followed by stage 2 and stage 3; dgrad: B of
  // stage 0, followed by B of stage 1, stage 2 and A of stage 3; wgrad: B of
  // stage 0, followed by stages 1, 2 and A of stage 3), up to and including
  // issue_last, not counting the epilogue's own operations in between.
  static constexpr int kAfterStage0 = kPairs ? 2 * kDmaPerStage : 2 * kDmaPerStage + kDmaPerStage / 2;

  // The per-stage step (wgrad; fwd and dgrad load stages in pairs, see
  // step_pairs, which keeps the same MFMA and fragment-read order).
  // Stage kt, held in buffer S = kt % 4.  On entry its 8 B fragments are in fbc
  // and its A fragments of row blocks 0..3 in fal.  First half: read the A
  // fragments of row blocks 4..7 into fah, issue operand B of stage kt+3 (zeros
  // past the last stage) and run the 32 MFMAs of row blocks 0..3; then wait for
  // stage kt+1 and pass the barrier, after which no wave reads buffer S any
  // more.  Second half: issue operand A of stage kt+4 into buffer S, read stage
  // kt+1's B fragments into fbn and its first A fragments into fal (in the order
  // the next half consumes them) and run the 32 MFMAs of row blocks 4..7.  Each
  // half spreads its 4 loads per wave over its MFMAs, and the step is
  // branch-free: one scheduling region per half in which loads, LDS reads and
  // MFMAs interleave.
  //
  // The wait for stage kt+1 must allow exactly the memory operations issued
  // after its last loads (operand B, one step before stage kt's): the 16 loads
  // of stage kt+2 and stage kt+3 plus the extra operations issued after those
  // (the previous unit's last stores), which the caller tracks in e2 (two steps
  // back) and e1 (one step back).
  //
  // kFirst: one of a unit's first 4 steps, where e1 and e2 may be nonzero; in
  // all later steps they are zero and the wait is a constant (no compare chain
  // in the steady-state loop).
  template <int S, bool kFirst>
  __device__ __forceinline__ void step(Acc& acc, const bf16x8 (&fbc)[8], bf16x8 (&fbn)[8],
                                       bf16x8 (&fal)[4], bf16x8 (&fah)[4], const Unit& x, int kt, int& e1,
                                       int& e2) const {
    if constexpr (kPairs) {
      step_pairs<S, kFirst>(acc, fbc, fbn, fal, fah, x, kt, e1);
      return;
    }
    constexpr int S1 = (S + 1) & 3, S3 = (S + 3) & 3;
    static_assert(kDmaPerStage == 8, "4 loads per operand and wave");
    // first half: row blocks 0..3; reads of fah early, operand B of stage kt+3
    // after every second column block
    const DmaStage db = dma_begin<BTC>(x.b, stage_b<S3>() + w * 1024, kt + 3, kt + 3 < x.nk);
    const uint32_t kvb = MASK && !BTC ? stage_valid_bytes(x.b, kt + 3) : 0;
#pragma unroll
    for (int jb = 0; jb < 8; ++jb) {
      mma_col(acc, fbc[jb], fal, 0, jb);
      if (jb < 4) fah[jb] = load_frag<ATC>(stage_a<S>(), wi * 128 + 64 + 16 * jb, lane);
      if (jb & 1) {
        if constexpr (MASK && !BTC) dma_one_masked(db, off_b[jb >> 1], cb_b[jb >> 1], kvb, jb >> 1);
        else dma_one(db, off_b[jb >> 1], jb >> 1);
      }
    }
    if constexpr (kFirst) {
      wait_vm(2 * kDmaPerStage + e2 + e1);  // stage kt+1 has landed
      e2 = e1;
      e1 = 0;
    } else {
      wait_vm_lgkm<2 * kDmaPerStage>();
    }
    lds_barrier();  // ... in every wave; stage kt's reads all returned
    // second half: row blocks 4..7; stage kt+1's fragments in the order the next
    // half consumes them (fb[0], fa[0..3], fb[1..7]), operand A of stage kt+4
    // into stage kt's buffer (after the last stage these reads are discarded)
    const DmaStage da = dma_begin<ATC>(x.a, stage_a<S>() + w * 1024, kt + 4, kt + 4 < x.nk);
    const uint32_t kva = MASK && !ATC ? stage_valid_bytes(x.a, kt + 4) : 0;
#pragma unroll
    for (int jb = 0; jb < 8; ++jb) {
      mma_col(acc, fbc[jb], fah, 4, jb);
      if (jb == 0) {
        fbn[0] = load_frag<BTC>(stage_b<S1>(), wj * 128, lane);
        fal[0] = load_frag<ATC>(stage_a<S1>(), wi * 128, lane);
      } else if (jb < 4) {
        fal[jb] = load_frag<ATC>(stage_a<S1>(), wi * 128 + 16 * jb, lane);
        fbn[jb] = load_frag<BTC>(stage_b<S1>(), wj * 128 + 16 * jb, lane);
      } else {
        fbn[jb] = load_frag<BTC>(stage_b<S1>(), wj * 128 + 16 * jb, lane);
      }
      if (jb & 1) {
        if constexpr (MASK && !ATC) dma_one_masked(da, off_a[jb >> 1], cb_a[jb >> 1], kva, jb >> 1);
        else dma_one(da, off_a[jb >> 1], jb >> 1);
      }
    }
  }

  // Stage 0's B fragments and A fragments of row blocks 0..3 (after its wait).
  // The step with stages in pairs (kPairs).  Operand A of stages 2m and 2m+1
  // is issued in the second half of step 2m-3 (odd), into the buffers of
  // stages 2m-4 and 2m-3, which no wave reads any more once every wave is past
  // step 2m-3's first half.  Two loads per column block there, 8 per half step
  // at most, because a burst of loads in one half stalls the MFMAs behind them.
  //
  // fwd (kPairB): operand B of stages 2m, 2m+1 follows in the first half of
  // step 2m-2 (even).  Only odd steps synchronise: they wait for the pair their
  // second half starts reading (nothing is issued after it by then, so the
  // wait is for all of this wave's loads) and pass one barrier, which makes the
  // pair visible everywhere and frees the buffers the next A and B pairs go to
  // (B's even-step loads go to buffers last read before that barrier).  An even
  // step reads the second stage of a pair waited for one step earlier.
  //
  // dgrad: operand B (transposed, whole lines) keeps its per-stage slot, the
  // first half of step kt-3 for stage kt, and every step waits and passes the
  // barrier.  The wait for stage kt+1 allows the loads issued after its last
  // one: for even kt, B of stage kt+1 is last and 16 follow (B of kt+2, the A
  // pair of kt+3 and kt+4, B of kt+3); for odd kt, A of stage kt+1 is last but
  // one in its pair and 9 follow (A of kt+2's last load, B of kt+2 and kt+3).
  // A unit's first two steps also count the loads of the prologue and the
  // previous unit's epilogue (e1): step 0 waits for B of stage 1 (followed by
  // stage 2, e1, A and B of stage 3: 16 + e1); step 1 for B of stage 2
  // (followed by e1, A of stage 3, B of stages 3 and 4: 12 + e1).
  template <int S, bool kFirst>
  __device__ __forceinline__ void step_pairs(Acc& acc, const bf16x8 (&fbc)[8], bf16x8 (&fbn)[8],
                                             bf16x8 (&fal)[4], bf16x8 (&fah)[4], const Unit& x, int kt,
                                             int e1) const {
    constexpr int S1 = (S + 1) & 3, S2 = (S + 2) & 3, S3 = (S + 3) & 3;
    constexpr bool kOdd = (S & 1) != 0;
    // first half: B loads (fwd: the pair kt+2, kt+3 on even steps but the first,
    // whose stages 2 and 3 came with the prologue; dgrad: stage kt+3)
    constexpr bool kIssueB = kPairB ? (!kOdd && !(kFirst && S == 0)) : true;
    DmaStage b0{}, b1{};
    uint32_t kb0 = 0, kb1 = 0;
    if constexpr (kIssueB) {
      if constexpr (kPairB) {
        b0 = dma_begin<BTC>(x.b, stage_b<S2>() + w * 1024, kt + 2, kt + 2 < x.nk);
        b1 = dma_begin<BTC>(x.b, stage_b<S3>() + w * 1024, kt + 3, kt + 3 < x.nk);
        if constexpr (MASK) {
          kb0 = stage_valid_bytes(x.b, kt + 2);
          kb1 = stage_valid_bytes(x.b, kt + 3);
        }
      } else {
        b0 = dma_begin<BTC>(x.b, stage_b<S3>() + w * 1024, kt + 3, kt + 3 < x.nk);
      }
    }
#pragma unroll
    for (int jb = 0; jb < 8; ++jb) {
      mma_col(acc, fbc[jb], fal, 0, jb);
      if (jb < 4) fah[jb] = load_frag<ATC>(stage_a<S>(), wi * 128 + 64 + 16 * jb, lane);
      if constexpr (kIssueB) {
        const int q = jb >> 1;
        if constexpr (kPairB) {
          if ((jb & 1) == 0) {
            dma_q<BTC>(b0, off_b[q], cb_b[q], kb0, q);
            dma_q<BTC>(b1, off_b[q], cb_b[q], kb1, q);
          }
        } else if (jb & 1) {
          dma_q<BTC>(b0, off_b[q], cb_b[q], 0, q);
        }
      }
    }
    if constexpr (kPairB) {
      if constexpr (kOdd) wait_vm_lgkm<0>();  // stages kt+1, kt+2 have landed; stage kt's reads returned
    } else if constexpr (kFirst && S == 0) {
      wait_vm(2 * kDmaPerStage + e1);
    } else if constexpr (kFirst && S == 1) {
      wait_vm(kDmaPerStage + kDmaPerStage / 2 + e1);
    } else {
      wait_vm_lgkm<kOdd ? kDmaPerStage + 1 : 2 * kDmaPerStage>();  // stage kt+1 has landed
    }
    if constexpr (!kPairB || kOdd) lds_barrier();  // ... in every wave; stage kt's reads returned
    // second half: operand A of stages kt+3, kt+4 on odd steps
    DmaStage a0{}, a1{};
    uint32_t ka0 = 0, ka1 = 0;
    if constexpr (kOdd) {
      a0 = dma_begin<ATC>(x.a, stage_a<S3>() + w * 1024, kt + 3, kt + 3 < x.nk);
      a1 = dma_begin<ATC>(x.a, stage_a<S>() + w * 1024, kt + 4, kt + 4 < x.nk);
      if constexpr (MASK) {
        ka0 = stage_valid_bytes(x.a, kt + 3);
        ka1 = stage_valid_bytes(x.a, kt + 4);
      }
    }
#pragma unroll
    for (int jb = 0; jb < 8; ++jb) {
      mma_col(acc, fbc[jb], fah, 4, jb);
      if (jb == 0) {
        fbn[0] = load_frag<BTC>(stage_b<S1>(), wj * 128, lane);
        fal[0] = load_frag<ATC>(stage_a<S1>(), wi * 128, lane);
      } else if (jb < 4) {
        fal[jb] = load_frag<ATC>(stage_a<S1>(), wi * 128 + 16 * jb, lane);
        fbn[jb] = load_frag<BTC>(stage_b<S1>(), wj * 128 + 16 * jb, lane);
      } else {
        fbn[jb] = load_frag<BTC>(stage_b<S1>(), wj * 128 + 16 * jb, lane);
      }
      if constexpr (kOdd) {
        const int q = jb >> 1;
        if ((jb & 1) == 0) {
          dma_q<ATC>(a0, off_a[q], cb_a[q], ka0, q);
          dma_q<ATC>(a1, off_a[q], cb_a[q], ka1, q);
        }
      }
    }
  }

  __device__ __forceinline__ void first_frags(bf16x8 (&fb)[8], bf16x8 (&fal)[4]) const {
    fb[0] = load_frag<BTC>(stage_b<0>(), wj * 128, lane);
#pragma unroll
    for (int b = 0; b < 4; ++b) fal[b] = load_frag<ATC>(stage_a<0>(), wi * 128 + 16 * b, lane);
#pragma unroll
    for (int b = 1; b < 8; ++b) fb[b] = load_frag<BTC>(stage_b<0>(), wj * 128 + 16 * b, lane);
  }
};

}  // namespace
}  // namespace mdg
