// gfx950 (CDNA4) kernels of the deterministic ragged BF16 grouped GEMM.
//
// Operations (Cake ragged BF16 grouped GEMM API page, operations table), for
// expert e owning rows [s_e, t_e) of the packed activations:
//   fwd    Y [s_e:t_e] = X[s_e:t_e] @ W[e]^T
//   dgrad  dX[s_e:t_e] = G[s_e:t_e] @ W[e]          (W read in place)
//   wgrad  dW[e]       = G[s_e:t_e]^T @ X[s_e:t_e]
// All three are one tile GEMM  C[i][j] = sum_r A(i, r) * B(j, r):
//   fwd    i = row, j = n, r = k:   A = X (r contiguous),   B = W[e] (r contiguous)
//   dgrad  i = row, j = k, r = n:   A = G (r contiguous),   B = W[e] (j contiguous)
//   wgrad  i = n,   j = k, r = row: A = G (i contiguous),   B = X (j contiguous)
//
// Structure of one launch:
//  * Offsets are read on the device only.  Each workgroup loads offs into LDS,
//    clamps them to a non-decreasing sequence in [0, M] (bad offsets stay memory
//    safe and groups never overlap) and builds, with block-wide scans, the
//    prefix of work units per group.  No host sync, no atomics.
//  * Persistent grid: workgroup b walks work items v(b), v(b) + P, ... where v
//    spreads consecutive workgroup ids (dealt round-robin over the 8 XCDs) so
//    that each XCD works on a contiguous run of units, whose tiles share operand
//    panels in that XCD's L2.
//  * Units are 256 x 256 output tiles (fwd/dgrad: one row tile of one group;
//    wgrad: one row chunk of one expert).  fwd/dgrad cut the units left over
//    after whole rounds into reduction ranges (the tail split below).
//  * The reduction is staged 32 deep into a ring of 4 LDS buffers per operand
//    by buffer loads that write LDS directly (no registers); the buffer range
//    check turns rows past a group's or chunk's end into zeros.  Up to three
//    stages are in flight while the MFMAs of the current one run; the next
//    unit's first stages load during the current epilogue.  A wgrad unit of at
//    most 96 rows runs its few stages from those alone.  Where an operand is
//    read along its rows (fwd; dgrad's A), two consecutive stages hold the two
//    halves of each 128-byte line and are loaded as a pair, so that the L1
//    fetches every line from the L2 once (see Pipe::kPairs).
//  * LDS layouts follow the memory layout of each operand, with 16-byte-chunk
//    XOR swizzles that keep the fragment reads free of bank conflicts:
//      r-contiguous operand  [256 rows][32 r]  read with ds_read_b128;
//      i/j-contiguous operand [32 r][256 cols] read with ds_read_b64_tr_b16, the
//      gfx950 transposing LDS read, which hands each lane 4 consecutive r of one
//      column, so no operand is ever transposed in registers.
//  * v_mfma_f32_16x16x32_bf16 with fp32 accumulators in AGPRs, one fixed
//    reduction order: results are bitwise reproducible.
//  * Epilogues pass each wave's results through LDS so that global accesses
//    cover whole 256-byte row segments.
//  * wgrad reads G and X where they lie, both with the reduction (rows)
//    strided; row chunks of a split expert write fp32 partials that a second
//    kernel adds in chunk order (a fixed-order split of the reduction).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>

#include "grouped_gemm.h"
#include "kernel_common.h"
#include "tile_epilogue.h"
#include "tile_pipe.h"

// Scratch of the allocation-free fwd entry point (grouped_det_gemm_fwd_noalloc):
// the tail plan head and the fp32 partial tiles of the tail split, sized for
// the largest fwd call.  Each device holds its own copy for the life of the
// process.  Host code must not pass this name to a kernel (on the host it is a
// stand-in, not a device address): it uses the per-device address that
// fwd_scratch_address() looks up below.  Nothing in it has to start at zero:
// the GEMM kernel writes the plan and the partial tiles before the reduce
// kernel, next on the same stream, reads them.
static __device__ __align__(256) uint8_t scratch[mdg::kFwdScratchBytes];

namespace mdg {
namespace {

// bf16 pair + bf16 pair, each element RNE_bf16(RN32(f32(a) + f32(b))): both
// widen exactly to fp32, one IEEE fp32 add, one rounding to bf16.
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  const float lo = __fadd_rn(__uint_as_float(a << 16), __uint_as_float(b << 16));
  const float hi = __fadd_rn(__uint_as_float(a & 0xffff0000u), __uint_as_float(b & 0xffff0000u));
  return pack_bf16x2(lo, hi);
}

// Cache policy of the accumulating epilogues' destination reads and writes:
// non-temporal.  The destination is touched once per call, and without the hint
// its lines push the operand panels other units still read out of the L2
// (measured: fine-grained and many-expert shapes 3-6 % faster, bitwise the same).
constexpr int kStreaming = 2;

// dst = RN32(dst + acc) over the wave's fp32 sub-tile: one IEEE fp32 add per
// element of the finished product (no contraction).  The destination reads of
// the next half slab are in flight while the current one is staged and added.
__device__ __forceinline__ void epilogue_accumulate(const Acc& acc, const OutTile& t, uint8_t* xb,
                                                    int lane) {
  const Staging x = staging(xb, lane, false);
  f32x4 old[2][8];
#pragma unroll
  for (int q = 0; q < 8; ++q) old[0][q] = __builtin_amdgcn_raw_buffer_load_b128(t.rs, slab_off(t, 0, q, 0), 0, kStreaming);
#pragma unroll
  for (int hs = 0; hs < 8; ++hs) {
    const int ib = hs >> 1, jh = hs & 1;
    __builtin_amdgcn_sched_barrier(0);  // one half slab at a time (bounds the registers in use)
    if (hs + 1 < 8) {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        old[(hs + 1) & 1][q] = __builtin_amdgcn_raw_buffer_load_b128(t.rs, slab_off(t, (hs + 1) >> 1, q, (hs + 1) & 1), 0, kStreaming);
    }
    stage_slab<kStoreF32>(acc, x, ib, jh);
    u32x4 v[8];
    unstage_slab(v, x);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const f32x4 n = __builtin_bit_cast(f32x4, v[q]);
      f32x4 o = old[hs & 1][q];
      o[0] = __fadd_rn(o[0], n[0]);
      o[1] = __fadd_rn(o[1], n[1]);
      o[2] = __fadd_rn(o[2], n[2]);
      o[3] = __fadd_rn(o[3], n[3]);
      __builtin_amdgcn_raw_buffer_store_b128(o, t.rs, slab_off(t, ib, q, jh), 0, kStreaming);
    }
  }
}

// dst = RNE_bf16(RN32(f32(dst) + f32(RNE_bf16(acc)))) over the wave's bf16
// sub-tile: the dW tile is rounded to bf16 first (the overwrite result), then
// added to the destination the way two bf16 tensors are added.  The
// destination reads of the next slab are in flight while the current one is
// staged and added.
__device__ __forceinline__ void epilogue_accumulate_bf16(const Acc& acc, const OutTile& t, uint8_t* xb,
                                                         int lane) {
  const Staging x = staging(xb, lane, true);
  u32x4 old[2][8];
#pragma unroll
  for (int q = 0; q < 8; ++q) old[0][q] = __builtin_amdgcn_raw_buffer_load_b128(t.rs, slab_off(t, 0, q, 0), 0, kStreaming);
#pragma unroll
  for (int ib = 0; ib < 4; ++ib) {
    __builtin_amdgcn_sched_barrier(0);  // one slab at a time (bounds the registers in use)
    if (ib + 1 < 4) {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        old[(ib + 1) & 1][q] = __builtin_amdgcn_raw_buffer_load_b128(t.rs, slab_off(t, ib + 1, q, 0), 0, kStreaming);
    }
    stage_slab<kStoreBf16>(acc, x, ib, 0);
    u32x4 v[8];
    unstage_slab(v, x);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      u32x4 o = old[ib & 1][q];
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] = add_bf16x2(o[c], v[q][c]);
      __builtin_amdgcn_raw_buffer_store_b128(o, t.rs, slab_off(t, ib, q, 0), 0, kStreaming);
    }
  }
}

// The epilogue of one unit in its store mode; returns the number of vector
// memory operations it issued.
template <int OP, int OUT>
__device__ __forceinline__ int run_epilogue(const Acc& acc, const Unit& cur, const OutTile& ot,
                                            uint8_t* xb, int lane, bool rmw) {
  if constexpr (OP != kWgrad) {
    if (cur.mode == kStoreBf16) {
      epilogue_store<kStoreBf16>(acc, ot, xb, lane);
      return epilogue_ops<kStoreBf16>();
    }
    epilogue_store<kStoreF32>(acc, ot, xb, lane);  // a piece of a split tail unit: fp32 partial tile
    return epilogue_ops<kStoreF32>();
  } else {
    if (rmw) {
      if constexpr (OUT == kStoreBf16Acc) {
        epilogue_accumulate_bf16(acc, ot, xb, lane);
        return epilogue_ops<kStoreBf16Acc>();
      } else {
        epilogue_accumulate(acc, ot, xb, lane);
        return epilogue_ops<kStoreF32Acc>();
      }
    }
    if (OUT == kStoreBf16 && cur.mode == kStoreBf16) {
      epilogue_store<kStoreBf16>(acc, ot, xb, lane);
      return epilogue_ops<kStoreBf16>();
    }
    epilogue_store<kStoreF32>(acc, ot, xb, lane);
    return epilogue_ops<kStoreF32>();
  }
}

// Per unit, with stages of 32 reductions in a ring of 4 LDS buffers:
//   * stages 0..2 are loaded ahead (for every unit but the first, during the
//     previous unit's epilogue), operand A of stage 3 right after it;
//   * stage kt: issue operand B of stage kt+3 into the buffer stage kt-1 used;
//     read the second half of stage kt's fragments while the MFMAs of its
//     first half run; wait for stage kt+1 and pass one barrier; issue operand
//     A of stage kt+4 into stage kt's buffer and read the first half of stage
//     kt+1's fragments while the MFMAs of stage kt's second half run.
// One barrier per stage, and no MFMA waits on an LDS read.  A wgrad unit of at
// most 3 real stages (a short unit) has them all loaded ahead and runs them
// without the ring, so no load follows the previous epilogue's stores and its
// own end does not wait for them (vector memory operations complete in order).
// OUT: the output's store mode (bf16 for fwd and dgrad; bf16, fp32 or their
// accumulating forms for wgrad).  Units of split wgrad experts store fp32
// partials.
template <int OP, int OUT, bool MASK, bool PAIRS>
__global__ __launch_bounds__(kThreads, 1) void grouped_gemm_kernel(GemmParams p) {
  using Pp = Pipe<OP, MASK, PAIRS>;
  constexpr bool ATC = Pp::ATC;
  constexpr bool BTC = Pp::BTC;
  __shared__ int s_end[kMaxGroups];
  __shared__ int s_uprefix[kMaxGroups + 1];
  __shared__ int s_sprefix[kMaxGroups];
  __shared__ int s_scratch[4];

  GroupTable tb{s_end, s_uprefix, s_sprefix, s_scratch};
  const int total = uniform(build_group_table<OP>(p, tb));  // (from LDS: make it visibly uniform)
  const UnitShape us = unit_shape<OP>(p);
  const Plan pl = make_plan<OP>(p, total);
  if (OP != kWgrad && p.tail_head != nullptr && blockIdx.x == 0 && threadIdx.x == 0) {
    p.tail_head[0] = pl.tail;  // read by the tail reduce kernel
    p.tail_head[1] = pl.split;
  }

  const int P = gridDim.x;
  const int bid = blockIdx.x;
  const int vb = (P % 8 == 0) ? (bid % 8) * (P / 8) + bid / 8 : bid;

  Pp pipe;
  pipe.lane = threadIdx.x & 63;
  pipe.w = uniform(threadIdx.x >> 6);
  pipe.wi = pipe.w >> 1;
  pipe.wj = pipe.w & 1;
  // DMA offsets depend only on the operands' row strides (fixed per launch).
  const int lda = OP == kFwd ? p.k * 2 : p.n * 2;
  const int ldb = p.k * 2;
  dma_offsets<ATC>(pipe.off_a, lda, pipe.w, pipe.lane);
  dma_offsets<BTC>(pipe.off_b, ldb, pipe.w, pipe.lane);
  if constexpr (MASK) {
    dma_chunks_rc(pipe.cb_a, pipe.w, pipe.lane);
    dma_chunks_rc(pipe.cb_b, pipe.w, pipe.lane);
  }

  // wgrad: every unit ends in a long epilogue (the main_grad read-modify-write)
  // and the units of a persistent launch start together, so the first
  // epilogues of all workgroups coincide and contend for HBM (measured: unit 0's
  // take ~20 us on all CUs at once, ~10 us once they have drifted apart).
  // Half of each XCD's workgroups start ~16k cycles later, which spreads them
  // from the first unit on (+1 to +2 % on the Mixtral-like, gate_up and fine
  // shapes; bitwise the same).  Not worth it for launches of a few units.
  if (OP == kWgrad && ((bid >> 3) & 1) && total >= 4 * P) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i) __builtin_amdgcn_s_sleep(127);
  }
  Unit cur = decode_item<OP>(p, tb, us, total, pl, vb);
  if (cur.valid) pipe.prefetch_first(cur);
  int tail = 0;  // memory operations issued between stage 2 and stage 3's operand A of the current unit
  for (int u = vb; cur.valid; u += P) {
    Acc acc;
    const bool rmw = (OUT == kStoreF32Acc || OUT == kStoreBf16Acc) && cur.mode == OUT;
    if (Pp::is_short(cur)) {
      zero(acc);
      // All of this unit's stages were loaded ahead; only the previous unit's
      // epilogue operations were issued after them, and those stores drain
      // while this unit computes and stages its own results (no load of this
      // unit is in flight at its end, so nothing waits for them here).
      if (cur.nkr > 0) {
        wait_vm(tail);  // this unit's stages have landed ...
        lds_barrier();  // ... in every wave
        pipe.template short_stage<0>(acc);
        if (cur.nkr > 1) pipe.template short_stage<1>(acc);
        if (cur.nkr > 2) pipe.template short_stage<2>(acc);
      }
      wait_vm_lgkm<63>();  // this wave's LDS reads have returned ...
      lds_barrier();       // ... in every wave, before the next unit's loads
    } else {
      // The rest of stage 3, now that the previous epilogue is done with its
      // buffers.  Issued only here, by a unit that drains all its loads before
      // its epilogue, so no stage load is ever in flight into the staging
      // buffers when an epilogue (of either kind of unit) writes them, and the
      // compiler sees as much.
      pipe.issue_last(cur);
      zero(acc);
      if (cur.nk > 0) {
        bf16x8 fbA[8], fbB[8], fal[4], fah[4];
        int e1 = tail, e2 = 0;
        wait_vm(Pp::kAfterStage0 + tail);  // stage 0 (kPairs: stages 0, 1) has landed
        lds_barrier();                     // ... in every wave
        pipe.first_frags(fbA, fal);
        // nk is a positive multiple of 4: the first 4 steps, then the steady state
        // The first 4 steps always run; after them, steps of stages past nkr
        // (zeros) are skipped.  A step's wait counts only loads issued before it
        // (by the prefetch and earlier steps), so leaving out the last steps
        // changes no wait; their loads, already in flight, drain at the wait
        // after the loop.  (Guarding the first 4 steps as well made the compiler
        // schedule the whole loop worse: measured 3-5 % slower.)
        const int nkr = cur.nkr;
        pipe.template step<0, true>(acc, fbA, fbB, fal, fah, cur, 0, e1, e2);
        pipe.template step<1, true>(acc, fbB, fbA, fal, fah, cur, 1, e1, e2);
        pipe.template step<2, true>(acc, fbA, fbB, fal, fah, cur, 2, e1, e2);
        pipe.template step<3, true>(acc, fbB, fbA, fal, fah, cur, 3, e1, e2);
        int kt = 4;
        for (; kt + 4 <= nkr; kt += 4) {
          pipe.template step<0, false>(acc, fbA, fbB, fal, fah, cur, kt, e1, e2);
          pipe.template step<1, false>(acc, fbB, fbA, fal, fah, cur, kt + 1, e1, e2);
          pipe.template step<2, false>(acc, fbA, fbB, fal, fah, cur, kt + 2, e1, e2);
          pipe.template step<3, false>(acc, fbB, fbA, fal, fah, cur, kt + 3, e1, e2);
        }
        if (kt < nkr) {
          pipe.template step<0, false>(acc, fbA, fbB, fal, fah, cur, kt, e1, e2);
          if (kt + 1 < nkr) pipe.template step<1, false>(acc, fbB, fbA, fal, fah, cur, kt + 1, e1, e2);
          if (kt + 2 < nkr) pipe.template step<2, false>(acc, fbA, fbB, fal, fah, cur, kt + 2, e1, e2);
        }
      }
      wait_vm_lgkm<0>();
      __syncthreads();  // every wave is done reading LDS before the next unit's loads
    }

    // Epilogue, overlapped with the next unit's first stages: stages 0..2 load
    // into their buffers while the results pass through the staging buffers
    // (the last stage buffers, 8 KiB per wave) to memory; operand A of stage 3
    // follows once every wave is done with them (at the top of the next unit).
    const Unit nxt = decode_item<OP>(p, tb, us, total, pl, u + P);
    if (nxt.valid) pipe.prefetch_first(nxt);
    const int ln = lane_here();
    const OutTile ot = out_tile(cur.out, cur.ldc, cur.i_valid, cur.j_valid, pipe.wi, pipe.wj, ln,
                                is_bf16_mode(cur.mode) ? 2 : 4);
    // Waves 0, 1 stage through s_a3, waves 2, 3 through s_b3.  Each branch names
    // its array, so the compiler can tell the staging accesses apart from the
    // stage loads still landing in the other buffers (a pointer selected at run
    // time would make it wait for all of them first).
    if (pipe.w < 2) tail = run_epilogue<OP, OUT>(acc, cur, ot, s_a3 + (pipe.w & 1) * 8192, ln, rmw);
    else tail = run_epilogue<OP, OUT>(acc, cur, ot, s_b3 + (pipe.w & 1) * 8192, ln, rmw);
    wait_vm_lgkm<63>();  // the staging reads have returned ...
    lds_barrier();       // ... in every wave
    cur = nxt;
  }
  wait_vm_lgkm<0>();
}

// ---------------------------------------------------------------------------
// wgrad: fixed-order sum of the chunk partials of split experts
// ---------------------------------------------------------------------------
// blockIdx.y picks the y-th split expert (in expert order); blockIdx.x strides
// over its N*K elements, 4 per thread.  Partials are added in chunk order
// ((p0 + p1) + p2) + ..., then the same epilogue as an unsplit expert runs.
__global__ __launch_bounds__(kThreads) void wgrad_reduce_kernel(GemmParams p) {
  __shared__ int s_end[kMaxGroups];
  __shared__ int s_uprefix[kMaxGroups + 1];
  __shared__ int s_sprefix[kMaxGroups];
  __shared__ int s_scratch[4];
  __shared__ int s_pick[2];

  GroupTable tb{s_end, s_uprefix, s_sprefix, s_scratch};
  build_group_table<kWgrad>(p, tb);
  const int E = p.num_groups;
  const int t = threadIdx.x;

  // Ordinal of each split expert among split experts.
  int flags[4], cnt = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = 4 * t + q;
    flags[q] = 0;
    if (e < E) {
      const int gs = (e == 0) ? 0 : s_end[e - 1];
      flags[q] = group_slices<kWgrad>(s_end[e] - gs, p) > 1;
    }
    cnt += flags[q];
  }
  if (t == 0) s_pick[0] = -1;
  int total;
  int ord = block_excl_sum(cnt, s_scratch, &total);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (flags[q] && ord == (int)blockIdx.y) s_pick[0] = 4 * t + q;
    ord += flags[q];
  }
  __syncthreads();
  const int e = s_pick[0];
  if (e < 0) return;

  const int gs = (e == 0) ? 0 : s_end[e - 1];
  const int chunks = group_slices<kWgrad>(s_end[e] - gs, p);
  const int64_t nk4 = (int64_t)p.n * p.k / 4;
  const f32x4* part = reinterpret_cast<const f32x4*>(p.partial) + (int64_t)s_sprefix[e] * nk4;
  for (int64_t x = (int64_t)blockIdx.x * kThreads + t; x < nk4; x += (int64_t)gridDim.x * kThreads) {
    f32x4 s = part[x];
    for (int c = 1; c < chunks; ++c) {
      const f32x4 v = part[(int64_t)c * nk4 + x];
      s[0] = __fadd_rn(s[0], v[0]);
      s[1] = __fadd_rn(s[1], v[1]);
      s[2] = __fadd_rn(s[2], v[2]);
      s[3] = __fadd_rn(s[3], v[3]);
    }
    const int64_t o = (int64_t)e * nk4 + x;
    if (p.out_fp32) {
      f32x4* out = reinterpret_cast<f32x4*>(p.out) + o;
      if (p.accumulate) {
        f32x4 old = *out;
        old[0] = __fadd_rn(old[0], s[0]);
        old[1] = __fadd_rn(old[1], s[1]);
        old[2] = __fadd_rn(old[2], s[2]);
        old[3] = __fadd_rn(old[3], s[3]);
        *out = old;
      } else {
        *out = s;
      }
    } else {
      u32x2* out = reinterpret_cast<u32x2*>(p.out) + o;
      u32x2 pk;
      pk[0] = pack_bf16x2(s[0], s[1]);
      pk[1] = pack_bf16x2(s[2], s[3]);
      if (p.accumulate) {
        const u32x2 old = *out;
        pk[0] = add_bf16x2(old[0], pk[0]);
        pk[1] = add_bf16x2(old[1], pk[1]);
      }
      *out = pk;
    }
  }
}

// ---------------------------------------------------------------------------
// fwd/dgrad: fixed-order sum of the tail pieces
// ---------------------------------------------------------------------------
// blockIdx.y picks the tail unit, blockIdx.x a set of rows of its tile.  The
// plan and the tile destinations come from the workspace head written by the
// GEMM kernel just before on the same stream.  Each thread adds 8 consecutive
// columns of one row over the pieces in range order ((p0 + p1) + p2) + ...,
// rounds to bf16 and writes the valid part of the tile.
__global__ __launch_bounds__(kThreads) void tail_reduce_kernel(GemmParams p) {
  const int T = uniform(p.tail_head[0]);
  const int S = uniform(p.tail_head[1]);
  const int t = blockIdx.y;
  if (t >= T || S < 2) return;
  const TailUnit tu = tail_table(p)[t];
  const float* part = p.partial + (int64_t)t * S * (kTileI * kTileJ);
  const int col = (threadIdx.x & 31) * 8;
  for (int row = blockIdx.x * 8 + (threadIdx.x >> 5); row < kTileI; row += gridDim.x * 8) {
    const f32x4* src = reinterpret_cast<const f32x4*>(part + row * kTileJ + col);
    f32x4 lo = src[0], hi = src[1];
    for (int s = 1; s < S; ++s) {
      const f32x4* q = reinterpret_cast<const f32x4*>(part + (int64_t)s * (kTileI * kTileJ) + row * kTileJ + col);
      const f32x4 a = q[0], b = q[1];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        lo[c] = __fadd_rn(lo[c], a[c]);
        hi[c] = __fadd_rn(hi[c], b[c]);
      }
    }
    if (row < tu.i_valid && col < tu.j_valid) {
      u32x4 pk;
      pk[0] = pack_bf16x2(lo[0], lo[1]);
      pk[1] = pack_bf16x2(lo[2], lo[3]);
      pk[2] = pack_bf16x2(hi[0], hi[1]);
      pk[3] = pack_bf16x2(hi[2], hi[3]);
      *reinterpret_cast<u32x4*>(tu.out + (int64_t)row * tu.ldc + col) = pk;
    }
  }
}

// ---------------------------------------------------------------------------
// rows that belong to no group
// ---------------------------------------------------------------------------
// Writes zeros over rows t .. m_rows-1 of a [m_rows, row_bytes] output, where t
// is the last group end the GEMM kernels use: the maximum of the offsets
// clamped to [0, m_rows] (offs[E-1] itself for a valid array), found by each
// workgroup from the E offsets.  16 bytes per thread and iteration over a
// grid-stride loop; with no such rows every workgroup exits after the offsets.
__global__ __launch_bounds__(kThreads) void zero_rows_kernel(uint8_t* out, const int32_t* offs, int num_groups,
                                                             int64_t m_rows, int64_t row_bytes) {
  __shared__ int s_max[kThreads / 64];
  const int M = (int)m_rows;
  int v = 0;
  for (int e = threadIdx.x; e < num_groups; e += kThreads) v = max(v, min(max(offs[e], 0), M));
  v = wave_incl_max(v);
  if ((threadIdx.x & 63) == 63) s_max[threadIdx.x >> 6] = v;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) t = max(t, s_max[i]);
  const int64_t begin = (int64_t)t * row_bytes / 16, end = m_rows * row_bytes / 16;
  u32x4* dst = reinterpret_cast<u32x4*>(out);
  const u32x4 z = {0u, 0u, 0u, 0u};
  for (int64_t i = begin + (int64_t)blockIdx.x * kThreads + threadIdx.x; i < end;
       i += (int64_t)gridDim.x * kThreads)
    dst[i] = z;
}

}  // namespace

namespace {
constexpr int kMaxDevices = 64;
std::once_flag g_scratch_once[kMaxDevices];
void* g_scratch_ptr[kMaxDevices];
hipError_t g_scratch_err[kMaxDevices];
}  // namespace

hipError_t fwd_scratch_address(int device, void** ptr) {
  if (device < 0 || device >= kMaxDevices) return hipErrorInvalidDevice;
  std::call_once(g_scratch_once[device], [device]() {
    void* p = nullptr;
    g_scratch_err[device] = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    g_scratch_ptr[device] = p;
  });
  if (g_scratch_err[device] != hipSuccess) return g_scratch_err[device];
  if (g_scratch_ptr[device] == nullptr || (reinterpret_cast<uintptr_t>(g_scratch_ptr[device]) & 255u) != 0)
    return hipErrorInvalidSymbol;
  *ptr = g_scratch_ptr[device];
  return hipSuccess;
}

hipError_t launch_gemm(Op op, const GemmParams& p, int grid, hipStream_t stream) {
  const dim3 g(grid), blk(kThreads);
  switch (op) {
    case kFwd: {  // the reduction is k
      // paired stages when the experts average at least kPairRows rows (W reused
      // from the L2 by several row tiles); measured as the better schedule there
      const bool pairs = p.m_rows >= (int64_t)kPairRows * p.num_groups;
      if (p.k % kTileR == 0) {
        if (pairs) hipLaunchKernelGGL((grouped_gemm_kernel<kFwd, kStoreBf16, false, true>), g, blk, 0, stream, p);
        else hipLaunchKernelGGL((grouped_gemm_kernel<kFwd, kStoreBf16, false, false>), g, blk, 0, stream, p);
      } else {
        if (pairs) hipLaunchKernelGGL((grouped_gemm_kernel<kFwd, kStoreBf16, true, true>), g, blk, 0, stream, p);
        else hipLaunchKernelGGL((grouped_gemm_kernel<kFwd, kStoreBf16, true, false>), g, blk, 0, stream, p);
      }
      break;
    }
    case kDgrad:  // the reduction is n
      if (p.n % kTileR == 0) hipLaunchKernelGGL((grouped_gemm_kernel<kDgrad, kStoreBf16, false, true>), g, blk, 0, stream, p);
      else hipLaunchKernelGGL((grouped_gemm_kernel<kDgrad, kStoreBf16, true, true>), g, blk, 0, stream, p);
      break;
    case kWgrad:
      if (!p.out_fp32 && !p.accumulate)
        hipLaunchKernelGGL((grouped_gemm_kernel<kWgrad, kStoreBf16, false, false>), g, blk, 0, stream, p);
      else if (!p.out_fp32)
        hipLaunchKernelGGL((grouped_gemm_kernel<kWgrad, kStoreBf16Acc, false, false>), g, blk, 0, stream, p);
      else if (!p.accumulate)
        hipLaunchKernelGGL((grouped_gemm_kernel<kWgrad, kStoreF32, false, false>), g, blk, 0, stream, p);
      else
        hipLaunchKernelGGL((grouped_gemm_kernel<kWgrad, kStoreF32Acc, false, false>), g, blk, 0, stream, p);
      break;
  }
  return hipGetLastError();
}

hipError_t launch_zero_rows(void* out, const int32_t* offs, int num_groups, int64_t m_rows, int64_t row_bytes,
                            int grid, hipStream_t stream) {
  hipLaunchKernelGGL(zero_rows_kernel, dim3(grid), dim3(kThreads), 0, stream, static_cast<uint8_t*>(out), offs,
                     num_groups, m_rows, row_bytes);
  return hipGetLastError();
}

hipError_t launch_tail_reduce(const GemmParams& p, int grid_x, int grid_y, hipStream_t stream) {
  hipLaunchKernelGGL(tail_reduce_kernel, dim3(grid_x, grid_y), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_wgrad_reduce(const GemmParams& p, int grid_x, int grid_y, hipStream_t stream) {
  hipLaunchKernelGGL(wgrad_reduce_kernel, dim3(grid_x, grid_y), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace mdg
