// gfx950 (CDNA4) kernels of the experts' gated feed-forward.
//
//   fwd    a = x W_gate^T, b = x W_up^T, h = a s(q(a)) b    (s the logistic function)
//   dgrad  dh = dY W_down, da = dh b (s + a s (1 - s) q'(a)), db = dh a s
//
// with q(a) = a (SiLU) or 2 sqrt(2/pi) (a + 0.044715 a^3) (the tanh form of GELU, as
// 1 + tanh(v) = 2 s(2 v)).  Both are the tile products of tile_pipe.h with another
// epilogue:
//
//  * fwd: a tile is 256 rows by 128 hidden columns.  Its 256 columns of operand B
//    alternate, 16 rows of W_gate and the 16 rows of W_up of the same hidden columns,
//    so that a lane's accumulators hold a and b of the same values and h is formed in
//    registers, from the fp32 sums, rounded once.  Neither projection goes to memory
//    unless the caller keeps them (bf16) for the gradient.
//  * dgrad: dh stays in fp32 accumulators; the epilogue reads a and b where they
//    lie and writes their gradients, so dh never goes to memory and no pass over
//    the hidden rows follows.
//
// The matrix pipe and the stages' loads bound both, as they bound the plain products: 16384
// rows over 8 groups of 2 x 14336 x 4096 take fwd 2.98 to 3.01 ms (1280 TFLOP/s; the plain product
// of the same size 3.08, its outputs twice as wide), 3.20 with the projections kept; dgrad 1.75 ms
// against 1.52 of the plain one, where a pass over the rows behind it (read dh, a and b, write
// both gradients) would take 0.48.  No products run beside an epilogue: dgrad's, 76 cycles a
// value of a wave for SiLU, is an eighth of its time.
//
// The order of every sum is fixed: results are bitwise reproducible.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gated.h"
#include "gated_act.h"
#include "grouped_gemm.h"
#include "kernel_common.h"
#include "tile_epilogue.h"
#include "tile_pipe.h"

namespace mdg {
namespace {

// ---------------------------------------------------------------------------
// one unit of work
// ---------------------------------------------------------------------------
struct GatedUnit {
  Unit u;
  int row0, f0, f_valid;  // first row, first hidden column, hidden columns
};

__device__ __forceinline__ GatedTail* gated_tail(const GemmParams& p) {
  return reinterpret_cast<GatedTail*>(reinterpret_cast<uint8_t*>(p.tail_head) + 256);
}

// Work item v of the plan: a whole unit, or a piece of a tail unit (tile_pipe.h's
// decode_item, for these kernels' operands and outputs).  `up`: in fwd, whether this
// wave loads W_up's rows of operand B.
template <int OP>
__device__ __forceinline__ GatedUnit decode_gated(const GatedParams& gp, const GroupTable& tb, const UnitShape& us,
                                                  int total, const Plan& pl, int v, int up) {
  const GemmParams& p = gp.g;
  GatedUnit y;
  Unit& x = y.u;
  x.valid = v < pl.items;
  if (!x.valid) return y;
  int u = v, t = 0, sp = 0;
  const bool piece = v >= pl.full;
  if (piece) {
    t = (v - pl.full) / pl.split;
    sp = v - pl.full - t * pl.split;
    u = pl.full + t;
  }
  const int e = uniform(find_group(tb.uprefix, p.num_groups, u));
  const int gs = uniform(e == 0 ? 0 : tb.end[e - 1]);
  const int gm = uniform(tb.end[e]) - gs;
  int rt, ct;
  panel_order(u - uniform(tb.uprefix[e]), (gm + kTileI - 1) / kTileI, us.n_j, 4, &rt, &ct);
  const int N = p.n, K = p.k;
  const uint8_t* A = reinterpret_cast<const uint8_t*>(p.a);
  const uint8_t* B = reinterpret_cast<const uint8_t*>(p.b);
  y.row0 = gs + rt * kTileI;
  x.i_valid = min(kTileI, gm - rt * kTileI);
  if (OP == kFwd) {
    y.f0 = ct * kGatedCols;
    y.f_valid = min(kGatedCols, gp.f - y.f0);
    x.a = Operand{A + (int64_t)y.row0 * K * 2, K * 2, x.i_valid * K * 2, K * 2};
    x.b = Operand{B + ((int64_t)e * N + (up ? gp.f : 0) + y.f0) * K * 2, K * 2, y.f_valid * K * 2, K * 2};
    x.nkr = (K + kTileR - 1) / kTileR;
  } else {
    y.f0 = ct * kTileJ;
    y.f_valid = min(kTileJ, gp.f - y.f0);
    x.a = Operand{A + (int64_t)y.row0 * N * 2, N * 2, x.i_valid * N * 2, N * 2};
    x.b = Operand{B + ((int64_t)e * N * K + y.f0) * 2, K * 2, N, y.f_valid * 2};
    x.nkr = (N + kTileR - 1) / kTileR;
  }
  x.nk = (x.nkr + 3) & ~3;
  x.out = nullptr;
  x.ldc = 0;
  x.j_valid = kTileJ;
  x.mode = kStoreBf16;
  if (piece) {
    if (sp == 0 && threadIdx.x == 0) gated_tail(p)[t] = GatedTail{y.row0, y.f0, x.i_valid, y.f_valid};
    const int g = x.nk / 4;
    const int g0 = sp * g / pl.split, g1 = (sp + 1) * g / pl.split;
    const int k0 = 4 * g0 * kTileR;
    x.nk = 4 * (g1 - g0);
    x.nkr = min(x.nk, x.nkr - 4 * g0);
    shift_rc(x.a, k0);
    if (OP == kFwd) shift_rc(x.b, k0);
    else shift_tc(x.b, k0);
    x.out = p.partial + (int64_t)(t * pl.split + sp) * (kTileI * kTileJ);
    x.ldc = kTileJ;
    x.i_valid = kTileI;
    x.mode = kStoreF32;
  }
  return y;
}

// ---------------------------------------------------------------------------
// epilogues
// ---------------------------------------------------------------------------
// fwd, a whole unit: h and, where the caller keeps them, the projections.  Column
// block jb of the wave's sub-tile is gate (jb even) or up (odd) of the 16 hidden
// columns 16 (jb / 2) .. of its 64.  The projections leave as bf16 rows of 64 gate and
// 64 up columns through the staging of tile_epilogue.h (32 rows at a time, 4 rows of
// 2 x 128 bytes a store); h as 64 rows of 128 bytes, 8 rows a store, 16-byte chunk c of
// row r at chunk c ^ (r / 2 % 8) (conflict-free both ways).  Returns the memory
// operations issued.  (KEEP is a template argument: a branch around the projections'
// slabs made the compiler spill 194 registers.)
template <bool KEEP, int ACT>
__device__ __forceinline__ int store_hidden(const Acc& acc, const GatedParams& gp, const GatedUnit& y, uint8_t* xb,
                                            int wi, int wj, int lane) {
  const int f = gp.f;
  if constexpr (KEEP) {
    const Staging x = staging(xb, lane, true);
    const int extent = (y.u.i_valid - 1) * f * 4 + f * 2 + y.f_valid * 2;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        gp.keep + (int64_t)y.row0 * 2 * f + y.f0, 0, uniform(extent), 0x00020000);
    const int col = wj * 64 + (lane & 7) * 8, row = wi * 128 + (lane >> 4);
    uint32_t base = (uint32_t)(row * f * 4 + ((lane & 8) ? f * 2 : 0) + col * 2);
    int left = col < y.f_valid ? y.u.i_valid - row : 0;
    opaque(base);
    opaque(left);
#pragma unroll
    for (int sb = 0; sb < 4; ++sb) {
      __builtin_amdgcn_sched_barrier(0);  // one slab at a time (bounds the registers in use)
#pragma unroll
      for (int bl = 0; bl < 2; ++bl)
#pragma unroll
        for (int jb = 0; jb < 8; ++jb) {
          const f32x4& a = acc[2 * sb + bl][jb];
          u32x2 pk;
          pk[0] = pack_bf16x2(acc_read(a[0]), acc_read(a[1]));
          pk[1] = pack_bf16x2(acc_read(a[2]), acc_read(a[3]));
          *reinterpret_cast<u32x2*>(x.w + bl * 4096 + (((8 * (jb & 1) + 2 * (jb >> 1)) ^ x.kw) << 4)) = pk;
        }
      u32x4 v[8];
      unstage_slab(v, x);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int r = sb * 32 + q * 4;
        __builtin_amdgcn_raw_buffer_store_b128(v[q], rs, r < left ? base + (uint32_t)(r * f * 4) : kOutOfRange, 0, 0);
      }
    }
  }
  const int extent = (y.u.i_valid - 1) * f * 2 + y.f_valid * 2;
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
      static_cast<uint16_t*>(gp.g.out) + (int64_t)y.row0 * f + y.f0, 0, uniform(extent), 0x00020000);
  const int col = wj * 64 + (lane & 7) * 8, row = wi * 128 + (lane >> 3);
  uint32_t base = (uint32_t)(row * f * 2 + col * 2);
  int left = col < y.f_valid ? y.u.i_valid - row : 0;
  // this lane's writes: row l % 16 of a block, 4 columns at byte 32 q + 8 (l / 16)
  int wo = (lane & 15) * 128 + ((lane >> 4) & 1) * 8, kw = ((lane & 15) >> 1) ^ (lane >> 5);
  int ro = (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 4)) << 4);
  opaque(base);
  opaque(left);
  opaque(wo);
  opaque(kw);
  opaque(ro);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 &a = acc[4 * half + ib][2 * q], &b = acc[4 * half + ib][2 * q + 1];
        u32x2 pk;
        pk[0] = pack_bf16x2(Act<ACT>::hidden(acc_read(a[0]), acc_read(b[0])), Act<ACT>::hidden(acc_read(a[1]), acc_read(b[1])));
        pk[1] = pack_bf16x2(Act<ACT>::hidden(acc_read(a[2]), acc_read(b[2])), Act<ACT>::hidden(acc_read(a[3]), acc_read(b[3])));
        *reinterpret_cast<u32x2*>(xb + wo + ib * 2048 + (((2 * q) ^ kw) << 4)) = pk;
      }
    }
    u32x4 v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)  // row 8 q + l / 8, whose swizzle is 4 (q % 2) + l / 16
      v[q] = *reinterpret_cast<const u32x4*>(xb + (ro ^ ((q & 1) << 6)) + q * 1024);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int r = half * 64 + q * 8;
      __builtin_amdgcn_raw_buffer_store_b128(v[q], rs, r < left ? base + (uint32_t)(r * f * 2) : kOutOfRange, 0, 0);
    }
  }
  return KEEP ? 48 : 16;
}

// dgrad, a whole unit: half slabs of 32 rows x 64 columns of dh pass through the
// fp32 staging, from which a lane takes 8 consecutive columns (two 16-byte chunks) of
// rows 8 q + l / 8; a and b of those are read, and their gradients written, 16 bytes
// each.  The next half slab's a and b load while one is worked on.
template <int ACT>
__device__ __forceinline__ int store_grads(const Acc& acc, const GatedParams& gp, const GatedUnit& y, uint8_t* xb,
                                           int wi, int wj, int lane) {
  const int f = gp.f;
  const Staging x = staging(xb, lane, false);
  const int extent = uniform((y.u.i_valid - 1) * f * 4 + f * 2 + y.f_valid * 2);
  const int64_t at = (int64_t)y.row0 * 2 * f + y.f0;
  const __amdgpu_buffer_rsrc_t in =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(gp.gate_up) + at, 0, extent, 0x00020000);
  const __amdgpu_buffer_rsrc_t out =
      __builtin_amdgcn_make_buffer_rsrc(static_cast<uint16_t*>(gp.g.out) + at, 0, extent, 0x00020000);
  const int row = wi * 128 + (lane >> 3), col = wj * 128 + (lane & 7) * 8;
  uint32_t base0 = (uint32_t)(row * f * 4 + col * 2), base1 = base0 + 128;
  int left0 = col < y.f_valid ? y.u.i_valid - row : 0, left1 = col + 64 < y.f_valid ? y.u.i_valid - row : 0;
  int c0 = (lane & 7) * 2, r0 = lane >> 3;
  opaque(base0);
  opaque(base1);
  opaque(left0);
  opaque(left1);
  opaque(c0);
  opaque(r0);
  const auto offset = [&](int hs, int q) -> uint32_t {
    const int r = (hs >> 1) * 32 + q * 8;
    return r < ((hs & 1) ? left1 : left0) ? ((hs & 1) ? base1 : base0) + (uint32_t)(r * f * 4) : kOutOfRange;
  };
  u32x4 a[2][4], b[2][4];
  const auto load = [&](int hs) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t o = offset(hs, q);
      a[hs & 1][q] = __builtin_amdgcn_raw_buffer_load_b128(in, o, 0, 0);
      b[hs & 1][q] = __builtin_amdgcn_raw_buffer_load_b128(in, o, f * 2, 0);
    }
  };
  load(0);
#pragma unroll
  for (int hs = 0; hs < 8; ++hs) {
    __builtin_amdgcn_sched_barrier(0);  // one half slab at a time (bounds the registers in use)
    if (hs + 1 < 8) load(hs + 1);
    stage_slab<kStoreF32>(acc, x, hs >> 1, hs & 1);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = 8 * q + r0;
      const f32x4 lo = *reinterpret_cast<const f32x4*>(xb + r * 256 + ((c0 ^ (r & 15)) << 4));
      const f32x4 hi = *reinterpret_cast<const f32x4*>(xb + r * 256 + (((c0 + 1) ^ (r & 15)) << 4));
      u32x4 da, db;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t av = a[hs & 1][q][c], bv = b[hs & 1][q][c];
        float p0, p1, g0, g1;
        Act<ACT>::grads(lo_f(av), lo_f(bv), c < 2 ? lo[2 * c] : hi[2 * c - 4], &p0, &g0);
        Act<ACT>::grads(hi_f(av), hi_f(bv), c < 2 ? lo[2 * c + 1] : hi[2 * c - 3], &p1, &g1);
        da[c] = pack_bf16x2(p0, p1);
        db[c] = pack_bf16x2(g0, g1);
      }
      const uint32_t o = offset(hs, q);
      __builtin_amdgcn_raw_buffer_store_b128(da, out, o, 0, 0);
      __builtin_amdgcn_raw_buffer_store_b128(db, out, o, f * 2, 0);
    }
  }
  return 128;
}

template <int OP, bool KEEP, int ACT>
__device__ __forceinline__ int gated_epilogue(const Acc& acc, const GatedParams& p, const GatedUnit& y, uint8_t* xb,
                                              int wi, int wj, int lane) {
  if (y.u.mode == kStoreF32) {  // a piece of a split tail unit: fp32 partial tile
    const OutTile ot = out_tile(y.u.out, kTileJ, kTileI, kTileJ, wi, wj, lane, 4);
    epilogue_store<kStoreF32>(acc, ot, xb, lane);
    return epilogue_ops<kStoreF32>();
  }
  if constexpr (OP == kFwd) return store_hidden<KEEP, ACT>(acc, p, y, xb, wi, wj, lane);
  else return store_grads<ACT>(acc, p, y, xb, wi, wj, lane);
}

// ---------------------------------------------------------------------------
// the tile kernel
// ---------------------------------------------------------------------------
// The persistent walk of grouped_gemm_kernels.hip's products (the same steps, stage
// waits and staging buffers), with the units and epilogues above.  (The walk of a unit's
// stages stands in both: as a function of tile_pipe.h it made the compiler schedule
// the other kernels anew.)
// KEEP: fwd keeps the projections.
template <int OP, bool KEEP, int ACT, bool MASK, bool PAIRS>
__global__ __launch_bounds__(kThreads, 1) void gated_kernel(GatedParams gp) {
  using Pp = Pipe<OP, MASK, PAIRS>;
  __shared__ int s_end[kMaxGroups];
  __shared__ int s_uprefix[kMaxGroups + 1];
  __shared__ int s_sprefix[kMaxGroups];
  __shared__ int s_scratch[4];
  const GemmParams& p = gp.g;

  GroupTable tb{s_end, s_uprefix, s_sprefix, s_scratch};
  const int total = uniform(build_group_table<OP>(p, tb));
  const UnitShape us = unit_shape<OP>(p);
  const Plan pl = make_plan<OP>(p, total);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.tail_head[0] = pl.tail;  // read by the reduce kernel
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
  dma_offsets<false>(pipe.off_a, (OP == kFwd ? p.k : p.n) * 2, pipe.w, pipe.lane);
  dma_offsets<OP == kDgrad>(pipe.off_b, p.k * 2, pipe.w, pipe.lane);
  // fwd: the 16 LDS segments of operand B (16 tile columns each) are gate and up in
  // turn, and wave w fills segments 4 q + w, so its rows are all W_gate's (w even) or all
  // W_up's: 16 (2 q + w / 2) .. of the tile's 128
  const int up = pipe.w & 1;
  if constexpr (OP == kFwd) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int row = (2 * q + (pipe.w >> 1)) * 16 + (pipe.lane >> 2);
      pipe.off_b[q] = (uint32_t)(row * p.k * 2 + ((pipe.lane & 3) ^ swz_rc(pipe.lane >> 2)) * 16);
    }
  }
  if constexpr (MASK) {
    dma_chunks_rc(pipe.cb_a, pipe.w, pipe.lane);
    dma_chunks_rc(pipe.cb_b, pipe.w, pipe.lane);
  }

  GatedUnit cur = decode_gated<OP>(gp, tb, us, total, pl, vb, up);
  if (cur.u.valid) pipe.prefetch_first(cur.u);
  int tail = 0;  // memory operations issued between stage 2 and stage 3's operand A of the current unit
  for (int u = vb; cur.u.valid; u += P) {
    Acc acc;
    const Unit& x = cur.u;
    pipe.issue_last(x);
    zero(acc);
    {
      bf16x8 fbA[8], fbB[8], fal[4], fah[4];
      int e1 = tail, e2 = 0;
      wait_vm(Pp::kAfterStage0 + tail);  // stage 0 (kPairs: stages 0, 1) has landed
      lds_barrier();                     // ... in every wave
      pipe.first_frags(fbA, fal);
      const int nkr = x.nkr;
      pipe.template step<0, true>(acc, fbA, fbB, fal, fah, x, 0, e1, e2);
      pipe.template step<1, true>(acc, fbB, fbA, fal, fah, x, 1, e1, e2);
      pipe.template step<2, true>(acc, fbA, fbB, fal, fah, x, 2, e1, e2);
      pipe.template step<3, true>(acc, fbB, fbA, fal, fah, x, 3, e1, e2);
      int kt = 4;
      for (; kt + 4 <= nkr; kt += 4) {
        pipe.template step<0, false>(acc, fbA, fbB, fal, fah, x, kt, e1, e2);
        pipe.template step<1, false>(acc, fbB, fbA, fal, fah, x, kt + 1, e1, e2);
        pipe.template step<2, false>(acc, fbA, fbB, fal, fah, x, kt + 2, e1, e2);
        pipe.template step<3, false>(acc, fbB, fbA, fal, fah, x, kt + 3, e1, e2);
      }
      if (kt < nkr) {
        pipe.template step<0, false>(acc, fbA, fbB, fal, fah, x, kt, e1, e2);
        if (kt + 1 < nkr) pipe.template step<1, false>(acc, fbB, fbA, fal, fah, x, kt + 1, e1, e2);
        if (kt + 2 < nkr) pipe.template step<2, false>(acc, fbA, fbB, fal, fah, x, kt + 2, e1, e2);
      }
    }
    wait_vm_lgkm<0>();
    __syncthreads();  // every wave is done reading LDS before the next unit's loads

    const GatedUnit nxt = decode_gated<OP>(gp, tb, us, total, pl, u + P, up);
    if (nxt.u.valid) pipe.prefetch_first(nxt.u);
    const int ln = lane_here();
    // (each branch names its staging array, so that the compiler can tell its
    // accesses from the loads landing in the others)
    if (pipe.w < 2) tail = gated_epilogue<OP, KEEP, ACT>(acc, gp, cur, s_a3 + (pipe.w & 1) * 8192, pipe.wi, pipe.wj, ln);
    else tail = gated_epilogue<OP, KEEP, ACT>(acc, gp, cur, s_b3 + (pipe.w & 1) * 8192, pipe.wi, pipe.wj, ln);
    wait_vm_lgkm<63>();  // the staging reads have returned ...
    lds_barrier();       // ... in every wave
    cur = nxt;
  }
  wait_vm_lgkm<0>();
}

// ---------------------------------------------------------------------------
// the tail pieces' sums
// ---------------------------------------------------------------------------
__device__ __forceinline__ void add8(f32x4 (&s)[2], const float* q) {
  const f32x4 lo = reinterpret_cast<const f32x4*>(q)[0], hi = reinterpret_cast<const f32x4*>(q)[1];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    s[0][c] = __fadd_rn(s[0][c], lo[c]);
    s[1][c] = __fadd_rn(s[1][c], hi[c]);
  }
}
__device__ __forceinline__ u32x4 pack8(const f32x4 (&s)[2]) {
  u32x4 v;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    v[2 * c] = pack_bf16x2(s[c][0], s[c][1]);
    v[2 * c + 1] = pack_bf16x2(s[c][2], s[c][3]);
  }
  return v;
}

// blockIdx.y picks the tail unit, blockIdx.x a set of rows of its tile; a thread adds 8
// consecutive hidden columns (fwd: of gate and up) of a row over the pieces in range
// order and runs what the tile kernel's epilogue runs.
template <int OP, int ACT>
__global__ __launch_bounds__(kThreads) void gated_reduce_kernel(GatedParams gp) {
  const GemmParams& p = gp.g;
  const int T = uniform(p.tail_head[0]), S = uniform(p.tail_head[1]), t = blockIdx.y;
  if (t >= T || S < 2) return;
  constexpr int kLanes = (OP == kFwd ? kGatedCols : kTileJ) / 8;  // threads of a row
  const GatedTail tu = gated_tail(p)[t];
  const int f = gp.f, j = (threadIdx.x % kLanes) * 8;
  // fwd: hidden column j of the tile is gate column 128 (j / 64) + 32 (j / 16 % 4) + j % 16, and up 16 further
  const int col = OP == kFwd ? (j >> 6) * 128 + ((j >> 4) & 3) * 32 + (j & 15) : j;
  for (int row = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes; row < kTileI;
       row += gridDim.x * (kThreads / kLanes)) {
    if (row >= tu.i_valid || j >= tu.f_valid) continue;
    const float* q = p.partial + (int64_t)t * S * (kTileI * kTileJ) + row * kTileJ + col;
    f32x4 a[2] = {reinterpret_cast<const f32x4*>(q)[0], reinterpret_cast<const f32x4*>(q)[1]}, b[2];
    if constexpr (OP == kFwd) {
      b[0] = reinterpret_cast<const f32x4*>(q + 16)[0];
      b[1] = reinterpret_cast<const f32x4*>(q + 16)[1];
    }
    for (int s = 1; s < S; ++s) {
      add8(a, q + (int64_t)s * (kTileI * kTileJ));
      if constexpr (OP == kFwd) add8(b, q + (int64_t)s * (kTileI * kTileJ) + 16);
    }
    const int64_t r = tu.row0 + row;
    if constexpr (OP == kFwd) {
      if (gp.keep != nullptr) {
        *reinterpret_cast<u32x4*>(gp.keep + r * 2 * f + tu.f0 + j) = pack8(a);
        *reinterpret_cast<u32x4*>(gp.keep + r * 2 * f + f + tu.f0 + j) = pack8(b);
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) a[c >> 2][c & 3] = Act<ACT>::hidden(a[c >> 2][c & 3], b[c >> 2][c & 3]);
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.out) + r * f + tu.f0 + j) = pack8(a);
    } else {
      const int64_t at = r * 2 * f + tu.f0 + j;
      const u32x4 av = *reinterpret_cast<const u32x4*>(gp.gate_up + at);
      const u32x4 bv = *reinterpret_cast<const u32x4*>(gp.gate_up + at + f);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float x = (c & 1) ? hi_f(av[c >> 1]) : lo_f(av[c >> 1]), y = (c & 1) ? hi_f(bv[c >> 1]) : lo_f(bv[c >> 1]);
        float da, db;
        Act<ACT>::grads(x, y, a[c >> 2][c & 3], &da, &db);
        a[c >> 2][c & 3] = da;
        b[c >> 2][c & 3] = db;
      }
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.out) + at) = pack8(a);
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.out) + at + f) = pack8(b);
    }
  }
}

}  // namespace

// Stages in pairs (tile_pipe.h), in us without / with: where experts average 1024 rows or
// more (8 of 2 x 4096 x 4096, 8192 rows 497 / 481; 16 of 2 x 2048 x 6144, 16384 rows 752 /
// 740; 32 of them 867 / 897; 64 of 2 x 1536 x 2048, 16384 rows 316 / 323), and where rows of k
// end inside a stage, which start inside cache lines that the two halves of a pair share (8 of 2 x
// 4096 x 4104, 8192 rows 654 / 618; 64 of 2 x 1536 x 2056, 20000 rows 473 / 440; 4 of 2 x 2048 x
// 2056, 4096 rows 110 / 99).
constexpr int kGatedPairRows = 1024;

template <int ACT, bool KEEP>
static void launch_gated_fwd(const GatedParams& p, int grid, hipStream_t s) {
  const dim3 g(grid), b(kThreads);
  if (p.g.k % kTileR != 0)
    hipLaunchKernelGGL((gated_kernel<kFwd, KEEP, ACT, true, true>), g, b, 0, s, p);
  else if (p.g.m_rows >= (int64_t)kGatedPairRows * p.g.num_groups)
    hipLaunchKernelGGL((gated_kernel<kFwd, KEEP, ACT, false, true>), g, b, 0, s, p);
  else
    hipLaunchKernelGGL((gated_kernel<kFwd, KEEP, ACT, false, false>), g, b, 0, s, p);
}

template <int ACT>
static void launch_gated_act(Op op, const GatedParams& p, int grid, hipStream_t s) {
  const dim3 g(grid), b(kThreads);
  if (op == kFwd) p.keep ? launch_gated_fwd<ACT, true>(p, grid, s) : launch_gated_fwd<ACT, false>(p, grid, s);
  else if (p.g.n % kTileR == 0) hipLaunchKernelGGL((gated_kernel<kDgrad, false, ACT, false, true>), g, b, 0, s, p);
  else hipLaunchKernelGGL((gated_kernel<kDgrad, false, ACT, true, true>), g, b, 0, s, p);
}

hipError_t launch_gated(Op op, const GatedParams& p, int grid, hipStream_t s) {
  if (p.act == kActSilu) launch_gated_act<kActSilu>(op, p, grid, s);
  else launch_gated_act<kActGeluTanh>(op, p, grid, s);
  return hipGetLastError();
}

hipError_t launch_gated_reduce(Op op, const GatedParams& p, int grid_x, int grid_y, hipStream_t s) {
  const dim3 g(grid_x, grid_y), b(kThreads);
  const bool silu = p.act == kActSilu;
  if (op == kFwd && silu) hipLaunchKernelGGL((gated_reduce_kernel<kFwd, kActSilu>), g, b, 0, s, p);
  else if (op == kFwd) hipLaunchKernelGGL((gated_reduce_kernel<kFwd, kActGeluTanh>), g, b, 0, s, p);
  else if (silu) hipLaunchKernelGGL((gated_reduce_kernel<kDgrad, kActSilu>), g, b, 0, s, p);
  else hipLaunchKernelGGL((gated_reduce_kernel<kDgrad, kActGeluTanh>), g, b, 0, s, p);
  return hipGetLastError();
}

}  // namespace mdg
