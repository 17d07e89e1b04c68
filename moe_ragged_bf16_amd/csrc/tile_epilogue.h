// The epilogue of a 256 x 256 output tile held by 4 waves as 128 x 128 sub-tiles
// of 8 x 8 accumulator blocks: accumulators through LDS to whole row segments in
// memory.  Shared by the GEMM kernels; included by .hip files only.
#pragma once

#include "grouped_gemm.h"
#include "kernel_common.h"

namespace mdg {
namespace {

// A wave's accumulators: block [ib][jb] is rows 16 ib .. and columns 16 jb .. of
// its sub-tile; lane l holds row l % 16 and columns 4 (l / 16) .. + 3 of a block.
typedef f32x4 Acc[8][8];

__device__ __forceinline__ void zero(Acc& acc) {
#pragma unroll
  for (int ib = 0; ib < 8; ++ib)
#pragma unroll
    for (int jb = 0; jb < 8; ++jb)
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[ib][jb][x] = 0.0f;
}

// Epilogue store modes: plain stores, and the read-modify-write of an
// accumulating wgrad (fp32: RN32(out + dW); bf16: the bf16 dW added in bf16).
enum Store : int { kStoreBf16 = 0, kStoreF32 = 1, kStoreF32Acc = 2, kStoreBf16Acc = 3 };

constexpr bool is_bf16_mode(int mode) { return mode == kStoreBf16 || mode == kStoreBf16Acc; }

// The output tile of one unit as seen by one wave: rows i < i_valid and
// columns j < j_valid of the 256 x 256 tile at `out` (row stride ldc elements;
// j_valid is a multiple of 8, so each lane's 16 bytes are all valid or all not).  The epilogue passes the accumulators through
// LDS (a "staging" buffer of 8 KiB per wave) so that every global access covers
// whole 256-byte row segments: one load or store instruction moves 4 rows x 256
// bytes, 16 bytes per lane, where the MFMA layout itself (lane = row) would give
// 32 rows x 16 bytes.  All global accesses are buffer operations on one
// descriptor covering the tile's valid extent; masked lanes get an offset the
// range check turns away, so a wave always issues the same instructions.
struct OutTile {
  __amdgpu_buffer_rsrc_t rs;
  int ldc_b;
  int rows_left;   // i_valid minus this lane's first row (wi * 128 + lane / 16)
  uint32_t base0;  // byte offset of this lane's 16 bytes in its first row (kOutOfRange if the columns are invalid)
  uint32_t base1;  // the same 64 columns further (fp32 second half)
};

__device__ __forceinline__ OutTile out_tile(void* out, int64_t ldc, int i_valid, int j_valid, int wi, int wj,
                                            int lane, int esz) {
  OutTile t;
  t.ldc_b = (int)ldc * esz;
  const int extent = i_valid > 0 ? (i_valid - 1) * t.ldc_b + j_valid * esz : 0;
  t.rs = __builtin_amdgcn_make_buffer_rsrc(out, 0, extent, 0x00020000);
  const int row0 = wi * 128 + (lane >> 4);
  const int col0 = wj * 128 + (lane & 15) * (16 / esz);
  const uint32_t b = (uint32_t)(row0 * t.ldc_b + col0 * esz);
  t.base0 = col0 < j_valid ? b : kOutOfRange;
  t.base1 = col0 + 64 < j_valid ? b + 256 : kOutOfRange;
  t.rows_left = i_valid - row0;
  opaque(t.base0);
  opaque(t.base1);
  opaque(t.rows_left);
  return t;
}

// Global byte offset of read q (rows 4q .. 4q+3) of row slab ib, column half jh
// (fp32 only: the wave's second 64 columns).  An invalid base stays out of
// range after the row step (kOutOfRange + less than 2^31).
__device__ __forceinline__ uint32_t slab_off(const OutTile& t, int ib, int q, int jh) {
  const int r = ib * 32 + q * 4;
  const uint32_t b = jh ? t.base1 : t.base0;
  return r < t.rows_left ? b + (uint32_t)(r * t.ldc_b) : kOutOfRange;
}

// Staging layout: 32 rows of 256 bytes; 16-byte chunk c of row r at chunk
// c ^ (r % 16), so that both the writes (16 rows per instruction) and the reads
// (16 lanes per row) spread over all banks.  A lane writes row
// 16 (block % 2) + l % 16, whose swizzle is l % 16.
struct Staging {
  uint8_t* w;  // this lane's write row: xb + (lane % 16) * 256 (+ 8 for odd lane/16 in bf16)
  uint8_t* r;  // this lane's first read row: xb + (lane / 16) * 256
  int kw;      // chunk term of this lane's writes: (lane % 16) ^ (lane / 32) (bf16) or ^ (lane / 16) (fp32)
  int sw;      // lane % 16: the read chunk
  int rl;      // lane / 16: the read row within each group of 4
};

__device__ __forceinline__ Staging staging(uint8_t* xb, int lane, bool bf16) {
  Staging x;
  int wo = (lane & 15) * 256 + (bf16 ? ((lane >> 4) & 1) * 8 : 0);
  int ro = (lane >> 4) * 256;
  int kw = (lane & 15) ^ (bf16 ? (lane >> 5) : (lane >> 4));
  int sw = lane & 15, rl = lane >> 4;
  opaque(wo);
  opaque(ro);
  opaque(kw);
  opaque(sw);
  opaque(rl);
  x.w = xb + wo;
  x.r = xb + ro;
  x.kw = kw;
  x.sw = sw;
  x.rl = rl;
  return x;
}

// Writes row slab sb (rows 32 sb .. 32 sb + 31 of the wave's sub-tile: row
// blocks 2 sb, 2 sb + 1) to the staging buffer: bf16, all 128 columns (lane l
// writes 4 columns, 8 bytes at byte 32 jb + 8 (l / 16)); fp32, the 64 columns
// of half jh (16 bytes at byte 64 (jb - 4 jh) + 16 (l / 16)).
template <int mode>
__device__ __forceinline__ void stage_slab(const Acc& acc, const Staging& x, int sb, int jh) {
#pragma unroll
  for (int bl = 0; bl < 2; ++bl) {
    const int ib = 2 * sb + bl;
    if constexpr (mode == kStoreBf16) {
#pragma unroll
      for (int jb = 0; jb < 8; ++jb) {
        const f32x4& a = acc[ib][jb];
        u32x2 pk;
        pk[0] = pack_bf16x2(acc_read(a[0]), acc_read(a[1]));
        pk[1] = pack_bf16x2(acc_read(a[2]), acc_read(a[3]));
        *reinterpret_cast<u32x2*>(x.w + bl * 4096 + (((2 * jb) ^ x.kw) << 4)) = pk;
      }
    } else {
#pragma unroll
      for (int jl = 0; jl < 4; ++jl) {
        const f32x4& a = acc[ib][4 * jh + jl];
        const f32x4 v = {acc_read(a[0]), acc_read(a[1]), acc_read(a[2]), acc_read(a[3])};
        *reinterpret_cast<f32x4*>(x.w + bl * 4096 + (((4 * jl) ^ x.kw) << 4)) = v;
      }
    }
  }
}

// Reads the staged slab back row-major: read q gives this lane 16 bytes of row
// 4q + lane/16 (whose swizzle is (4q + lane/16) % 16).
__device__ __forceinline__ void unstage_slab(u32x4 (&v)[8], const Staging& x) {
#pragma unroll
  for (int q = 0; q < 8; ++q)
    v[q] = *reinterpret_cast<const u32x4*>(x.r + q * 1024 + ((x.sw ^ ((4 * q + x.rl) & 15)) << 4));
}

// Vector memory operations one wave issues in the epilogue of each mode.
template <int mode>
constexpr int epilogue_ops() {
  return mode == kStoreBf16 ? 32 : mode == kStoreF32 || mode == kStoreBf16Acc ? 64 : 128;
}

// Stores the wave's sub-tile (bf16 or fp32).
template <int mode>
__device__ __forceinline__ void epilogue_store(const Acc& acc, const OutTile& t, uint8_t* xb, int lane) {
  constexpr int kHalves = mode == kStoreBf16 ? 1 : 2;
  const Staging x = staging(xb, lane, mode == kStoreBf16);
#pragma unroll
  for (int ib = 0; ib < 4; ++ib)
#pragma unroll
    for (int jh = 0; jh < kHalves; ++jh) {
      __builtin_amdgcn_sched_barrier(0);  // one slab at a time (bounds the registers in use)
      stage_slab<mode>(acc, x, ib, jh);
      u32x4 v[8];
      unstage_slab(v, x);
#pragma unroll
      for (int q = 0; q < 8; ++q) __builtin_amdgcn_raw_buffer_store_b128(v[q], t.rs, slab_off(t, ib, q, jh), 0, 0);
    }
}

}  // namespace
}  // namespace mdg
