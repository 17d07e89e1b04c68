// gfx950 (CDNA4) kernels of the ragged grouped product in 8 bits: quantisation
// to e4m3 with one power-of-two scale (e8m0) for each block of 128, and
//   Y[s_e:t_e] = (q_x s_x)[s_e:t_e] @ ((q_w s_w)[e])^T
// with bf16 output.
//
// Scales.  Of a block with largest magnitude m the scale is the smallest 2^e with
// m <= 448 * 2^e (448 is e4m3's largest value), e >= -127; then q = e4m3(x 2^-e),
// rounded to nearest even.  Being a power of two costs nothing in precision (a
// floating-point q keeps its relative precision wherever in its range it lies)
// and makes x 2^-e exact, so q has one rounding; and the matrix instruction
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies by such scales itself, so the whole
// reduction stays in its accumulators.  A block that holds a NaN or an
// infinity gets scale NaN (code 255) and q NaN.
//
// Sums.  The instruction (the unscaled 8-bit one alike) adds 8 consecutive products
// aligned to their largest exponent sum E, each cut toward zero to a multiple of
// 2^(E - 13); what it adds above that is fp32.  No 8-bit instruction of gfx950 keeps
// more, and widening the operands to bf16 for one that does would halve the matrix
// rate.  The cut is up to 7 * 2^-13 * 2^E for 8 products; on normally distributed
// operands (3001 rows, 16 experts of 1000 x 2000) 1.8 % of the bf16 outputs differ by
// it from those of fp32 sums, and the outputs' error against 64 bits is the same
// (1.6580e-3 and 1.6578e-3 in the 2-norm).
// One instruction covers a reduction of 128: a block.  Its per-lane scale
// applies to the 32 reductions that lane holds, and all four lanes of a row
// carry the row's scale of the block.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8.h"
#include "grouped_gemm.h"
#include "kernel_common.h"
#include "tile_epilogue.h"

#include <type_traits>

namespace mdg {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// quantisation
// ---------------------------------------------------------------------------
// e8m0 code of a block from the bits of its largest magnitude (as an integer, NaN
// and infinity above every number): with m = 1.f 2^x, e = x - 8 if 1.f <= 1.75,
// else x - 7.
__device__ __forceinline__ uint32_t scale_code(uint32_t amax) {
  const int x = (int)(amax >> 23);
  if (x == 255) return 255u;
  return (uint32_t)max(x - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0), 0);
}

// The factor 2^-e of a scale code (NaN for code 255).
__device__ __forceinline__ float inverse_scale(uint32_t code) {
  return __uint_as_float(code == 255u ? 0x7fc00000u : (254u - code) << 23);
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

// 16 consecutive values at p (bf16 or fp32, 16-byte aligned), of which `left` (a
// multiple of 8) are there; zeros for the others.
template <bool FP32>
__device__ __forceinline__ void load16(float (&f)[16], const void* base, int64_t at, int left) {
  const bool whole = left >= 16;
  if constexpr (FP32) {
    const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 v = i < 2 || whole ? q[i] : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < 4; ++c) f[4 * i + c] = v[c];
    }
  } else {
    const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + at);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x4 v = i < 1 || whole ? q[i] : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        f[8 * i + 2 * c] = __uint_as_float(v[c] << 16);
        f[8 * i + 2 * c + 1] = __uint_as_float(v[c] & 0xffff0000u);
      }
    }
  }
}

__device__ __forceinline__ uint32_t magnitude(float f) { return __float_as_uint(f) & 0x7fffffffu; }

__device__ __forceinline__ u32x4 quantize16(const float (&f)[16], uint32_t code) {
  const float inv = inverse_scale(code);
  u32x4 q;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    q[c] = pack_e4m3(f[4 * c] * inv, f[4 * c + 1] * inv, f[4 * c + 2] * inv, f[4 * c + 3] * inv);
  return q;
}

// Rows: 8 lanes take a block, 16 values each; blocks are dealt in memory order.
// Memory bounds it: 16384 x 4096 bf16 take 34.5 us, 5.8 TB/s (a large copy: 4.9, a
// third of these bytes are writes).
template <bool FP32>
__global__ __launch_bounds__(256) void quantize_rows_kernel(Fp8RowsParams p) {
  const int l8 = threadIdx.x & 7;
  const int64_t total = p.m_rows * p.blocks;
  for (int64_t b = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3); b < total; b += (int64_t)gridDim.x * 32) {
    const int64_t row = b / p.blocks;
    const int kb = (int)(b - row * p.blocks);
    const int col = kb * kFp8Block + l8 * 16;
    float f[16];
    uint32_t m = 0;
    if (col < p.k) {
      load16<FP32>(f, p.x, row * p.k + col, p.k - col);
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max(m, magnitude(f[i]));
    }
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
    const uint32_t code = scale_code(m);
    if (col < p.k) *reinterpret_cast<u32x4*>(p.q + row * p.pitch + col) = quantize16(f, code);
    uint8_t* s = p.scale + ((int64_t)(kb >> 2) * p.m_rows + row) * 4;
    if (l8 == 0) s[kb & 3] = (uint8_t)code;
    if (kb == p.blocks - 1 && l8 > (kb & 3) && l8 < 4) s[l8] = 0;  // the last word's unused scales
  }
}

// Weights: a workgroup takes a 128 x 128 block; thread t rows t / 8 + 32 i, 16
// columns at 16 (t % 8).  The transposed copy is the same bytes through LDS.  Memory
// bounds it: 64 experts' 1536 x 2048 bf16 with the copy take 142 us, 5.7 TB/s.
template <bool FP32, bool TRANSPOSE>
__global__ __launch_bounds__(256) void quantize_weight_kernel(Fp8WeightParams p) {
  __shared__ uint32_t s_max[4];
  __shared__ __attribute__((aligned(16))) uint8_t s_q[TRANSPOSE ? 128 * 144 : 16];
  const int t = threadIdx.x;
  const int nb = (p.n + 127) / 128, kb = (p.k + 127) / 128;
  const int bk = (int)(blockIdx.x % kb);
  const int64_t rest = blockIdx.x / kb;
  const int bn = (int)(rest % nb);
  const int64_t e = rest / nb;
  const int col = bk * 128 + (t & 7) * 16;
  float f[4][16];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = bn * 128 + (t >> 3) + 32 * i;
#pragma unroll
    for (int c = 0; c < 16; ++c) f[i][c] = 0.0f;
    if (row < p.n && col < p.k) load16<FP32>(f[i], p.w, (e * p.n + row) * p.k + col, p.k - col);
#pragma unroll
    for (int c = 0; c < 16; ++c) m = max(m, magnitude(f[i][c]));
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
  if ((t & 63) == 0) s_max[t >> 6] = m;
  __syncthreads();
  const uint32_t code = scale_code(max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3])));
  if (t == 0) {
    p.scale[(e * nb + bn) * kb + bk] = (uint8_t)code;
    if constexpr (TRANSPOSE) p.scale_t[(e * kb + bk) * nb + bn] = (uint8_t)code;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (t >> 3) + 32 * i, row = bn * 128 + r;
    const u32x4 q = quantize16(f[i], code);
    if (row < p.n && col < p.k) *reinterpret_cast<u32x4*>(p.q + (e * p.n + row) * p.pitch + col) = q;
    if constexpr (TRANSPOSE) *reinterpret_cast<u32x4*>(s_q + r * 144 + (t & 7) * 16) = q;
  }
  if constexpr (TRANSPOSE) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = (t >> 3) + 32 * i, k = bk * 128 + c, n = bn * 128 + (t & 7) * 16;
      u32x4 q;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        uint32_t v = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) v |= (uint32_t)s_q[((t & 7) * 16 + 4 * d + b) * 144 + c] << (8 * b);
        q[d] = v;
      }
      if (k < p.k && n < p.n) *reinterpret_cast<u32x4*>(p.qt + (e * p.k + k) * p.pitch_t + n) = q;
    }
  }
}

// ---------------------------------------------------------------------------
// the tile kernel: 256 x 256 output tiles
// ---------------------------------------------------------------------------
constexpr int kOperandBytes = kTileI * kFp8Block;  // one operand, one stage: 32 KiB
constexpr int kLoads = kOperandBytes / 4 / 1024;   // DMA loads of an operand a wave makes per stage
static_assert(kTileI == kTileJ && kLoads == 8, "a stage of an operand is 32 segments of 1 KiB, 8 for each of 4 waves");

__shared__ __attribute__((aligned(1024))) uint8_t s_a0[kOperandBytes];
__shared__ __attribute__((aligned(1024))) uint8_t s_a1[kOperandBytes];
__shared__ __attribute__((aligned(1024))) uint8_t s_b0[kOperandBytes];
__shared__ __attribute__((aligned(1024))) uint8_t s_b1[kOperandBytes];
__shared__ __attribute__((aligned(1024))) uint8_t s_out[4][4096];  // each wave's results on their way out

template <int B>
__device__ __forceinline__ uint8_t* buf_a() {
  if constexpr (B == 0) return s_a0;
  else return s_a1;
}
template <int B>
__device__ __forceinline__ uint8_t* buf_b() {
  if constexpr (B == 0) return s_b0;
  else return s_b1;
}

// c += b^T a under the scales in byte S of sb and sa.  Written as asm so that the
// tile kernel's 256 accumulators stay in AGPRs, in place.  The compiler does not see
// that a source written by a vector instruction needs two wait states before its
// use here: operands come from LDS (which it waits for), and scales through
// settle().  Nor does it see when the result is there: settle_results().  The build
// checks the generated code for both.  (An s_nop in front of each product cost 2 %.)
#define MDG_MFMA(REGS, SEL)                                                                            \
  asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 " SEL : REGS(c) : "v"(b), "v"(a), \
               "v"(sb), "v"(sa))
#define MDG_MFMA_BYTE(REGS)                                              \
  if constexpr (S == 0) MDG_MFMA(REGS, "op_sel_hi:[0,0,0]");             \
  else if constexpr (S == 1) MDG_MFMA(REGS, "op_sel:[1,1,0] op_sel_hi:[0,0,0]"); \
  else if constexpr (S == 2) MDG_MFMA(REGS, "op_sel_hi:[1,1,0]");        \
  else MDG_MFMA(REGS, "op_sel:[1,1,0] op_sel_hi:[1,1,0]")
// The accumulator in AGPRs (the tile kernel, whose 256 would not fit else) or VGPRs.
template <int S>
__device__ __forceinline__ void mfma_scaled(f32x4& c, const i32x8& b, const i32x8& a, uint32_t sb, uint32_t sa) {
  MDG_MFMA_BYTE("+a");
}
template <int S>
__device__ __forceinline__ void mfma_scaled_v(f32x4& c, const i32x8& b, const i32x8& a, uint32_t sb, uint32_t sa) {
  MDG_MFMA_BYTE("+v");
}
#undef MDG_MFMA_BYTE
#undef MDG_MFMA

// The wait states between the moves of scales and the products that take them.
template <int N>
__device__ __forceinline__ void settle(uint32_t (&x)[N], uint32_t& w) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(x[i]));
  asm volatile("s_nop 1" : "+v"(w));
}

// The wait states between the last products and the first other access of their
// results (12 for this instruction; the compiler does not see the need around the asm
// statements, and left alone it moves the reads up to the products).  Results in
// VGPRs are tied to the place; those in AGPRs are read by statements that stay behind
// it anyway.  The build checks the generated code.
__device__ __forceinline__ void settle_results() { asm volatile("s_nop 15"); }
template <int I, int J>
__device__ __forceinline__ void settle_results(f32x4 (&acc)[I][J]) {
  settle_results();
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) asm volatile("" : "+v"(acc[i][j]));
}

// Waits until all of this wave's LDS reads have returned.
__device__ __forceinline__ void wait_lgkm() { __builtin_amdgcn_s_waitcnt(0xC07F); }  // lgkmcnt(0), the others at their most

// One unit: a row tile of one group times a tile of its expert's columns.
struct Fp8Unit {
  const uint8_t* a;  // x rows of the tile, column 0
  const uint8_t* b;  // w[e] rows n of the tile, column 0
  const uint8_t* sw; // scales of this wave's 128 columns, block 0
  int row0;          // first row of the tile
  int i_valid, j_valid, j0;
  bool valid;
};

struct Scales {
  uint32_t x[8];  // per row block of the wave: 4 blocks' scales of this lane's row
  uint32_t w;     // 4 blocks' scales of the wave's columns
};

// Stage layout in LDS: 256 rows of 128 bytes, 16-byte chunk c of row r at chunk
// c ^ (r % 8): the 8 lanes that an LDS read serves together lie in 8 rows, and
// so in 8 different chunks (all banks once).  A lane of an operand fragment
// holds chunks l / 16 and l / 16 + 4 of row l % 16 (both operands alike: the order
// of the reduction inside a block is free).
struct Fp8Pipe {
  uint32_t off;       // DMA: byte offset of this lane's chunk in its first row
  uint32_t chunk;     // ... its byte position within the stage
  int fa, fb;         // LDS offset of this lane's first chunk of block 0 of its wave's A and B rows
  int k, w, wi, wj, lane;

  __device__ __forceinline__ void init(int k_) {
    k = k_;
    lane = threadIdx.x & 63;
    w = uniform(threadIdx.x >> 6);
    wi = w >> 1;
    wj = w & 1;
    const int row = w * 8 + (lane >> 3);
    chunk = (uint32_t)(((lane & 7) ^ (lane >> 3)) * 16);
    off = (uint32_t)row * (uint32_t)k + chunk;
    const int r = lane & 15, c = ((lane >> 4) ^ (r & 7)) * 16;
    fa = (wi * 128 + r) * 128 + c;
    fb = (wj * 128 + r) * 128 + c;
  }

  __device__ __forceinline__ static i32x8 frag(const uint8_t* buf, int at, int block) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(buf + at + block * 2048);
    const i32x4 hi = *reinterpret_cast<const i32x4*>(buf + (at ^ 64) + block * 2048);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }

  // One stage of an operand: from `base`, `bytes` to the end of the tile's valid
  // rows (loads past it read zeros), `left` of them in the current row (chunks
  // past it, in the last stage, read zeros).
  struct Stage {
    __amdgpu_buffer_rsrc_t rs;
    uint32_t left;
  };
  __device__ __forceinline__ Stage stage(const uint8_t* base, int rows, int kt) const {
    const int left = k - kt * kFp8Block;
    const int bytes = uniform(left > 0 && rows > 0 ? rows * k - kt * kFp8Block : 0);
    return Stage{__builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base) + (left > 0 ? kt * kFp8Block : 0), 0,
                                                   bytes, 0x00020000),
                 (uint32_t)max(left, 0)};
  }
  // Load q of a stage.
  __device__ __forceinline__ void load(const Stage& st, uint8_t* buf, int q) const {
    const uint32_t at = chunk < st.left ? off + (uint32_t)(q * 32) * (uint32_t)k : kOutOfRange;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(st.rs, (lds_void*)(buf + (q * 4 + w) * 1024), 16, at, 0, 0, 0);
  }
  template <int B>
  __device__ __forceinline__ void load_stage(const Fp8Unit& u, int kt) const {
    const Stage a = stage(u.a, u.i_valid, kt), b = stage(u.b, u.j_valid, kt);
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      load(a, buf_a<B>(), q);
      load(b, buf_b<B>(), q);
    }
  }

  // The scales of blocks 4 g .. 4 g + 3.  (Lanes of rows past the matrix and
  // blocks past the last read zeros; their products are zeros or not stored.)
  __device__ __forceinline__ void load_scales(Scales& s, const Fp8GemmParams& p, const Fp8Unit& u, int g) const {
    const bool in = 4 * g < p.blocks;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint32_t*>(p.xs) + (in ? (int64_t)g * p.m_rows + u.row0 : 0), 0,
        uniform(in ? (int)(p.m_rows - u.row0) * 4 : 0), 0x00020000);
    const uint32_t at = (uint32_t)(wi * 128 + (lane & 15)) * 4;
#pragma unroll
    for (int ib = 0; ib < 8; ++ib) s.x[ib] = __builtin_amdgcn_raw_buffer_load_b32(rs, at + ib * 64, 0, 0);
    const __amdgpu_buffer_rsrc_t rw =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(u.sw), 0, uniform(p.blocks), 0x00020000);
    uint32_t v = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(rw, 4 * g + i, 0, 0) << (8 * i);
    s.w = v;
  }

  // Fragments of a unit's stage 0 (landed in buffer 0).
  __device__ __forceinline__ void first_frags(i32x8 (&al)[4], i32x8 (&ah)[4], i32x8 (&b)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      b[i] = frag(s_b0, fb, i);
      if (i < 4) al[i] = frag(s_a0, fa, i);
      else ah[i - 4] = frag(s_a0, fa, i);
    }
  }

  // Stage kt (S = kt % 4, buffer S % 2) in two halves of 32 products, row blocks
  // 0..3 (al) and 4..7 (ah).  On entry its fragments are in registers (the last of
  // them still on their way from LDS) and the loads of stage kt + 1 are in flight.
  //  * After the first products: this wave's LDS reads have returned; behind the
  //    barrier every wave's have, so buffer S % 2 is free, and the loads of stage
  //    kt + 2 go out to it over the next 44 products.  For a unit's last two stages
  //    these are the next unit's stages 0 and 1 (stage S % 2), so the loads never
  //    pause between units.
  //  * Half way: stage kt + 1 has landed, behind the barrier in
  //    every wave; the second half reads its fragments, each b into the registers
  //    of the one that has been used.
  // A stage's loads thus have 3/4 to 1 1/2 steps to land.
  template <int S>
  __device__ __forceinline__ void step(Acc& acc, i32x8 (&al)[4], const i32x8 (&ah)[4], i32x8 (&ahn)[4], i32x8 (&b)[8],
                                       const Scales& sc, Scales& sn, const Fp8GemmParams& p, const Fp8Unit& u,
                                       const Fp8Unit& nx, int kt) const {
    constexpr int B = S & 1, N = B ^ 1;
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) mfma_scaled<S>(acc[ib][0], b[0], al[ib], sc.w, sc.x[ib]);
    wait_lgkm();
    lds_barrier();
    if constexpr (S == 3) load_scales(sn, p, u, (kt >> 2) + 1);
    const bool in = kt + 2 < p.blocks;
    const Stage sa = stage(in ? u.a : nx.a, in ? u.i_valid : nx.i_valid, in ? kt + 2 : B);
    const Stage sb = stage(in ? u.b : nx.b, in ? u.j_valid : nx.j_valid, in ? kt + 2 : B);
    auto issue = [&](int i) {
      if (i & 1) load(sb, buf_b<B>(), i >> 1);
      else load(sa, buf_a<B>(), i >> 1);
    };
#pragma unroll
    for (int jb = 1; jb < 8; ++jb)
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) {
        mfma_scaled<S>(acc[ib][jb], b[jb], al[ib], sc.w, sc.x[ib]);
        const int m = (jb - 1) * 4 + ib;
        if (m * kFirstLoads / 28 < (m + 1) * kFirstLoads / 28) issue(m * kFirstLoads / 28);
      }
    // Stage kt + 1 has landed.  After it were issued this step's loads so far and,
    // in a unit's first step, the previous unit's 32 stores.
    if (S == 0 && kt == 0) wait_vm_lgkm<kFirstLoads + epilogue_ops<kStoreBf16>()>();
    else wait_vm_lgkm<kFirstLoads>();
    lds_barrier();
#pragma unroll
    for (int jb = 0; jb < 8; ++jb) {
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) {
        mfma_scaled<S>(acc[4 + ib][jb], b[jb], ah[ib], sc.w, sc.x[4 + ib]);
        if (jb < 4 && ib == 3) issue(kFirstLoads + jb);
        if (ib == 1 && jb < 4) al[jb] = frag(buf_a<N>(), fa, jb);
        if (ib == 1 && jb >= 4) ahn[jb - 4] = frag(buf_a<N>(), fa, jb);
      }
      b[jb] = frag(buf_b<N>(), fb, jb);
    }
  }
  // Loads of a step that go out in its first half; the other 4 follow in the second.
  // All 16 within 16 products stalled the products behind them (16384 rows, 8
  // experts of 14336 x 4096: 810 us; over the first half 776, so 758, 8 + 8 763).
  static constexpr int kFirstLoads = 2 * kLoads - 4;
};

// Writes the wave's 128 x 128 sub-tile as bf16, 16 rows at a time through 4 KiB of
// LDS of its own (layout as in stage_slab: 256-byte rows, chunk c of row r at
// c ^ (r % 16)), so that a store covers whole 256-byte row segments.
__device__ __forceinline__ void store_tile(const Acc& acc, const OutTile& t, uint8_t* xb, int lane) {
  const Staging x = staging(xb, lane, true);
#pragma unroll
  for (int ib = 0; ib < 8; ++ib) {
    __builtin_amdgcn_sched_barrier(0);  // one slab at a time (bounds the registers in use)
#pragma unroll
    for (int jb = 0; jb < 8; ++jb) {
      const f32x4& a = acc[ib][jb];
      u32x2 pk;
      pk[0] = pack_bf16x2(acc_read(a[0]), acc_read(a[1]));
      pk[1] = pack_bf16x2(acc_read(a[2]), acc_read(a[3]));
      *reinterpret_cast<u32x2*>(x.w + (((2 * jb) ^ x.kw) << 4)) = pk;
    }
    u32x4 v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      v[q] = *reinterpret_cast<const u32x4*>(x.r + q * 1024 + ((x.sw ^ ((4 * q + x.rl) & 15)) << 4));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = ib * 16 + q * 4;
      __builtin_amdgcn_raw_buffer_store_b128(v[q], t.rs, r < t.rows_left ? t.base0 + (uint32_t)(r * t.ldc_b) : kOutOfRange,
                                             0, 0);
    }
  }
}

// Thread t handles groups 4 t .. 4 t + 3: clamped ends and the prefix of units.
__device__ __forceinline__ int fp8_group_table(const Fp8GemmParams& p, int n_j, int* s_end, int* s_uprefix,
                                               int* scratch) {
  const int E = p.num_groups, M = (int)p.m_rows, t = threadIdx.x;
  int endv[4], run = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = 4 * t + q;
    if (e < E) run = max(run, min(max(p.offs[e], 0), M));
    endv[q] = run;
  }
  const int before = block_excl_max(run, scratch);
  int units[4], sum = 0, start = before;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int end = max(before, endv[q]);
    const int rows = end - start;
    units[q] = 4 * t + q < E ? (rows + kTileI - 1) / kTileI * n_j : 0;
    if (4 * t + q < E) s_end[4 * t + q] = end;
    sum += units[q];
    start = end;
  }
  int total;
  int at = block_excl_sum(sum, scratch, &total);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (4 * t + q < E) s_uprefix[4 * t + q] = at;
    at += units[q];
  }
  if (t == 0) s_uprefix[E] = total;
  __syncthreads();
  return total;
}

// Unit v of the launch; one past the last has no rows and loads nothing.
__device__ __forceinline__ Fp8Unit fp8_unit(const Fp8GemmParams& p, const int* s_end, const int* s_uprefix, int n_j,
                                            int total, int v, int wj) {
  Fp8Unit u{p.x, p.w, p.ws, 0, 0, 0, 0, v < total};
  if (!u.valid) return u;
  const int e = uniform(find_group(s_uprefix, p.num_groups, v));
  const int gs = uniform(e == 0 ? 0 : s_end[e - 1]);
  const int gm = uniform(s_end[e]) - gs;
  int rt, ct;
  panel_order(v - uniform(s_uprefix[e]), (gm + kTileI - 1) / kTileI, n_j, 4, &rt, &ct);
  u.row0 = gs + rt * kTileI;
  u.i_valid = min(kTileI, gm - rt * kTileI);
  u.j0 = ct * kTileJ;
  u.j_valid = min(kTileJ, p.n - u.j0);
  u.a = p.x + (int64_t)u.row0 * p.k;
  u.b = p.w + ((int64_t)e * p.n + u.j0) * p.k;
  const int nb = (p.n + kFp8Block - 1) / kFp8Block;
  u.sw = p.ws + ((int64_t)e * nb + min(u.j0 / kFp8Block + wj, nb - 1)) * p.blocks;
  return u;
}

// A persistent grid of workgroups that walk the units.  A unit's stages 0 and 1
// and the first fragments are loaded during the previous unit's last steps (see
// Fp8Pipe::step) and its results leave by stores nothing waits for until two
// steps into the next unit.
//
// 16384 rows over 8 experts' 14336 x 4096 take 738 us, 2.61 PFLOP/s (the library's
// largest 8-bit products here reach 3.1), 32768 over 64 experts' 1536 x 2048 116 us:
// 1.78 PFLOP/s of the rows' own products, 2.2 with those of partly filled tiles.
// What bounds it: a step's matrix work is 2048 cycles and it takes about 2900 (the
// counters have the matrix pipe busy 71 % of the cycles in the first, 50 % in the
// second, whose units have 12 or 16 steps).  In copies of the kernel, with
// its loads left out the first took 15 % less, with loads that always hit the L2 7 %,
// with the fragments' LDS reads left out 2 %, with all data zero (the clock then
// holds; the card's power limits it otherwise, to about 1.9 of 2.4 GHz) 13 %.
// Results that left between the products of the steps around a unit's end, rather
// than behind its last one, gained nothing; tails of up to 128 rows given to the
// middle kernel lost 3 to 5 % (their weights are read once more), and so did a half
// tile for them here.
__global__ __launch_bounds__(kThreads, 1) void fp8_gemm_kernel(Fp8GemmParams p) {
  __shared__ int s_end[kMaxGroups];
  __shared__ int s_uprefix[kMaxGroups + 1];
  __shared__ int s_scratch[4];
  const int n_j = (p.n + kTileJ - 1) / kTileJ;
  const int total = uniform(fp8_group_table(p, n_j, s_end, s_uprefix, s_scratch));
  const int P = gridDim.x, bid = blockIdx.x;
  const int vb = (P % 8 == 0) ? (bid % 8) * (P / 8) + bid / 8 : bid;
  Fp8Pipe pipe;
  pipe.init(p.k);
  const int nk = p.blocks;
  Fp8Unit u = fp8_unit(p, s_end, s_uprefix, n_j, total, vb, pipe.wj);
  if (!u.valid) return;
  i32x8 al[4], ah[4], ahn[4], b[8];
  Scales sc, sn;
  pipe.load_scales(sc, p, u, 0);
  pipe.load_stage<0>(u, 0);
  pipe.load_stage<1>(u, 1);
  wait_vm_lgkm<0>();
  lds_barrier();
  pipe.first_frags(al, ah, b);
  for (int v = vb; u.valid; v += P) {
    const Fp8Unit nx = fp8_unit(p, s_end, s_uprefix, n_j, total, v + P, pipe.wj);
    Acc acc;
    zero(acc);
    settle(sc.x, sc.w);
    int kt = 0;
    for (; kt + 4 <= nk; kt += 4) {
      pipe.step<0>(acc, al, ah, ahn, b, sc, sn, p, u, nx, kt);
      pipe.step<1>(acc, al, ahn, ah, b, sc, sn, p, u, nx, kt + 1);
      pipe.step<2>(acc, al, ah, ahn, b, sc, sn, p, u, nx, kt + 2);
      pipe.step<3>(acc, al, ahn, ah, b, sc, sn, p, u, nx, kt + 3);
      sc = sn;
      settle(sc.x, sc.w);
    }
    if (kt < nk) {
      pipe.step<0>(acc, al, ah, ahn, b, sc, sn, p, u, nx, kt);
      if (kt + 1 < nk) pipe.step<1>(acc, al, ahn, ah, b, sc, sn, p, u, nx, kt + 1);
      if (kt + 2 < nk) pipe.step<2>(acc, al, ah, ahn, b, sc, sn, p, u, nx, kt + 2);
    }
    if (nk == 1) {  // no second step has loaded the next unit's stage 1
      wait_vm_lgkm<0>();
      lds_barrier();
      pipe.load_stage<1>(nx, 1);
    }
    pipe.load_scales(sc, p, nx, 0);
    const int ln = lane_here();
    const OutTile ot = out_tile(p.y + (int64_t)u.row0 * p.n + u.j0, p.n, u.i_valid, u.j_valid, pipe.wi, pipe.wj, ln, 2);
    settle_results();
    store_tile(acc, ot, s_out[pipe.w], ln);
    if (nk & 1) {
      // the last step's fragments came from buffer 1; the next unit's stage 0 is in
      // buffer 0, loaded before the 32 stores
      wait_vm_lgkm<epilogue_ops<kStoreBf16>()>();
      lds_barrier();
      pipe.first_frags(al, ah, b);
    }
    u = nx;
  }
  wait_vm_lgkm<0>();
}

// ---------------------------------------------------------------------------
// the small kernel: few rows to a group
// ---------------------------------------------------------------------------
// With few rows a product is the reading of its weights.  A workgroup takes 32
// columns (rows of w[e]) and up to kFp8SmallRows rows of one group; its waves
// share the reduction out in pieces of 4 blocks (512 bytes of each weight row),
// each wave loading weights straight from memory to registers, 16 KiB in flight at
// once, without LDS or barriers; rows of x come from the caches.  The waves' sums
// are added in wave order through LDS.  The memory's rate bounds it: 2 experts'
// 14336 x 4096 weights in 24 us, 4.8 TB/s, 64 experts' 1536 x 2048 (488 rows) in 40 us,
// 4.9 TB/s (a large copy: 4.9).  (Quantising bf16 rows in each wave instead of a
// launch before took as long: 29.8 against 28.8 us for one token.  The non-temporal
// hint lost 7 %: a lane group's two halves of a cache line are two loads.)
constexpr int kSmallCols = kFp8SmallCols;

// Row pieces of TILE rows, group by group.  A wave finds the piece that holds unit
// `slot` of `per` units to a piece: expert, its first row and rows, and the unit's
// number within its group; returns the number of units, which slot reaches where there is none.
// (64 groups at a time with shuffles: no LDS, no barrier.)
struct Piece {
  int e, start, rows, unit;
};
template <int TILE>
__device__ __forceinline__ int find_piece(const Fp8GemmParams& p, int slot, int per, Piece* out) {
  const int lane = threadIdx.x & 63, E = p.num_groups, M = (int)p.m_rows;
  int carry = 0, before = 0;
  for (int base = 0; base < E; base += 64) {
    const int v = base + lane < E ? min(max(p.offs[base + lane], 0), M) : 0;
    const int incl = max(wave_incl_max(v), carry);
    int prev = __shfl_up(incl, 1, 64);
    if (lane == 0) prev = carry;
    const int m = incl - prev;
    const int units = (m + TILE - 1) / TILE * per;
    const int upto = before + wave_incl_sum(units);
    const uint64_t over = __ballot(slot < upto);
    if (over != 0 && slot >= before) {
      const int src = __ffsll((unsigned long long)over) - 1;
      out->e = uniform(base + src);
      out->start = uniform(__shfl(prev, src, 64));
      out->rows = uniform(__shfl(m, src, 64));
      out->unit = uniform(slot - (__shfl(upto, src, 64) - __shfl(units, src, 64)));
    }
    before = uniform(__shfl(upto, 63, 64));
    carry = __shfl(incl, 63, 64);
  }
  return before;
}

template <int S>
__device__ __forceinline__ f32x4 mfma_small(const i32x8& w, const i32x8& x, f32x4 c, uint32_t sw, uint32_t sx) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 0, 0, S, sw, S, sx);
}

// MB row blocks of 16; acc[i][j]: row block i, column block j.
template <int MB>
__device__ __forceinline__ void small_product(const Fp8GemmParams& p, int e, int row0, int rows, int n0,
                                              f32x4 (&acc)[MB][2]) {
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const int k = p.k, r = lane & 15, c = (lane >> 4) * 16;
  const int cols = min(kSmallCols, p.n - n0);
  const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.w) + ((int64_t)e * p.n + n0) * k, 0, uniform(cols * k), 0x00020000);
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.x) + (int64_t)row0 * k, 0, uniform(rows * k), 0x00020000);
  const int nb = (p.n + kFp8Block - 1) / kFp8Block;
  const uint8_t* ws = p.ws + ((int64_t)e * nb + n0 / kFp8Block) * p.blocks;
  const __amdgpu_buffer_rsrc_t rs =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(ws), 0, uniform(p.blocks), 0x00020000);
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int g = w; 4 * g < p.blocks; g += 4) {
    // 16 bytes at chunk h of block b of row `row` (chunks past the row's end read zeros)
    auto chunk = [&](__amdgpu_buffer_rsrc_t rsrc, int row, int b, int h) {
      const int at = (4 * g + b) * kFp8Block + h * 64 + c;
      return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                           rsrc, at < k ? (uint32_t)(row * k + at) : kOutOfRange, 0, 0));
    };
    auto join = [](const i32x4& lo, const i32x4& hi) { return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); };
    i32x4 wf[4][2][2], xf[MB == 1 ? 4 : 1][2];
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) wf[b][j][h] = chunk(rw, j * 16 + r, b, h);
    uint32_t sx[MB], sw = 0;
    const __amdgpu_buffer_rsrc_t rxs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint32_t*>(p.xs) + (int64_t)g * p.m_rows + row0, 0, uniform(rows * 4), 0x00020000);
#pragma unroll
    for (int i = 0; i < MB; ++i) sx[i] = __builtin_amdgcn_raw_buffer_load_b32(rxs, (uint32_t)(i * 16 + r) * 4, 0, 0);
#pragma unroll
    for (int b = 0; b < 4; ++b)
      sw |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(rs, 4 * g + b, 0, 0) << (8 * b);
    if constexpr (MB == 1) {
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) xf[b][h] = chunk(rx, r, b, h);
    }
    // All of these loads go out before anything waits (left to itself the
    // compiler moves each next to its use: 33 us instead of 25 for two experts'
    // 14336 x 4096).
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        if constexpr (MB > 1) {
#pragma unroll
          for (int h = 0; h < 2; ++h) xf[0][h] = chunk(rx, i * 16 + r, b, h);
        }
        const i32x8 x = MB == 1 ? join(xf[MB == 1 ? b : 0][0], xf[MB == 1 ? b : 0][1]) : join(xf[0][0], xf[0][1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const i32x8 wv = join(wf[b][j][0], wf[b][j][1]);
          if (b == 0) acc[i][j] = mfma_small<0>(wv, x, acc[i][j], sw, sx[i]);
          else if (b == 1) acc[i][j] = mfma_small<1>(wv, x, acc[i][j], sw, sx[i]);
          else if (b == 2) acc[i][j] = mfma_small<2>(wv, x, acc[i][j], sw, sx[i]);
          else acc[i][j] = mfma_small<3>(wv, x, acc[i][j], sw, sx[i]);
        }
      }
  }
}

// Adds the waves' sums in wave order and stores rows < rows, columns < n as bf16:
// lane l of a block holds row l % 16 and columns 4 (l / 16) .. + 3.
template <int MB>
__device__ __forceinline__ void small_store(const Fp8GemmParams& p, int row0, int rows, int n0,
                                            const f32x4 (&acc)[MB][2], f32x4* s_acc) {
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) s_acc[((i * 2 + j) * 4 + w) * 64 + lane] = acc[i][j];
  __syncthreads();
#pragma unroll
  for (int t0 = 0; t0 < MB * 2; t0 += 4) {
    const int t = t0 + w;
    if (t >= MB * 2) break;
    f32x4 s = s_acc[t * 4 * 64 + lane];
#pragma unroll
    for (int q = 1; q < 4; ++q) s += s_acc[(t * 4 + q) * 64 + lane];
    const int row = (t >> 1) * 16 + (lane & 15), col = n0 + (t & 1) * 16 + (lane >> 4) * 4;
    if (row < rows && col < p.n) {
      u32x2 pk;
      pk[0] = pack_bf16x2(s[0], s[1]);
      pk[1] = pack_bf16x2(s[2], s[3]);
      *reinterpret_cast<u32x2*>(p.y + (int64_t)(row0 + row) * p.n + col) = pk;
    }
  }
}

template <int MB>
__device__ __forceinline__ void small_unit(const Fp8GemmParams& p, int e, int row0, int rows, int n0, f32x4* s_acc) {
  f32x4 acc[MB][2];
  small_product<MB>(p, e, row0, rows, n0, acc);
  small_store<MB>(p, row0, rows, n0, acc, s_acc);
}

__global__ __launch_bounds__(256, 3) void fp8_small_kernel(Fp8GemmParams p) {
  __shared__ f32x4 s_acc[kFp8SmallRows / 16 * 2 * 4 * 64];
  Piece u;
  if ((int)blockIdx.y >= find_piece<kFp8SmallRows>(p, blockIdx.y, 1, &u)) return;
  const int row0 = u.start + u.unit * kFp8SmallRows, rows = min(kFp8SmallRows, u.rows - u.unit * kFp8SmallRows);
  const int n0 = blockIdx.x * kSmallCols;
  if (rows <= 16) small_unit<1>(p, u.e, row0, rows, n0, s_acc);
  else if (rows <= 32) small_unit<2>(p, u.e, row0, rows, n0, s_acc);
  else small_unit<4>(p, u.e, row0, rows, n0, s_acc);
}

// ---------------------------------------------------------------------------
// the middle kernel: 128 x 128 tiles
// ---------------------------------------------------------------------------
// For groups too small for 256 x 256 tiles, or launches too small to fill the GPU
// with them.  Four waves of
// 64 x 64, the same stages and LDS layout as the tile kernel's at half the rows
// (16 KiB an operand), two buffers, two workgroups to a CU, one of which computes
// while the other waits.  A CU's stages then move 64 bytes per clock of matrix work,
// about what it can load, which bounds it: 2048 x 2048 x 2048 takes 15 us and 16 groups
// of 188 rows on average x 1000 x 2000 16 us, where the tile kernel takes 23 and 36.
// (Four buffers and one workgroup to a CU: 15.5 and 16.5 us, and 27 % longer where
// there are more units than CUs.)
constexpr int kMidTile = kFp8MidTile;
constexpr int kMidBytes = kMidTile * kFp8Block;

// Buffer B of operand A (0) or B (1); each a static array of its own, so that the
// compiler can tell reads of one from loads still landing in another.
template <int OPERAND, int B>
__device__ __forceinline__ uint8_t* mid_buffer() {
  __shared__ __attribute__((aligned(1024))) uint8_t s_buf[kMidBytes];
  return s_buf;
}

__global__ __launch_bounds__(256, 2) void fp8_mid_kernel(Fp8GemmParams p) {
  const int n_j = (p.n + kMidTile - 1) / kMidTile;
  // Workgroups go round the XCDs; each XCD takes consecutive units (which share
  // weights and rows), an eighth of them all.  The grid is an upper bound, so this
  // goes by the units there are: by the grid's size the first XCDs would get more.
  Piece u;
  const int total = find_piece<kMidTile>(p, -1, n_j, &u), share = (total + 7) / 8;
  const int v = (int)(blockIdx.x & 7) * share + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= share || v >= total) return;
  find_piece<kMidTile>(p, v, n_j, &u);
  const int e = u.e, gs = u.start, gm = u.rows;
  int rt, ct;
  panel_order(u.unit, (gm + kMidTile - 1) / kMidTile, n_j, 4, &rt, &ct);
  const int row0 = gs + rt * kMidTile, j0 = ct * kMidTile;
  const int i_valid = min(kMidTile, gm - rt * kMidTile), j_valid = min(kMidTile, p.n - j0);
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6), wi = w >> 1, wj = w & 1;
  const int k = p.k, nk = p.blocks;
  const uint8_t* xa = p.x + (int64_t)row0 * k;
  const uint8_t* xb = p.w + ((int64_t)e * p.n + j0) * k;
  const int nb = (p.n + kFp8Block - 1) / kFp8Block;
  const uint8_t* ws = p.ws + ((int64_t)e * nb + ct) * nk;  // (a tile's 128 columns are one block's)
  const uint32_t chunk = (uint32_t)(((lane & 7) ^ (lane >> 3)) * 16);
  const uint32_t off = (uint32_t)(w * 8 + (lane >> 3)) * (uint32_t)k + chunk;

  auto load_stage = [&](auto buffer, int kt) {
    constexpr int B = decltype(buffer)::value;
    const int left = k - kt * kFp8Block;
    const bool in = left > 0;
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(xa) + (in ? kt * kFp8Block : 0), 0, uniform(in ? i_valid * k - kt * kFp8Block : 0), 0x00020000);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(xb) + (in ? kt * kFp8Block : 0), 0, uniform(in ? j_valid * k - kt * kFp8Block : 0), 0x00020000);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t at = (int)chunk < left ? off + (uint32_t)(q * 32) * (uint32_t)k : kOutOfRange;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(mid_buffer<0, B>() + (q * 4 + w) * 1024), 16, at, 0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(mid_buffer<1, B>() + (q * 4 + w) * 1024), 16, at, 0, 0, 0);
    }
  };
  const int r = lane & 15, c = ((lane >> 4) ^ (r & 7)) * 16;
  const int fa = (wi * 64 + r) * 128 + c, fb = (wj * 64 + r) * 128 + c;
  uint32_t sx[4], sw, nx[4], nw;  // scales of 4 blocks, and of the next 4
  auto load_scales = [&](uint32_t (&x)[4], uint32_t* ww, int g) {
    const bool in = 4 * g < nk;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint32_t*>(p.xs) + (in ? (int64_t)g * p.m_rows + row0 : 0), 0,
        uniform(in ? (int)(p.m_rows - row0) * 4 : 0), 0x00020000);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = __builtin_amdgcn_raw_buffer_load_b32(rs, (uint32_t)(wi * 64 + i * 16 + r) * 4, 0, 0);
    const __amdgpu_buffer_rsrc_t rws = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(ws), 0, uniform(nk), 0x00020000);
    uint32_t v = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) v |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(rws, 4 * g + i, 0, 0) << (8 * i);
    *ww = v;
  };
  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // Stage kt (S = kt % 4, buffer S % 2): wait for its loads (the next stage's 8
  // follow them) and read its fragments; a second barrier after the reads frees its
  // buffer for stage kt + 2.
  auto step = [&](auto number, int kt) {
    constexpr int S = decltype(number)::value, B = S & 1;
    wait_vm_lgkm<8>();
    lds_barrier();
    i32x8 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = Fp8Pipe::frag(mid_buffer<0, B>(), fa, i);
      b[i] = Fp8Pipe::frag(mid_buffer<1, B>(), fb, i);
    }
    wait_lgkm();
    lds_barrier();  // every wave has its fragments
    if constexpr (S == 3) load_scales(nx, &nw, (kt >> 2) + 1);
    load_stage(std::integral_constant<int, B>{}, kt + 2);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) mfma_scaled_v<S>(acc[i][j], b[j], a[i], sw, sx[i]);
    if constexpr (S == 3) {
#pragma unroll
      for (int i = 0; i < 4; ++i) sx[i] = nx[i];
      sw = nw;
      settle(sx, sw);
    }
  };
  load_scales(sx, &sw, 0);
  load_stage(std::integral_constant<int, 0>{}, 0);
  load_stage(std::integral_constant<int, 1>{}, 1);
  settle(sx, sw);
  int kt = 0;
  for (; kt + 4 <= nk; kt += 4) {
    step(std::integral_constant<int, 0>{}, kt);
    step(std::integral_constant<int, 1>{}, kt + 1);
    step(std::integral_constant<int, 2>{}, kt + 2);
    step(std::integral_constant<int, 3>{}, kt + 3);
  }
  if (kt < nk) {
    step(std::integral_constant<int, 0>{}, kt);
    if (kt + 1 < nk) step(std::integral_constant<int, 1>{}, kt + 1);
    if (kt + 2 < nk) step(std::integral_constant<int, 2>{}, kt + 2);
  }
  wait_vm_lgkm<0>();
  __syncthreads();
  settle_results(acc);
  // 16 rows x 64 columns of a wave at a time through LDS to 128-byte row segments
  uint8_t* xo = mid_buffer<0, 0>() + w * 2048;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x2 pk;
      pk[0] = pack_bf16x2(acc[i][j][0], acc[i][j][1]);
      pk[1] = pack_bf16x2(acc[i][j][2], acc[i][j][3]);
      *reinterpret_cast<u32x2*>(xo + r * 128 + (((2 * j + (lane >> 5)) ^ (r & 7)) << 4) + ((lane >> 4) & 1) * 8) = pk;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int rr = q * 8 + (lane >> 3), cc = lane & 7;
      const u32x4 v4 = *reinterpret_cast<const u32x4*>(xo + rr * 128 + ((cc ^ (rr & 7)) << 4));
      const int row = wi * 64 + i * 16 + rr, col = wj * 64 + cc * 8;
      if (row < i_valid && col < j_valid)
        *reinterpret_cast<u32x4*>(p.y + (int64_t)(row0 + row) * p.n + j0 + col) = v4;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace

hipError_t launch_fp8_quantize_rows(const Fp8RowsParams& p, hipStream_t s) {
  const int64_t blocks = (p.m_rows * p.blocks + 31) / 32;
  const dim3 g((unsigned)(blocks < 8192 ? blocks : 8192)), b(256);
  if (p.fp32) hipLaunchKernelGGL((quantize_rows_kernel<true>), g, b, 0, s, p);
  else hipLaunchKernelGGL((quantize_rows_kernel<false>), g, b, 0, s, p);
  return hipGetLastError();
}

hipError_t launch_fp8_quantize_weight(const Fp8WeightParams& p, hipStream_t s) {
  const int64_t blocks = (int64_t)p.experts * ((p.n + 127) / 128) * ((p.k + 127) / 128);
  const dim3 g((unsigned)blocks), b(256);
  if (p.qt) {
    if (p.fp32) hipLaunchKernelGGL((quantize_weight_kernel<true, true>), g, b, 0, s, p);
    else hipLaunchKernelGGL((quantize_weight_kernel<false, true>), g, b, 0, s, p);
  } else {
    if (p.fp32) hipLaunchKernelGGL((quantize_weight_kernel<true, false>), g, b, 0, s, p);
    else hipLaunchKernelGGL((quantize_weight_kernel<false, false>), g, b, 0, s, p);
  }
  return hipGetLastError();
}

hipError_t launch_fp8_small(const Fp8GemmParams& p, int pieces, hipStream_t s) {
  const dim3 g((p.n + kSmallCols - 1) / kSmallCols, pieces), b(256);
  hipLaunchKernelGGL(fp8_small_kernel, g, b, 0, s, p);
  return hipGetLastError();
}

hipError_t launch_fp8_mid(const Fp8GemmParams& p, int grid, hipStream_t s) {
  hipLaunchKernelGGL(fp8_mid_kernel, dim3(grid), dim3(256), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_fp8_gemm(const Fp8GemmParams& p, int grid, hipStream_t s) {
  hipLaunchKernelGGL(fp8_gemm_kernel, dim3(grid), dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace mdg
