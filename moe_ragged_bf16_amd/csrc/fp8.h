// Internal interface between the C ABI (capi_fp8.cpp) and the gfx950 kernels of
// the grouped product in 8 bits (fp8_kernels.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mdg {

constexpr int kFp8Block = 128;   // values that share a scale along a row (weights: 128 x 128)
constexpr int kFp8SmallRows = 64; // rows of a unit of the small kernel
constexpr int kFp8SmallCols = 32; // ... and columns
constexpr int kFp8MidTile = 128;  // rows and columns of a unit of the middle kernel

// Rows of 8-bit values lie at a pitch of whole 16-byte chunks, zeros behind k.
inline int64_t fp8_pitch(int64_t k) { return (k + 15) / 16 * 16; }

// Scales of rows: e8m0 codes, four consecutive blocks of a row to a 32-bit word,
// word [block / 4][row].
struct Fp8RowsParams {
  const void* x;      // [m_rows, k] bf16 or fp32
  uint8_t* q;         // [m_rows, pitch] e4m3
  uint8_t* scale;     // [ceil(blocks / 4)][m_rows][4]
  int64_t m_rows;
  int32_t k, pitch, blocks;  // blocks = ceil(k / 128)
  int32_t fp32;
};

struct Fp8WeightParams {
  const void* w;      // [experts, n, k] bf16 or fp32
  uint8_t* q;         // [experts, n, pitch]
  uint8_t* scale;     // [experts, ceil(n / 128), ceil(k / 128)]
  uint8_t* qt;        // [experts, k, pitch_t] or nullptr
  uint8_t* scale_t;   // [experts, ceil(k / 128), ceil(n / 128)]
  int32_t experts, n, k;
  int32_t pitch, pitch_t;
  int32_t fp32;
};

struct Fp8GemmParams {
  const uint8_t* x;       // [m_rows, k] e4m3, k the pitch
  const uint32_t* xs;     // [ceil(blocks / 4)][m_rows] words of 4 scales
  const uint8_t* w;       // [experts, n, k] e4m3
  const uint8_t* ws;      // [experts, ceil(n / 128), blocks]
  const int32_t* offs;    // [experts]
  uint16_t* y;            // [m_rows, n] bf16
  int64_t m_rows;
  int32_t n, k, num_groups, blocks;
};

hipError_t launch_fp8_quantize_rows(const Fp8RowsParams& p, hipStream_t s);
hipError_t launch_fp8_quantize_weight(const Fp8WeightParams& p, hipStream_t s);
hipError_t launch_fp8_small(const Fp8GemmParams& p, int pieces, hipStream_t s);
hipError_t launch_fp8_mid(const Fp8GemmParams& p, int grid, hipStream_t s);
hipError_t launch_fp8_gemm(const Fp8GemmParams& p, int grid, hipStream_t s);

}  // namespace mdg
