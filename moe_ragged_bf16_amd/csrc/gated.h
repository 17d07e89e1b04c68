// Internal interface between the C ABI (capi_gated.cpp) and the gfx950 kernels of
// the experts' gated feed-forward (gated_kernels.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "grouped_gemm.h"

namespace mdg {

constexpr int kGatedCols = kTileJ / 2;  // hidden columns of a fwd tile: gate and up of each

constexpr int kGatedSmallCols = 16;         // hidden columns of the small kernel's units
constexpr int kGatedSmallRows = 64;         // and their rows, at most
constexpr int kGatedMidTile = 128;          // rows, and columns of operand B, of the middle kernel's tiles

enum Activation : int { kActSilu = 0, kActGeluTanh = 1 };

struct GatedParams {
  // The product.  fwd: a = x, b = w, out = h, n = 2 f, k; dgrad: a = dy, b = w_down,
  // out = dgate_up, n, k = f.
  GemmParams g;
  const uint16_t* gate_up;  // dgrad: [m_rows, 2 f] as fwd kept them
  uint16_t* keep;           // fwd: [m_rows, 2 f] the projections, or nullptr
  int32_t f;
  int32_t act;              // kActSilu or kActGeluTanh
};

// Where a split tail unit's tile goes (written by the tile kernel, read by the
// reduce kernel; in place of GemmParams' TailUnit).
struct GatedTail {
  int32_t row0, f0, i_valid, f_valid;
};

hipError_t launch_gated(Op op, const GatedParams& p, int grid, hipStream_t s);
hipError_t launch_gated_small(const GatedParams& p, int pieces, hipStream_t s);  // fwd
hipError_t launch_gated_mid(Op op, const GatedParams& p, int tile, int grid, hipStream_t s);  // tile: kGatedMidTile or half
hipError_t launch_gated_reduce(Op op, const GatedParams& p, int grid_x, int grid_y, hipStream_t s);

}  // namespace mdg
