// Internal interface between the C ABI (capi_clip.cpp) and the gfx950 kernels of
// the gradient norm and clipping (clip_kernels.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mdg {

constexpr int kClipWords = 1008;        // 32-bit ones of the table in a launch's arguments (4 KiB in all)
constexpr int kClipUnitBytes = 32768;   // bytes of a tensor that a workgroup takes at a time
constexpr int kClipBlocks = 1024;       // workgroups of a launch, at most
constexpr int kClipPartials = 1024;     // partial sums that every scaling workgroup adds up itself, at most

// Words of a tensor: its address's low half, 22 bits above them (16 of the address, 6 of the
// size), the size's low half, and where outputs are apart the output's address in two.  (An address
// has 48 bits.)  The size is 2 elements + (1: fp32), of 38 bits.
constexpr int clip_words(bool apart) { return apart ? 5 : 3; }
constexpr int clip_tensors(bool apart) { return kClipWords / clip_words(apart); }  // of one launch

// The tensors of one launch, by value.
struct ClipTable {
  uint32_t words[kClipWords];           // [words of a tensor][capacity]
  int32_t count;
  int32_t apart;                        // outputs have addresses of their own
  int32_t blocks;                       // of the norm kernel (and partial sums of this launch)
  int32_t first;                        // partial sums of the launches before it
  int32_t partials;                     // of all launches
  float max_norm, eps;
  int32_t finished;                     // scaling: partial[0] is the norm itself
  double* partial;                      // [partials]
  const float* norm_in;                 // scaling: the norm, or nullptr: from the partial sums
  float* norm_out;                      // scaling and finishing: where the norm goes, or nullptr (finishing: to partial[0])
};
static_assert(sizeof(ClipTable) <= 4096, "kernel arguments");

hipError_t launch_clip_norm(const ClipTable& t, hipStream_t s);
hipError_t launch_clip_finish(const ClipTable& t, hipStream_t s);
hipError_t launch_clip_scale(const ClipTable& t, int blocks, hipStream_t s);

}  // namespace mdg
