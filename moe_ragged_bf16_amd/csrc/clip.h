// Internal interface between the C ABI (capi_clip.cpp) and the gfx950 kernels of
// the gradient norm and clipping (clip_kernels.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mdg {

constexpr int kClipWords = 492;         // of the table in a launch's arguments (below 4 KiB)
constexpr int kClipUnitBytes = 32768;   // bytes of a tensor that a workgroup takes at a time
constexpr int kClipBlocks = 1024;       // workgroups of a launch, at most

// Tensors of one launch: two words each where an output is its own gradient (or there are
// none), else three.
constexpr int clip_tensors(bool apart) { return kClipWords / (apart ? 3 : 2); }

// The tensors of one launch, by value.
struct ClipTable {
  uint64_t words[kClipWords];           // addresses [capacity], elements [capacity], outputs' addresses
  int32_t count;
  int32_t apart;                        // outputs have addresses of their own
  int32_t blocks;                       // of the norm kernel (and partial sums of this launch)
  int32_t first;                        // partial sums of the launches before it
  int32_t partials;                     // of all launches
  float max_norm, eps;
  double* partial;                      // [partials]
  const float* norm_in;                 // scaling: the norm, or nullptr: from the partial sums
  float* norm_out;                      // scaling and finishing: where the norm goes, or nullptr
};
static_assert(sizeof(ClipTable) <= 4096, "kernel arguments");

hipError_t launch_clip_norm(const ClipTable& t, hipStream_t s);
hipError_t launch_clip_finish(const ClipTable& t, hipStream_t s);
hipError_t launch_clip_scale(const ClipTable& t, int blocks, hipStream_t s);

}  // namespace mdg
