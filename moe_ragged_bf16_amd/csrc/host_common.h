// Host helpers shared by the C ABI's sources: the device query and the argument
// checks every entry point makes before it enqueues anything.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <mutex>

#include "moe_ragged_bf16.h"

namespace mdg {

struct DeviceInfo {
  bool ok = false;
  bool gfx950 = false;
  int cus = 0;
};

inline DeviceInfo g_dev[64];
inline std::once_flag g_dev_once[64];

inline int query_device(DeviceInfo* out, int* device) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return MDG_EHIP;
  *device = dev;
  std::call_once(g_dev_once[dev], [dev]() {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return;
    g_dev[dev].gfx950 = strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    g_dev[dev].cus = prop.multiProcessorCount;
    g_dev[dev].ok = true;
  });
  if (!g_dev[dev].ok) return MDG_EHIP;
  *out = g_dev[dev];
  return MDG_OK;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

inline Range range_of(const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + (uintptr_t)(bytes > 0 ? bytes : 0)};
}

inline bool overlaps(Range a, Range b) {
  if (a.hi == a.lo || b.hi == b.lo) return false;
  return a.lo < b.hi && b.lo < a.hi;
}

inline mdg_status status(int st) { return static_cast<mdg_status>(st); }

}  // namespace mdg
