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

// The current device is one the kernels run on; *dev (where given) its properties.
inline int check_device(DeviceInfo* dev = nullptr) {
  DeviceInfo own;
  int device = -1;
  if (!dev) dev = &own;
  const int st = query_device(dev, &device);
  if (st != MDG_OK) return st;
  return dev->gfx950 ? MDG_OK : MDG_EUNSUPPORTED;
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

// A workspace of at least `need` bytes on 256 (any where none is needed).
inline int check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (need == 0) return MDG_OK;
  if (!workspace || bytes < need) return MDG_EWORKSPACE;
  return (reinterpret_cast<uintptr_t>(workspace) & 255u) == 0 ? MDG_OK : MDG_EINVAL;
}

inline mdg_status status(int st) { return static_cast<mdg_status>(st); }

}  // namespace mdg
