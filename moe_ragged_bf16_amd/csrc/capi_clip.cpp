// C ABI of the gradient norm and clipping (include/moe_ragged_bf16.h): argument
// checks before anything is enqueued, the tensors dealt to launches, launches.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <memory>
#include <new>

#include "clip.h"
#include "host_common.h"
#include "moe_ragged_bf16.h"

namespace mdg {
namespace {

constexpr int64_t kMaxTensors = 65536;
constexpr int64_t kMaxElements = (int64_t)1 << 36;  // of a tensor: its size has 38 bits in a launch's arguments

int64_t bytes_of(const mdg_gradient& g) { return g.elements * (g.dtype == MDG_FP32 ? 4 : 2); }
int64_t units_of(const mdg_gradient& g) { return (bytes_of(g) + kClipUnitBytes - 1) / kClipUnitBytes; }
int64_t launches_of(int64_t count, bool apart) { return (count + clip_tensors(apart) - 1) / clip_tensors(apart); }
size_t workspace_of(int64_t count) { return (size_t)launches_of(count, false) * kClipBlocks * sizeof(double); }

// (an address of more than 48 bits is none of the device's)
bool on_element(const void* p, int dtype) {
  return reinterpret_cast<uintptr_t>(p) % (dtype == MDG_FP32 ? 4 : 2) == 0 && reinterpret_cast<uintptr_t>(p) >> 48 == 0;
}

int check_gradients(const mdg_gradient* g, int64_t count, bool scaled) {
  if (count < 0 || (count > 0 && !g)) return MDG_EINVAL;
  if (count > kMaxTensors) return MDG_EUNSUPPORTED;
  // Of all tensors.  The kernels count a launch's in 32 bits, and a workgroup's count passes
  // the last one by up to a launch's workgroups.
  int64_t units = 0;
  for (int64_t i = 0; i < count; ++i) {
    const mdg_gradient& x = g[i];
    if ((x.dtype != MDG_BF16 && x.dtype != MDG_FP32) || x.elements < 0) return MDG_EINVAL;
    if (x.elements > kMaxElements) return MDG_EUNSUPPORTED;
    if (x.elements > 0 && (!x.data || !on_element(x.data, x.dtype))) return MDG_EINVAL;
    if (scaled && x.elements > 0 && (!x.out || !on_element(x.out, x.dtype))) return MDG_EINVAL;
    units += units_of(x);
    if (units > INT32_MAX - kClipBlocks) return MDG_EUNSUPPORTED;
  }
  return MDG_OK;
}

// Every output apart from every other output and from every other tensor's gradient,
// from its own but where it is in place, and from the norms and the workspace.
int check_outputs(const mdg_gradient* g, int64_t count, const Range (&others)[3]) {
  std::unique_ptr<Range[]> outs(new (std::nothrow) Range[count > 0 ? count : 1]);
  if (!outs) return MDG_ENOMEM;
  int64_t n = 0;
  for (int64_t i = 0; i < count; ++i)
    if (g[i].elements > 0) outs[n++] = range_of(g[i].out, bytes_of(g[i]));
  const auto below = [](const Range& a, const Range& b) { return a.lo < b.lo; };
  std::sort(outs.get(), outs.get() + n, below);
  for (int64_t i = 1; i < n; ++i)
    if (outs[i].lo < outs[i - 1].hi) return MDG_EOVERLAP;
  const auto hits = [&](const Range& r) {  // (the outputs are apart: their ends rise too)
    const Range* o = std::upper_bound(outs.get(), outs.get() + n, r,
                                      [](const Range& a, const Range& b) { return a.lo < b.hi; });
    return o != outs.get() + n && overlaps(*o, r);
  };
  for (int64_t i = 0; i < count; ++i)
    if (g[i].data != g[i].out && hits(range_of(g[i].data, bytes_of(g[i])))) return MDG_EOVERLAP;
  for (const Range& r : others)
    if (hits(r)) return MDG_EOVERLAP;
  return MDG_OK;
}

// The tensors of launch `k`, with the outputs where they are apart; `blocks` the
// workgroups its units fill.
ClipTable table_of(const mdg_gradient* g, int64_t count, int64_t k, bool apart) {
  ClipTable t{};
  const int capacity = clip_tensors(apart);
  int64_t units = 0;
  for (int64_t i = k * capacity; i < std::min(count, (k + 1) * capacity); ++i) {
    const bool some = g[i].elements > 0;  // (pointers of empty tensors may be anything)
    const uint64_t src = some ? reinterpret_cast<uint64_t>(g[i].data) : 0, dst = some ? reinterpret_cast<uint64_t>(g[i].out) : 0;
    const uint64_t size = 2 * (uint64_t)g[i].elements + (g[i].dtype == MDG_FP32);
    uint32_t* w = t.words + t.count;
    w[0] = (uint32_t)src;
    w[capacity] = (uint32_t)(src >> 32) | (uint32_t)(size >> 32) << 16;
    w[2 * capacity] = (uint32_t)size;
    if (apart) {
      w[3 * capacity] = (uint32_t)dst;
      w[4 * capacity] = (uint32_t)(dst >> 32);
    }
    ++t.count;
    units += units_of(g[i]);
  }
  t.apart = apart;
  t.blocks = (int32_t)std::max<int64_t>(1, std::min<int64_t>(units, kClipBlocks));
  return t;
}

// Enqueues the norm's launches; `last` gets what reads their sums.
int enqueue_norm(const mdg_gradient* g, int64_t count, double* partial, hipStream_t s, int32_t* partials) {
  int32_t first = 0;
  for (int64_t k = 0; k < launches_of(count, false); ++k) {
    ClipTable t = table_of(g, count, k, false);
    t.partial = partial;
    t.first = first;
    first += t.blocks;
    if (launch_clip_norm(t, s) != hipSuccess) return MDG_EHIP;
  }
  *partials = first;
  return MDG_OK;
}

}  // namespace
}  // namespace mdg

using namespace mdg;

extern "C" {

MDG_API size_t grad_norm_workspace_bytes(int64_t count) {
  return count < 0 || count > kMaxTensors ? 0 : workspace_of(count);
}

MDG_API mdg_status grad_norm(const mdg_gradient* gradients, int64_t count, float* norm, void* workspace,
                             size_t workspace_bytes, void* stream) {
  int st = check_gradients(gradients, count, false);
  if (st != MDG_OK) return status(st);
  if (!norm || !aligned4(norm)) return status(MDG_EINVAL);
  const size_t need = workspace_of(count);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MDG_OK) return status(st);
  const Range out = range_of(norm, 4), ws = range_of(workspace, (int64_t)need);
  if (overlaps(out, ws)) return status(MDG_EOVERLAP);
  for (int64_t i = 0; i < count; ++i) {
    const Range r = range_of(gradients[i].data, bytes_of(gradients[i]));
    if (overlaps(out, r) || overlaps(ws, r)) return status(MDG_EOVERLAP);
  }
  if ((st = check_device()) != MDG_OK) return status(st);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  ClipTable t{};
  t.partial = static_cast<double*>(workspace);
  if ((st = enqueue_norm(gradients, count, t.partial, s, &t.partials)) != MDG_OK) return status(st);
  t.norm_out = norm;
  return status(launch_clip_finish(t, s) == hipSuccess ? MDG_OK : MDG_EHIP);
}

MDG_API mdg_status grad_clip(const mdg_gradient* gradients, int64_t count, float max_norm, const float* norm_in,
                             float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_gradients(gradients, count, true);
  if (st != MDG_OK) return status(st);
  if (isnan(max_norm) || max_norm < 0.0f || !aligned4(norm_in) || !aligned4(norm)) return status(MDG_EINVAL);
  if (norm_in ? norm != nullptr : norm == nullptr) return status(MDG_EINVAL);
  const size_t need = norm_in ? 0 : workspace_of(count);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MDG_OK) return status(st);
  const Range others[3] = {range_of(norm_in, norm_in ? 4 : 0), range_of(norm, norm ? 4 : 0),
                           range_of(workspace, (int64_t)need)};
  if (overlaps(others[1], others[2])) return status(MDG_EOVERLAP);
  for (int64_t i = 0; i < count; ++i) {
    const Range r = range_of(gradients[i].data, bytes_of(gradients[i]));
    if (overlaps(others[1], r) || overlaps(others[2], r)) return status(MDG_EOVERLAP);
  }
  if ((st = check_outputs(gradients, count, others)) != MDG_OK) return status(st);
  if ((st = check_device()) != MDG_OK) return status(st);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  double* partial = static_cast<double*>(workspace);
  int32_t partials = 0;
  if (!norm_in && (st = enqueue_norm(gradients, count, partial, s, &partials)) != MDG_OK) return status(st);
  // More sums than a scaling workgroup's threads load at once are added up once, by a launch
  // of its own: added up by every workgroup of every launch their cost grows with the list's square
  // (each workgroup / once, in us, captured: 400 tensors of 60000 fp32 values, 1536 sums, 78 / 78, 1000 of them 159 / 150, 5000
  // 1092 / 896; 65536 of 20000 41500 / 4940).
  const bool finished = partials > kClipPartials;
  if (finished) {
    ClipTable t{};
    t.partial = partial;
    t.partials = partials;
    if (launch_clip_finish(t, s) != hipSuccess) return status(MDG_EHIP);
    partials = 0;
  }
  bool apart = false;
  for (int64_t i = 0; i < count; ++i) apart = apart || (gradients[i].elements > 0 && gradients[i].out != gradients[i].data);
  const int64_t launches = std::max<int64_t>(1, launches_of(count, apart));  // (without tensors: the norm, 0)
  for (int64_t k = launches - 1; k >= 0; --k) {
    ClipTable t = table_of(gradients, count, k, apart);
    if (norm_in && t.count == 0) return status(MDG_OK);
    t.partial = partial;
    t.partials = partials;
    t.finished = finished;
    t.norm_in = norm_in;
    t.norm_out = k == 0 ? norm : nullptr;
    t.max_norm = max_norm;
    t.eps = 1e-6f;
    if (launch_clip_scale(t, t.blocks, s) != hipSuccess) return status(MDG_EHIP);
  }
  return status(MDG_OK);
}

}  // extern "C"
