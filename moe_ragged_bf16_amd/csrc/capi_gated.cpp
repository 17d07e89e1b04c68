// C ABI of the experts' gated feed-forward (include/moe_ragged_bf16.h): argument
// checks before anything is enqueued, launch sizes, launches.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gated.h"
#include "grouped_gemm.h"
#include "host_common.h"
#include "moe_ragged_bf16.h"

namespace mdg {
namespace {

int check_sizes(int64_t m_rows, int64_t n, int64_t f, int32_t num_groups) {
  if (m_rows < 0 || n <= 0 || f <= 0 || num_groups <= 0) return MDG_EINVAL;
  if (num_groups > kMaxGroups || m_rows > kMaxRows) return MDG_EUNSUPPORTED;
  if (n % kKAlign != 0 || f % kNAlign != 0) return MDG_EUNSUPPORTED;
  if (n > (1 << 20) || f > (1 << 19) || 2 * n * f > INT32_MAX) return MDG_EUNSUPPORTED;
  return MDG_OK;
}

bool activation(int act, GatedParams* p) {
  const float c = 1.59576912160573071f;  // 2 sqrt(2 / pi)
  if (act == MDG_SILU) p->q0 = 1.0f, p->q1 = 0.0f;
  else if (act == MDG_GELU_TANH) p->q0 = c, p->q1 = c * 0.044715f;
  else return false;
  return true;
}

// Units of the tile kernel, at most: row tiles of every group, the last one of each
// possibly partial, times column tiles.
int64_t units_of(Op op, int64_t m_rows, int64_t f, int32_t num_groups) {
  const int64_t cols = op == kFwd ? kGatedCols : kTileJ;
  return ((m_rows + kTileI - 1) / kTileI + num_groups) * ((f + cols - 1) / cols);
}

// fp32 partial tiles of the tail split (as for the plain products).
int64_t slots_of(int64_t units) { return std::min<int64_t>(units * kMaxSplit, kBalanceSlots); }

size_t workspace_of(Op op, int64_t m_rows, int64_t n, int64_t f, int32_t num_groups) {
  if (check_sizes(m_rows, n, f, num_groups) != MDG_OK) return 0;
  return (size_t)kTailHeadBytes + (size_t)slots_of(units_of(op, m_rows, f, num_groups)) * kTileI * kTileJ * sizeof(float);
}

int run(Op op, GatedParams* p, int64_t m_rows, int64_t f, int32_t num_groups, void* workspace, void* stream) {
  DeviceInfo dev;
  int device = -1;
  const int st = query_device(&dev, &device);
  if (st != MDG_OK) return st;
  if (!dev.gfx950) return MDG_EUNSUPPORTED;
  const int64_t units = units_of(op, m_rows, f, num_groups), slots = slots_of(units);
  char* ws = static_cast<char*>(workspace);
  p->g.tail_head = reinterpret_cast<int32_t*>(ws);
  p->g.partial = reinterpret_cast<float*>(ws + kTailHeadBytes);
  p->g.tail_slots = (int32_t)slots;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  int64_t grid = std::min<int64_t>(units + slots, dev.cus > 0 ? dev.cus : 256);
  if (grid >= 8) grid -= grid % 8;
  if (launch_gated(op, *p, (int)grid, s) != hipSuccess) return MDG_EHIP;
  if (slots < 2) return MDG_OK;
  const int reduce = (int)std::min<int64_t>(kBalanceSlots / 2, slots / 2);
  return launch_gated_reduce(op, *p, 8, reduce, s) == hipSuccess ? MDG_OK : MDG_EHIP;
}

int check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (!workspace || bytes < need) return MDG_EWORKSPACE;
  return (reinterpret_cast<uintptr_t>(workspace) & 255u) == 0 ? MDG_OK : MDG_EINVAL;
}

}  // namespace
}  // namespace mdg

using namespace mdg;

extern "C" {

MDG_API size_t grouped_gated_gemm_fwd_workspace_bytes(int64_t m_rows, int64_t f, int64_t k, int32_t num_groups) {
  return workspace_of(kFwd, m_rows, k, f, num_groups);
}

MDG_API size_t grouped_gated_gemm_dgrad_workspace_bytes(int64_t m_rows, int64_t n, int64_t f, int32_t num_groups) {
  return workspace_of(kDgrad, m_rows, n, f, num_groups);
}

MDG_API mdg_status grouped_gated_gemm_fwd(const void* x, const void* w, const int32_t* offs, void* h, void* gate_up,
                                          int activation_code, int64_t m_rows, int64_t f, int64_t k,
                                          int32_t num_groups, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_sizes(m_rows, k, f, num_groups);
  if (st != MDG_OK) return status(st);
  GatedParams p{};
  if (!activation(activation_code, &p)) return status(MDG_EINVAL);
  if (!w || !offs || (m_rows > 0 && (!x || !h))) return status(MDG_EINVAL);
  if (!aligned16(x) || !aligned16(w) || !aligned4(offs) || !aligned16(h) || !aligned16(gate_up)) return status(MDG_EINVAL);
  const size_t need = workspace_of(kFwd, m_rows, k, f, num_groups);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MDG_OK) return status(st);
  const Range in[3] = {range_of(x, m_rows * k * 2), range_of(w, (int64_t)num_groups * 2 * f * k * 2),
                       range_of(offs, (int64_t)num_groups * 4)};
  const Range out[3] = {range_of(h, m_rows * f * 2), range_of(gate_up, gate_up ? m_rows * f * 4 : 0),
                        range_of(workspace, (int64_t)need)};
  for (int i = 0; i < 3; ++i) {
    for (const Range& r : in)
      if (overlaps(out[i], r)) return status(MDG_EOVERLAP);
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i], out[j])) return status(MDG_EOVERLAP);
  }
  if (m_rows == 0) return status(MDG_OK);
  p.g.a = static_cast<const uint16_t*>(x);
  p.g.b = static_cast<const uint16_t*>(w);
  p.g.offs = offs;
  p.g.out = h;
  p.g.m_rows = m_rows;
  p.g.n = (int32_t)(2 * f);
  p.g.k = (int32_t)k;
  p.g.num_groups = num_groups;
  p.keep = static_cast<uint16_t*>(gate_up);
  p.f = (int32_t)f;
  return status(run(kFwd, &p, m_rows, f, num_groups, workspace, stream));
}

MDG_API mdg_status grouped_gated_gemm_dgrad(const void* dy, const void* w_down, const void* gate_up,
                                            const int32_t* offs, void* dgate_up, int activation_code, int64_t m_rows,
                                            int64_t n, int64_t f, int32_t num_groups, void* workspace,
                                            size_t workspace_bytes, void* stream) {
  int st = check_sizes(m_rows, n, f, num_groups);
  if (st != MDG_OK) return status(st);
  GatedParams p{};
  if (!activation(activation_code, &p)) return status(MDG_EINVAL);
  if (!w_down || !offs || (m_rows > 0 && (!dy || !gate_up || !dgate_up))) return status(MDG_EINVAL);
  if (!aligned16(dy) || !aligned16(w_down) || !aligned16(gate_up) || !aligned4(offs) || !aligned16(dgate_up))
    return status(MDG_EINVAL);
  const size_t need = workspace_of(kDgrad, m_rows, n, f, num_groups);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MDG_OK) return status(st);
  const Range in[4] = {range_of(dy, m_rows * n * 2), range_of(w_down, (int64_t)num_groups * n * f * 2),
                       range_of(gate_up, m_rows * f * 4), range_of(offs, (int64_t)num_groups * 4)};
  const Range out = range_of(dgate_up, m_rows * f * 4), ws = range_of(workspace, (int64_t)need);
  for (const Range& r : in)
    if (overlaps(out, r) || overlaps(ws, r)) return status(MDG_EOVERLAP);
  if (overlaps(out, ws)) return status(MDG_EOVERLAP);
  if (m_rows == 0) return status(MDG_OK);
  p.g.a = static_cast<const uint16_t*>(dy);
  p.g.b = static_cast<const uint16_t*>(w_down);
  p.g.offs = offs;
  p.g.out = dgate_up;
  p.g.m_rows = m_rows;
  p.g.n = (int32_t)n;
  p.g.k = (int32_t)f;
  p.g.num_groups = num_groups;
  p.gate_up = static_cast<const uint16_t*>(gate_up);
  p.f = (int32_t)f;
  return status(run(kDgrad, &p, m_rows, f, num_groups, workspace, stream));
}

}  // extern "C"
