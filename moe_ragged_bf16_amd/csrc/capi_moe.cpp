// C ABI of routing, planning, dispatch and combine (include/moe_ragged_bf16.h):
// argument checks before anything is enqueued, launch sizes, launches.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "grouped_gemm.h"
#include "host_common.h"
#include "moe.h"
#include "moe_ragged_bf16.h"

namespace mdg {
namespace {

size_t align256(size_t b) { return (b + 255) / 256 * 256; }

// Every output apart from every input and from every other output.
bool outputs_apart(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  for (const Range* o = outs.begin(); o != outs.end(); ++o) {
    for (const Range& i : ins)
      if (overlaps(*o, i)) return false;
    for (const Range* q = outs.begin(); q != o; ++q)
      if (overlaps(*o, *q)) return false;
  }
  return true;
}

bool aligned_to(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

int check_device() {
  DeviceInfo dev;
  int device = -1;
  const int st = query_device(&dev, &device);
  if (st != MDG_OK) return st;
  return dev.gfx950 ? MDG_OK : MDG_EUNSUPPORTED;
}

int check_dtype(int dtype) { return dtype == MDG_BF16 || dtype == MDG_FP32 ? MDG_OK : MDG_EINVAL; }
int64_t dtype_bytes(int dtype) { return dtype == MDG_FP32 ? 4 : 2; }

int check_route_sizes(int64_t tokens, int32_t experts, int32_t top_k) {
  if (tokens < 0 || experts <= 0 || top_k <= 0) return MDG_EINVAL;
  if (experts > kRouteMaxExperts || top_k > kRouteMaxTopK || top_k > experts) return MDG_EUNSUPPORTED;
  if (tokens > kMaxRows / top_k) return MDG_EUNSUPPORTED;
  return MDG_OK;
}

// How a route call is cut: blocks of `threads`, each with consecutive tokens.
// One block when its threads cover the tokens in at most 4 steps (no second
// launch); otherwise at most kRouteMaxBlocks, of 256 threads until every block
// has work for more.
struct RouteCut {
  int blocks, threads;
  int64_t rows_per_block;
};

RouteCut route_cut(int64_t tokens, int32_t experts) {
  const int most = experts <= 512 ? kRouteThreads : kRouteThreads / 2;  // the block's sums stay within 64 KiB of LDS
  const int64_t lanes = std::max<int64_t>(1, tokens * route_lanes(experts));
  RouteCut c;
  if (lanes <= 4 * most) {
    c.blocks = 1;
    c.threads = (int)std::min<int64_t>(most, (lanes + 63) / 64 * 64);
  } else {
    const int64_t per_block = (lanes + kRouteMaxBlocks - 1) / kRouteMaxBlocks;
    c.threads = (int)std::max<int64_t>(256, std::min<int64_t>(most, (per_block + 63) / 64 * 64));
    c.blocks = (int)std::min<int64_t>(kRouteMaxBlocks, (lanes + c.threads - 1) / c.threads);
  }
  c.rows_per_block = (tokens + c.blocks - 1) / c.blocks;
  return c;
}

// Workspace of a cut call: shares and counter of the finishing kernel, then the
// blocks' probability sums, counts and routed tokens.
constexpr size_t kRouteHead = 1024 * 8 + 256;  // a share for every expert at most

size_t route_workspace(int64_t tokens, int32_t experts) {
  const RouteCut c = route_cut(tokens, experts);
  return c.blocks == 1 ? 0 : align256(kRouteHead + (size_t)c.blocks * ((size_t)experts * 8 + 4));
}

int check_rows_sizes(int64_t tokens, int32_t top_k, int32_t experts) {
  if (tokens < 0 || top_k <= 0 || experts <= 0) return MDG_EINVAL;
  if (experts > kMaxGroups || top_k > kRouteMaxTopK) return MDG_EUNSUPPORTED;
  if (tokens > kMaxRows / top_k) return MDG_EUNSUPPORTED;
  return MDG_OK;
}

int64_t plan_chunk(int64_t slots) {
  const int64_t most = (int64_t)kPlanChunk * kPlanMaxBlocks;
  return kPlanChunk * std::max<int64_t>(1, (slots + most - 1) / most);
}
int plan_blocks(int64_t slots) {
  const int64_t c = plan_chunk(slots);
  return (int)std::max<int64_t>(1, (slots + c - 1) / c);
}
size_t plan_workspace(int64_t slots, int32_t experts) {
  const int b = plan_blocks(slots);
  return b == 1 ? 0 : align256((size_t)b * experts * 4);
}

int check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need == 0) return MDG_OK;
  if (!ws || bytes < need) return MDG_EWORKSPACE;
  return aligned_to(ws, 256) ? MDG_OK : MDG_EINVAL;
}

// Sizes and types shared by the calls that move rows.
int check_rows(int64_t tokens, int32_t top_k, int32_t experts, int64_t hidden, int dtype) {
  int st = check_rows_sizes(tokens, top_k, experts);
  if (st != MDG_OK) return st;
  if ((st = check_dtype(dtype)) != MDG_OK) return st;
  if (hidden <= 0) return MDG_EINVAL;
  if (hidden * dtype_bytes(dtype) % 16 != 0 || hidden > (1 << 20)) return MDG_EUNSUPPORTED;
  return MDG_OK;
}

RowsParams rows_params(int64_t tokens, int32_t top_k, int32_t experts, int64_t hidden, int dtype) {
  RowsParams p{};
  p.tokens = tokens;
  p.slots = tokens * top_k;
  p.top_k = top_k;
  p.experts = experts;
  p.pieces = (int32_t)(hidden * dtype_bytes(dtype) / 16);
  p.fp32 = dtype == MDG_FP32;
  return p;
}

mdg_status launched(hipError_t err) { return status(err == hipSuccess ? MDG_OK : MDG_EHIP); }

}  // namespace
}  // namespace mdg

using namespace mdg;

extern "C" {

MDG_API size_t moe_route_fwd_workspace_bytes(int64_t tokens, int32_t experts) {
  return check_route_sizes(tokens, experts, 1) == MDG_OK ? route_workspace(tokens, experts) : 0;
}

MDG_API mdg_status moe_route_fwd(const void* logits, int dtype, const uint8_t* token_mask, float* weight,
                                 int32_t* idx, int32_t* counts, float* loss, float* balance, int64_t tokens,
                                 int32_t experts, int32_t top_k, int normalize, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  int st = check_route_sizes(tokens, experts, top_k);
  if (st != MDG_OK || (st = check_dtype(dtype)) != MDG_OK) return status(st);
  if (!counts || !loss || !balance || (tokens > 0 && (!logits || !weight || !idx))) return status(MDG_EINVAL);
  const int64_t esz = dtype_bytes(dtype);
  if (!aligned_to(logits, (int)esz) || !aligned4(weight) || !aligned4(idx) || !aligned4(counts) || !aligned4(loss) ||
      !aligned4(balance))
    return status(MDG_EINVAL);
  const size_t need = route_workspace(tokens, experts);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MDG_OK) return status(st);
  const int64_t slots = tokens * top_k;
  if (!outputs_apart({range_of(weight, slots * 4), range_of(idx, slots * 4), range_of(counts, (int64_t)experts * 4),
                      range_of(loss, 4), range_of(balance, (int64_t)experts * 4), range_of(workspace, (int64_t)need)},
                     {range_of(logits, tokens * experts * esz), range_of(token_mask, token_mask ? tokens : 0)}))
    return status(MDG_EOVERLAP);
  if ((st = check_device()) != MDG_OK) return status(st);

  const RouteCut cut = route_cut(tokens, experts);
  RouteParams p{};
  p.logits = logits;
  p.mask = token_mask;
  p.weight = weight;
  p.idx = idx;
  p.counts = counts;
  p.loss = loss;
  p.balance = balance;
  p.tokens = tokens;
  p.rows_per_block = cut.rows_per_block;
  p.experts = experts;
  p.top_k = top_k;
  p.normalize = normalize != 0;
  p.fp32 = dtype == MDG_FP32;
  p.vec = aligned16(logits) && experts % route_values(experts) == 0;  // (both sides' times: the kernels' LogitBits)
  p.blocks = cut.blocks;
  if (cut.blocks > 1) {
    char* ws = static_cast<char*>(workspace);
    p.part_share = reinterpret_cast<double*>(ws);
    p.part_done = reinterpret_cast<int32_t*>(ws + kRouteHead - 256);
    p.part_sum = reinterpret_cast<float*>(ws + kRouteHead);
    p.part_cnt = reinterpret_cast<int32_t*>(p.part_sum + (size_t)cut.blocks * experts);
    p.part_routed = p.part_cnt + (size_t)cut.blocks * experts;
  }
  return launched(launch_route_fwd(p, cut.threads, static_cast<hipStream_t>(stream)));
}

MDG_API mdg_status moe_route_bwd(const void* logits, int dtype, const float* weight, const int32_t* idx,
                                 const float* balance, const float* dweight, const float* dloss, void* dlogits,
                                 int64_t tokens, int32_t experts, int32_t top_k, int normalize, void* stream) {
  int st = check_route_sizes(tokens, experts, top_k);
  if (st != MDG_OK || (st = check_dtype(dtype)) != MDG_OK) return status(st);
  if (!balance || (tokens > 0 && (!logits || !weight || !idx || !dlogits))) return status(MDG_EINVAL);
  const int64_t esz = dtype_bytes(dtype);
  if (!aligned_to(logits, (int)esz) || !aligned_to(dlogits, (int)esz) || !aligned4(weight) || !aligned4(idx) ||
      !aligned4(balance) || !aligned4(dweight) || !aligned4(dloss))
    return status(MDG_EINVAL);
  const int64_t slots = tokens * top_k, row_bytes = tokens * experts * esz;
  if (!outputs_apart({range_of(dlogits, row_bytes)},
                     {range_of(logits, row_bytes), range_of(weight, slots * 4), range_of(idx, slots * 4),
                      range_of(balance, (int64_t)experts * 4), range_of(dweight, dweight ? slots * 4 : 0),
                      range_of(dloss, dloss ? 4 : 0)}))
    return status(MDG_EOVERLAP);
  if (tokens == 0) return status(MDG_OK);
  if ((st = check_device()) != MDG_OK) return status(st);
  RouteBwdParams p{};
  p.logits = logits;
  p.weight = weight;
  p.idx = idx;
  p.balance = balance;
  p.dweight = dweight;
  p.dloss = dloss;
  p.dlogits = dlogits;
  p.tokens = tokens;
  p.experts = experts;
  p.top_k = top_k;
  p.normalize = normalize != 0;
  p.fp32 = dtype == MDG_FP32;
  p.vec = aligned16(logits) && aligned16(dlogits) && experts % route_values(experts) == 0;
  return launched(launch_route_bwd(p, static_cast<hipStream_t>(stream)));
}

MDG_API size_t moe_plan_workspace_bytes(int64_t tokens, int32_t top_k, int32_t experts) {
  return check_rows_sizes(tokens, top_k, experts) == MDG_OK ? plan_workspace(tokens * top_k, experts) : 0;
}

MDG_API mdg_status moe_plan(const int32_t* idx, int32_t* offs, int32_t* dest, int64_t tokens, int32_t top_k,
                            int32_t experts, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_rows_sizes(tokens, top_k, experts);
  if (st != MDG_OK) return status(st);
  if (!offs || (tokens > 0 && (!idx || !dest))) return status(MDG_EINVAL);
  if (!aligned4(idx) || !aligned4(offs) || !aligned4(dest)) return status(MDG_EINVAL);
  const int64_t slots = tokens * top_k;
  const size_t need = plan_workspace(slots, experts);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MDG_OK) return status(st);
  if (!outputs_apart({range_of(offs, (int64_t)experts * 4), range_of(dest, slots * 4),
                      range_of(workspace, (int64_t)need)},
                     {range_of(idx, slots * 4)}))
    return status(MDG_EOVERLAP);
  if ((st = check_device()) != MDG_OK) return status(st);
  PlanParams p{};
  p.idx = idx;
  p.offs = offs;
  p.dest = dest;
  p.hist = static_cast<int32_t*>(workspace);
  p.slots = slots;
  p.chunk = plan_chunk(slots);
  p.experts = experts;
  p.blocks = plan_blocks(slots);
  p.runs = experts <= 512 ? kPlanThreads / 64 : kPlanThreads / 128;  // the runs' counts stay within 32 KiB of LDS
  return launched(launch_plan(p, static_cast<hipStream_t>(stream)));
}

MDG_API mdg_status moe_dispatch_fwd(const void* x, const int32_t* dest, const int32_t* offs, void* rows,
                                    int64_t tokens, int32_t top_k, int32_t experts, int64_t hidden, int dtype,
                                    void* stream) {
  int st = check_rows(tokens, top_k, experts, hidden, dtype);
  if (st != MDG_OK) return status(st);
  if (!offs || (tokens > 0 && (!x || !dest || !rows))) return status(MDG_EINVAL);
  if (!aligned16(x) || !aligned4(dest) || !aligned4(offs) || !aligned16(rows)) return status(MDG_EINVAL);
  RowsParams p = rows_params(tokens, top_k, experts, hidden, dtype);
  const int64_t row = (int64_t)p.pieces * 16;
  if (!outputs_apart({range_of(rows, p.slots * row)},
                     {range_of(x, tokens * row), range_of(dest, p.slots * 4), range_of(offs, (int64_t)experts * 4)}))
    return status(MDG_EOVERLAP);
  if (tokens == 0) return status(MDG_OK);
  if ((st = check_device()) != MDG_OK) return status(st);
  p.in = x;
  p.dest = dest;
  p.offs = offs;
  p.out = rows;
  return launched(launch_dispatch(p, static_cast<hipStream_t>(stream)));
}

MDG_API mdg_status moe_dispatch_bwd(const void* drows, const int32_t* dest, void* dx, int64_t tokens, int32_t top_k,
                                    int64_t hidden, int dtype, void* stream) {
  int st = check_rows(tokens, top_k, 1, hidden, dtype);
  if (st != MDG_OK) return status(st);
  if (tokens > 0 && (!drows || !dest || !dx)) return status(MDG_EINVAL);
  if (!aligned16(drows) || !aligned4(dest) || !aligned16(dx)) return status(MDG_EINVAL);
  RowsParams p = rows_params(tokens, top_k, 1, hidden, dtype);
  const int64_t row = (int64_t)p.pieces * 16;
  if (!outputs_apart({range_of(dx, tokens * row)}, {range_of(drows, p.slots * row), range_of(dest, p.slots * 4)}))
    return status(MDG_EOVERLAP);
  if (tokens == 0) return status(MDG_OK);
  if ((st = check_device()) != MDG_OK) return status(st);
  p.in = drows;
  p.dest = dest;
  p.out = dx;
  return launched(launch_gather_sum(p, static_cast<hipStream_t>(stream)));
}

MDG_API mdg_status moe_combine_fwd(const void* y, const float* weight, const int32_t* dest, void* out, int64_t tokens,
                                   int32_t top_k, int64_t hidden, int dtype, void* stream) {
  int st = check_rows(tokens, top_k, 1, hidden, dtype);
  if (st != MDG_OK) return status(st);
  if (tokens > 0 && (!y || !weight || !dest || !out)) return status(MDG_EINVAL);
  if (!aligned16(y) || !aligned4(weight) || !aligned4(dest) || !aligned16(out)) return status(MDG_EINVAL);
  RowsParams p = rows_params(tokens, top_k, 1, hidden, dtype);
  const int64_t row = (int64_t)p.pieces * 16;
  if (!outputs_apart({range_of(out, tokens * row)},
                     {range_of(y, p.slots * row), range_of(weight, p.slots * 4), range_of(dest, p.slots * 4)}))
    return status(MDG_EOVERLAP);
  if (tokens == 0) return status(MDG_OK);
  if ((st = check_device()) != MDG_OK) return status(st);
  p.in = y;
  p.weight = weight;
  p.dest = dest;
  p.out = out;
  return launched(launch_gather_sum(p, static_cast<hipStream_t>(stream)));
}

MDG_API mdg_status moe_combine_bwd(const void* dout, const void* y, const float* weight, const int32_t* dest,
                                   const int32_t* offs, void* dy, float* dweight, int64_t tokens, int32_t top_k,
                                   int32_t experts, int64_t hidden, int dtype, void* stream) {
  int st = check_rows(tokens, top_k, experts, hidden, dtype);
  if (st != MDG_OK) return status(st);
  if (!offs || (tokens > 0 && (!dout || !y || !weight || !dest || !dy || !dweight))) return status(MDG_EINVAL);
  if (!aligned16(dout) || !aligned16(y) || !aligned4(weight) || !aligned4(dest) || !aligned4(offs) ||
      !aligned16(dy) || !aligned4(dweight))
    return status(MDG_EINVAL);
  RowsParams p = rows_params(tokens, top_k, experts, hidden, dtype);
  const int64_t row = (int64_t)p.pieces * 16;
  if (!outputs_apart({range_of(dy, p.slots * row), range_of(dweight, p.slots * 4)},
                     {range_of(dout, tokens * row), range_of(y, p.slots * row), range_of(weight, p.slots * 4),
                      range_of(dest, p.slots * 4), range_of(offs, (int64_t)experts * 4)}))
    return status(MDG_EOVERLAP);
  if (tokens == 0) return status(MDG_OK);
  if ((st = check_device()) != MDG_OK) return status(st);
  p.in = y;
  p.dout = dout;
  p.weight = weight;
  p.dest = dest;
  p.offs = offs;
  p.out = dy;
  p.dweight = dweight;
  return launched(launch_combine_bwd(p, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
