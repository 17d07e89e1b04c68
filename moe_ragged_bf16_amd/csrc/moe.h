// Internal interface between the C ABI (capi_moe.cpp) and the gfx950 kernels of
// routing, planning, dispatch and combine (moe_kernels.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mdg {

constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopK = 32;
constexpr int kRouteMaxBlocks = 256;  // blocks of a route call that leave partial sums
constexpr int kRouteThreads = 1024;   // most threads of a route block
constexpr int kPlanThreads = 1024;
constexpr int kPlanChunk = 4096;      // slots one plan block sorts (a multiple, beyond kPlanMaxBlocks blocks)
constexpr int kPlanMaxBlocks = 256;

struct RouteParams {
  const void* logits;
  const uint8_t* mask;  // [tokens] 0: the token is not routed; nullptr: all are
  float* weight;        // [tokens, top_k]
  int32_t* idx;         // [tokens, top_k]
  int32_t* counts;      // [experts]
  float* loss;          // []
  float* balance;       // [experts] d loss / d (sum over tokens of the expert's probability)
  float* part_sum;      // [blocks, experts] workspace: probability sums of a block's tokens
  int32_t* part_cnt;    // [blocks, experts]
  int32_t* part_routed; // [blocks]
  double* part_share;   // finishing workgroups' shares of the loss
  int32_t* part_done;   // finishing workgroups that are through
  int64_t tokens;
  int64_t rows_per_block;
  int32_t experts, top_k, normalize, fp32;
  int32_t vec;          // rows of logits start on 16 bytes and experts fill whole 16-byte pieces
  int32_t blocks;
};

struct RouteBwdParams {
  const void* logits;
  const float* weight;
  const int32_t* idx;
  const float* balance;
  const float* dweight;  // nullptr: no gradient of the weights
  const float* dloss;    // nullptr: no gradient of the loss
  void* dlogits;
  int64_t tokens;
  int32_t experts, top_k, normalize, fp32, vec;
};

struct PlanParams {
  const int32_t* idx;  // [slots]
  int32_t* offs;       // [experts]
  int32_t* dest;       // [slots]
  int32_t* hist;       // [blocks, experts] workspace
  int64_t slots;
  int64_t chunk;       // slots of a block
  int32_t experts, blocks, runs;
};

struct RowsParams {
  const void* in;        // dispatch: x [tokens, row]; gather: rows [slots, row]; combine_bwd: y [slots, row]
  const void* dout;      // combine_bwd: [tokens, row]
  const int32_t* dest;   // [tokens, top_k]
  const int32_t* offs;   // [experts] (only the last is read: rows from there on are zeroed)
  const float* weight;   // [tokens, top_k]; nullptr: ones
  void* out;
  float* dweight;        // combine_bwd: [tokens, top_k]
  int64_t tokens;
  int64_t slots;         // tokens * top_k
  int32_t top_k, experts;
  int32_t pieces;        // 16-byte pieces of a row
  int32_t fp32;
};

hipError_t launch_route_fwd(const RouteParams& p, int threads, hipStream_t s);
hipError_t launch_route_bwd(const RouteBwdParams& p, hipStream_t s);
hipError_t launch_plan(const PlanParams& p, hipStream_t s);
hipError_t launch_dispatch(const RowsParams& p, hipStream_t s);
hipError_t launch_gather_sum(const RowsParams& p, hipStream_t s);
hipError_t launch_combine_bwd(const RowsParams& p, hipStream_t s);

// Lanes that share one row of logits, and the logits each of them holds.
constexpr int route_values(int experts) { return experts <= 512 ? 8 : 16; }
constexpr int route_lanes(int experts) {
  int l = 1;
  while (l * route_values(experts) < experts) l *= 2;
  return l;
}

}  // namespace mdg
