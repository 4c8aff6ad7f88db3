// Device-side interface of the mixture-of-experts operators: launch functions (defined in
// experts.hip, rows.hip and route.hip) and their argument blocks.
#pragma once

#include "kernels.h"

namespace agg {

// ---- experts' products with few rows an expert
struct StreamArgs {
  const uint8_t* a;     // rows taken through x
  const uint8_t* b;     // n_experts x K x N
  uint16_t* c;          // slots x N (gated: N / 2) bfloat16
  int64_t N, K;
  ExpertArgs x;
  int strips, ksplit;   // strips of the output's columns; parts of K
  float* ws;            // ksplit > 1: ksplit x slots x N floats
  int64_t ws_bytes;
  uint32_t* counts;     // ksplit > 1: n_experts x strips counters, zero before and after
};

hipError_t launch_expert_stream(const StreamArgs& args, int dtype, hipStream_t stream);
// The tiled kernel: args as kEpiExperts reads them, tiles of bm x bn.
hipError_t launch_expert_tiles(const GemmArgs& args, int bm, int bn, int dtype, int grid, hipStream_t stream);

// ---- row operators
struct NormArgs {
  const void* x;              // rows x cols, float or bfloat16
  const uint16_t* residual;   // bfloat16 or null
  uint16_t* residual_out;     // bfloat16 or null
  const uint16_t* weight;     // bfloat16, or null: no norm, x (+ residual) itself is quantised
  void* out;                  // bfloat16 or e4m3
  float* scales;              // fp8: a scale per row, or null: `scale` for all
  int64_t rows, cols;
  int64_t ld_x, ld_r, ld_ro, ld_out;   // elements from one row to the next
  float eps, scale;
  int x_fp32, out_fp8;
};
hipError_t launch_norm(const NormArgs& a, int cus, hipStream_t stream);

struct CombineArgs {
  const uint16_t* y;          // slots x n bfloat16
  const int32_t* token_slot;  // tokens x top_k, -1: none
  const float* weights;       // tokens x top_k
  void* out;                  // tokens x n, bfloat16 or float
  int64_t tokens, n, slots;
  int top_k, out_fp32;
};
hipError_t launch_combine(const CombineArgs& a, hipStream_t stream);

// ---- routing
struct RouteArgs {
  const void* logits;         // tokens x experts, float or bfloat16
  const float* bias;          // experts, or null
  int32_t* ids;               // tokens x top_k
  float* weights;             // tokens x top_k
  int64_t tokens, ld;
  int experts, top_k, groups, top_groups;
  int logits_bf16, sigmoid, renorm;
  float scale;
};
hipError_t launch_route(const RouteArgs& a, hipStream_t stream);

// (token, choice) pairs of one block of the plan's kernels
constexpr int kPlanPairs = AGG_PLAN_PAIRS;
struct PlanArgs {
  const int32_t* ids;         // tokens x top_k
  int32_t* offsets;           // n_local + 1
  int32_t* slot_token;        // tokens * top_k
  int32_t* token_slot;        // tokens * top_k
  int32_t* work;              // (pairs / kPlanPairs + 1) x (n_local + 1)
  int64_t pairs;
  int top_k, first, n_local;
};
hipError_t launch_plan(const PlanArgs& a, hipStream_t stream);

}  // namespace agg
