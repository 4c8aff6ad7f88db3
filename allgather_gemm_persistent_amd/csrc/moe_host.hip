// The C entry points of the mixture-of-experts operators: checks, then one or two launches on the
// caller's stream. What they use of the ctx, beside its device, is a workspace of the call's stream or
// capture (moe_gemm with a split K), so calls on several streams do not meet.
#include "moe.h"
#include "plan.h"

using namespace agg;

namespace {

#define HIP_TRY(expr)                                                                   \
  do {                                                                                  \
    hipError_t e_ = (expr);                                                             \
    if (e_ != hipSuccess) return fail(AGG_E_HIP, "%s: %s", #expr, hipGetErrorString(e_)); \
  } while (0)

hipStream_t S(agg_stream s) { return reinterpret_cast<hipStream_t>(s); }

int enter(const agg_ctx* ctx) {
  if (!ctx) return fail(AGG_E_ARG, "ctx is NULL");
  HIP_TRY(hipSetDevice(ctx_device(ctx)));
  return AGG_OK;
}

int norm_call(agg_ctx* ctx, const NormArgs& a, int x_dtype, int out_dtype, agg_stream stream) {
  if (int rc = agg_check_norm_args(a.rows, a.cols, x_dtype, a.x, a.ld_x, a.residual, a.ld_r, a.residual_out, a.ld_ro,
                                   a.weight, a.eps, out_dtype, a.out, a.ld_out, a.scales, a.scale))
    return rc;
  if (int rc = enter(ctx)) return rc;
  if (a.rows == 0 || a.cols == 0) return AGG_OK;
  HIP_TRY(launch_norm(a, ctx_units(ctx), S(stream)));
  return AGG_OK;
}

}  // namespace

extern "C" int rms_norm(agg_ctx* ctx, int64_t rows, int64_t cols, int x_dtype, const void* x, int64_t ld_x,
                        const void* residual, int64_t ld_residual, void* residual_out, int64_t ld_residual_out,
                        const void* weight, float eps, int out_dtype, void* out, int64_t ld_out, float* scales,
                        float scale, agg_stream stream) {
  if (!weight) return fail(AGG_E_ARG, "weight is NULL");
  const NormArgs a{x, static_cast<const uint16_t*>(residual), static_cast<uint16_t*>(residual_out),
                   static_cast<const uint16_t*>(weight), out, scales, rows, cols, ld_x, ld_residual, ld_residual_out,
                   ld_out, eps, scale, x_dtype == AGG_FP32, out_dtype == AGG_FP8_E4M3};
  return norm_call(ctx, a, x_dtype, out_dtype, stream);
}

extern "C" int quant_rows(agg_ctx* ctx, int64_t rows, int64_t cols, int x_dtype, const void* x, int64_t ld_x,
                          void* out, int64_t ld_out, float* scales, float scale, agg_stream stream) {
  const NormArgs a{x, nullptr, nullptr, nullptr, out, scales, rows, cols, ld_x, 0, 0, ld_out, 0.0f, scale,
                   x_dtype == AGG_FP32, 1};
  return norm_call(ctx, a, x_dtype, AGG_FP8_E4M3, stream);
}

extern "C" int moe_route(agg_ctx* ctx, int64_t tokens, int experts, int top_k, int logits_dtype, const void* logits,
                         int64_t ld, const float* bias, int score, int groups, int top_groups, int renorm,
                         float scale, int32_t* ids, float* weights, agg_stream stream) {
  if (int rc = agg_check_route_args(tokens, experts, top_k, logits_dtype, logits, ld, score, groups, top_groups, scale,
                                    ids, weights))
    return rc;
  if (int rc = enter(ctx)) return rc;
  if (tokens == 0) return AGG_OK;
  const RouteArgs a{logits, bias, ids, weights, tokens, ld, experts, top_k, groups, top_groups,
                    logits_dtype == AGG_BF16, score == AGG_SCORE_SIGMOID, renorm != 0, scale};
  HIP_TRY(launch_route(a, S(stream)));
  return AGG_OK;
}

extern "C" int moe_plan(agg_ctx* ctx, int64_t tokens, int top_k, const int32_t* ids, int first, int n_local,
                        int32_t* offsets, int32_t* slot_token, int32_t* token_slot, int32_t* work,
                        agg_stream stream) {
  if (int rc = agg_check_plan_args(tokens, top_k, ids, first, n_local, offsets, slot_token, token_slot, work)) return rc;
  if (int rc = enter(ctx)) return rc;
  const PlanArgs a{ids, offsets, slot_token, token_slot, work, tokens * top_k, top_k, first, n_local};
  HIP_TRY(launch_plan(a, S(stream)));
  return AGG_OK;
}

extern "C" int moe_gemm(agg_ctx* ctx, int64_t slots, int n_experts, int64_t n, int64_t k, int dtype, int gated,
                        int64_t a_rows, const void* a, int64_t ld_a, const float* a_scale, const int32_t* slot_token,
                        const void* b, const float* b_scale, const int32_t* offsets, void* out, agg_stream stream) {
  if (int rc = agg_check_moe_gemm_args(slots, n_experts, n, k, dtype, gated, a_rows, a, ld_a, a_scale, slot_token, b,
                                       b_scale, offsets, out))
    return rc;
  if (int rc = enter(ctx)) return rc;
  if (slots == 0 || n == 0) return AGG_OK;
  const int eb = dtype == AGG_FP8_E4M3 ? 1 : 2;
  const int64_t cols = gated ? 2 * n : n;
  const ExpertArgs x{offsets, slot_token, a_scale, b_scale, slots, a_rows, ld_a * eb, n_experts, gated != 0};
  const int units = ctx_units(ctx);
  const TileShape forced = ctx_forced_tile(ctx);
  const ExpertShape shape = forced.bm ? ExpertShape{false, 0, 0, forced}
                                      : choose_expert_shape(dtype, slots, n_experts, n, k, gated, units);
  if (shape.stream) {
    StreamArgs s{static_cast<const uint8_t*>(a), static_cast<const uint8_t*>(b), static_cast<uint16_t*>(out),
                 cols, k, x, shape.strips, shape.ksplit, nullptr, 0, nullptr};
    if (s.ksplit > 1) {
      s.ws_bytes = int64_t(s.ksplit) * slots * cols * int64_t(sizeof(float));
      if (int rc = ctx_moe_workspace(ctx, stream, size_t(s.ws_bytes), &s.ws, &s.counts)) return rc;
    }
    HIP_TRY(launch_expert_stream(s, dtype, S(stream)));
    return AGG_OK;
  }
  GemmArgs g{};
  g.a = static_cast<const uint8_t*>(a);
  g.b = static_cast<const uint8_t*>(b);
  g.c = static_cast<uint16_t*>(out);
  g.N = cols;
  g.K = k;
  g.M = slots;
  g.n_col_tiles = int((cols + shape.tile.bn - 1) / shape.tile.bn);
  g.ksplit = 1;
  g.kps = int((k * eb + 63) / 64);
  g.n_lists = g.list_cols = 1;
  g.scale = 1.0f;
  g.x = x;
  // no more workgroups than there can be tiles (every expert rounds its last row tile up), the same on
  // every XCD: the tiles are dealt to the XCDs in eighths
  int64_t most = (slots / shape.tile.bm + n_experts) * int64_t(g.n_col_tiles);
  most = (most + kXcds - 1) / kXcds * kXcds;
  // (64 x 64 tiles: two workgroups fit on a compute unit, so one's start and end hide behind the other's
  // main loop)
  const int64_t room = int64_t(units) * (shape.tile.bm == 64 ? 2 : 1);
  const int grid = int(most < room ? most : room);
  HIP_TRY(launch_expert_tiles(g, shape.tile.bm, shape.tile.bn, dtype, grid, S(stream)));
  return AGG_OK;
}

extern "C" int moe_combine(agg_ctx* ctx, int64_t tokens, int top_k, int64_t n, int64_t slots, const void* y,
                           const int32_t* token_slot, const float* weights, int out_dtype, void* out,
                           agg_stream stream) {
  if (int rc = agg_check_combine_args(tokens, top_k, n, slots, y, token_slot, weights, out_dtype, out)) return rc;
  if (int rc = enter(ctx)) return rc;
  if (tokens == 0 || n == 0) return AGG_OK;
  const CombineArgs a{static_cast<const uint16_t*>(y), token_slot, weights, out, tokens, n, slots, top_k,
                      out_dtype == AGG_FP32};
  HIP_TRY(launch_combine(a, S(stream)));
  return AGG_OK;
}
