// The C entry point of the product with an epilogue: checks, then one launch on the caller's stream.
#include "moe.h"
#include "plan.h"

using namespace agg;

#define HIP_TRY(expr)                                                                   \
  do {                                                                                  \
    hipError_t e_ = (expr);                                                             \
    if (e_ != hipSuccess) return fail(AGG_E_HIP, "%s: %s", #expr, hipGetErrorString(e_)); \
  } while (0)

extern "C" int linear(agg_ctx* ctx, int64_t m, int64_t n, int64_t k, int dtype, const void* a, int64_t ld_a,
                      const float* a_scale, const void* b, const float* b_scale, const void* bias, int act,
                      int residual_dtype, const void* residual, int64_t ld_residual, int out_dtype, void* out,
                      int64_t ld_out, agg_stream stream) {
  if (int rc = agg_check_linear_args(m, n, k, dtype, a, ld_a, a_scale, b, b_scale, bias, act, residual_dtype, residual,
                                     ld_residual, out_dtype, out, ld_out))
    return rc;
  if (!ctx) return fail(AGG_E_ARG, "ctx is NULL");
  HIP_TRY(hipSetDevice(ctx_device(ctx)));
  if (m == 0 || n == 0) return AGG_OK;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int eb = dtype == AGG_FP8_E4M3 ? 1 : 2;
  const ExpertArgs x{nullptr, nullptr, a_scale, b_scale, m, m, ld_a * eb, 1, 0};
  const LinearArgs y{static_cast<const uint16_t*>(bias), residual, out, ld_residual, ld_out, act,
                     residual_dtype == AGG_FP32, out_dtype == AGG_FP32};
  const int units = ctx_units(ctx);
  const TileShape forced = ctx_forced_tile(ctx);
  const int parts = ctx_forced_split(ctx);
  LinearShape shape = forced.bm ? split_linear(dtype, m, n, k, forced, parts ? parts : 1)
                                : choose_linear_shape(dtype, m, n, k, units);
  if (!forced.bm && !shape.stream && parts) shape = split_linear(dtype, m, n, k, shape.tile, parts);
  if (shape.stream) {
    StreamArgs t{static_cast<const uint8_t*>(a), static_cast<const uint8_t*>(b), nullptr, n, k, x, shape.strips,
                 shape.ksplit, nullptr, 0, nullptr, y};
    if (t.ksplit > 1) {
      t.ws_bytes = int64_t(t.ksplit) * m * n * int64_t(sizeof(float));
      if (int rc = ctx_moe_workspace(ctx, stream, size_t(t.ws_bytes), &t.ws, &t.counts)) return rc;
    }
    HIP_TRY(launch_linear_stream(t, dtype, s));
    return AGG_OK;
  }
  GemmArgs g{};
  g.a = static_cast<const uint8_t*>(a);
  g.b = static_cast<const uint8_t*>(b);
  g.N = n;
  g.K = k;
  g.M = m;
  g.n_col_tiles = int((n + shape.tile.bn - 1) / shape.tile.bn) * shape.ksplit;
  g.ksplit = shape.ksplit;
  g.kps = shape.kps;
  if (g.ksplit > 1) {
    if (int rc = ctx_moe_workspace(ctx, stream, size_t(g.ksplit) * size_t(m) * size_t(n) * sizeof(float), &g.ws, &g.scratch))
      return rc;
  }
  g.n_lists = g.list_cols = 1;
  g.scale = 1.0f;
  g.x = x;
  g.y = y;
  // (as moe_gemm's grid: no more workgroups than tiles, the same number on every XCD, two 64 x 64 tiles
  // on a compute unit)
  int64_t most = (m + shape.tile.bm - 1) / shape.tile.bm * int64_t(g.n_col_tiles);
  most = (most + kXcds - 1) / kXcds * kXcds;
  const int64_t room = int64_t(units) * (shape.tile.bm == 64 ? 2 : 1);
  const int grid = int(most < room ? most : room);
  HIP_TRY(launch_linear_tiles(g, shape.tile.bm, shape.tile.bn, dtype, grid, s));
  return AGG_OK;
}
