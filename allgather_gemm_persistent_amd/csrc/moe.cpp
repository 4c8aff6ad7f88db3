// The mixture-of-experts operators' host side that needs no GPU: argument checks and the choice of
// the experts' kernel.
#include <algorithm>
#include <cmath>

#include "plan.h"

namespace agg {

// The streaming kernel's and the tiles' limits and times below are fits to measured calls of 8
// experts of 8192 x 7168 and 3584 x 8192, 30 of 1000 x 1032 and 32 of 2048 x 1536, with 1 to 384 rows
// an expert, bf16 and fp8.
ExpertShape choose_expert_shape(int dtype, int64_t slots, int n_experts, int64_t n, int64_t k, int gated, int units) {
  ExpertShape r{false, 0, 1, {64, 64}};
  const bool fp8 = dtype == AGG_FP8_E4M3;
  const int64_t cols = gated ? 2 * n : n;
  // rows an expert holds if the slots are spread evenly over the experts that can hold any
  const int64_t busy = std::max<int64_t>(1, std::min<int64_t>(n_experts, slots));
  const double rows = double(slots) / double(busy);
  // Streaming takes 32 rows at a time: up to 16 on average nearly every expert needs one reading of
  // its weight (bf16 8192 x 7168, 16 rows: 159 us against 207 in tiles of 128 x 128; 24 rows: 261
  // against 210). A short K leaves each of its 8 waves too few blocks (K = 1000: 25 us against 20).
  if (rows <= 16 && k * (fp8 ? 1 : 2) >= 2048) {
    r.stream = true;
    const int64_t width = fp8 ? 256 : 128;
    r.strips = int((n + width - 1) / width);
    // fewer workgroups than 3/4 of the compute units: K in parts of 16 blocks of 32 or more, as many
    // as fill the units
    const int64_t groups = busy * r.strips;
    if (groups * 4 < int64_t(units) * 3 && int64_t(n_experts) * r.strips <= kMoeCounters) {
      int64_t parts = std::min<int64_t>({units / groups, (k + 511) / 512, 16});
      parts = std::min(parts, kMoeWsBytes / std::max<int64_t>(1, slots * cols * 4));
      r.ksplit = int(std::max<int64_t>(parts, 1));
    }
    return r;
  }
  // Tiles: waves of the grid times a wave's microseconds, a start and a rate per 2 bytes of K. An
  // expert's rows scatter around their mean, so its row tiles are counted at the mean and a deviation
  // to either side.
  struct Time { TileShape s; double start, bf16, bf16_gated, fp8, fp8_gated; };
  static const Time times[] = {
      {{256, 256}, 14, 0.0245, 0.0245, 0.0185, 0.0195}, {{256, 224}, 14, 0.0215, 0.0250, 0.0190, 0.0225},
      {{128, 128}, 3, 0.0115, 0.0118, 0.0118, 0.0150},  {{128, 64}, 2, 0.0062, 0.0092, 0.0074, 0.0120},
      {{64, 64}, 2, 0.0061, 0.0088, 0.0066, 0.0115}};
  const double spread = 1.2 * std::sqrt(rows);
  double best = 1e300;
  for (const Time& t : times) {
    double per = 0;
    for (double d : {-spread, 0.0, spread}) per += std::max(1.0, std::ceil((rows + d) / t.s.bm)) / 3;
    const double tiles = double(busy) * per * double((cols + t.s.bn - 1) / t.s.bn);
    const double rate = fp8 ? (gated ? t.fp8_gated : t.fp8) : (gated ? t.bf16_gated : t.bf16);
    const double cost = std::ceil(tiles / units) * (t.start + rate * double(k) * (fp8 ? 0.5 : 1.0));
    if (cost < best) {
      best = cost;
      r.tile = t.s;
    }
  }
  return r;
}

}  // namespace agg

using namespace agg;

namespace {

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

int need(const void* p, const char* what) {
  if (!p) return fail(AGG_E_ARG, "%s is NULL", what);
  if (misaligned(p)) return fail(AGG_E_ARG, "%s is not 16-byte aligned", what);
  return AGG_OK;
}

constexpr int64_t kMostRows = int64_t(1) << 30;

#define CHECK(expr)                  \
  do {                               \
    if (int rc_ = (expr)) return rc_; \
  } while (0)

// elements from one row to the next: at least `cols`, and rows that start on 16 bytes
int check_stride(int64_t ld, int64_t cols, int elem, const char* what) {
  if (ld < cols) return fail(AGG_E_ARG, "%s: a row stride of %lld is below the %lld columns", what, (long long)ld, (long long)cols);
  if ((ld * elem) % 16) return fail(AGG_E_ARG, "%s: a row stride of %lld bytes is not a multiple of 16", what, (long long)(ld * elem));
  return AGG_OK;
}

}  // namespace

extern "C" int agg_check_norm_args(int64_t rows, int64_t cols, int x_dtype, const void* x, int64_t ld_x,
                                   const void* residual, int64_t ld_residual, const void* residual_out,
                                   int64_t ld_residual_out, const void* weight, float eps, int out_dtype,
                                   const void* out, int64_t ld_out, const float* scales, float scale) {
  clear_error();
  if (rows < 0 || cols < 0) return fail(AGG_E_ARG, "negative size");
  if (x_dtype != AGG_BF16 && x_dtype != AGG_FP32) return fail(AGG_E_ARG, "x has dtype %d, not bf16 or fp32", x_dtype);
  if (out_dtype != AGG_BF16 && out_dtype != AGG_FP8_E4M3) return fail(AGG_E_ARG, "out has dtype %d, not bf16 or fp8", out_dtype);
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(AGG_E_ARG, "eps is negative or not finite");
  if (out_dtype == AGG_FP8_E4M3 && !scales && (!(scale > 0.0f) || !std::isfinite(scale)))
    return fail(AGG_E_ARG, "scale is not positive and finite");
  if (residual_out && !residual) return fail(AGG_E_ARG, "residual_out without a residual");
  if (cols % 8) return fail(AGG_E_ARG, "cols %lld is not a multiple of 8", (long long)cols);
  if (rows > kMostRows || cols > AGG_MAX_NORM_COLS)
    return fail(AGG_E_UNSUPPORTED, "%lld x %lld is beyond 2^30 rows or %d columns", (long long)rows, (long long)cols, AGG_MAX_NORM_COLS);
  if (rows == 0 || cols == 0) return AGG_OK;
  CHECK(need(x, "x"));
  CHECK(need(out, "out"));
  CHECK(check_stride(ld_x, cols, x_dtype == AGG_FP32 ? 4 : 2, "x"));
  if (ld_out < cols || ld_out % 8) return fail(AGG_E_ARG, "out: a row stride of %lld is below the columns or no multiple of 8", (long long)ld_out);
  if (weight && misaligned(weight)) return fail(AGG_E_ARG, "weight is not 16-byte aligned");
  if (residual) {
    CHECK(need(residual, "residual"));
    CHECK(check_stride(ld_residual, cols, 2, "residual"));
  }
  if (residual_out) {
    CHECK(need(residual_out, "residual_out"));
    CHECK(check_stride(ld_residual_out, cols, 2, "residual_out"));
  }
  return AGG_OK;
}

extern "C" int agg_check_route_args(int64_t tokens, int experts, int top_k, int logits_dtype, const void* logits,
                                    int64_t ld, int score, int groups, int top_groups, float scale,
                                    const int32_t* ids, const float* weights) {
  clear_error();
  if (tokens < 0) return fail(AGG_E_ARG, "negative size");
  if (experts < 1 || experts > AGG_MAX_EXPERTS) return fail(AGG_E_ARG, "%d experts, not 1 to %d", experts, AGG_MAX_EXPERTS);
  if (logits_dtype != AGG_BF16 && logits_dtype != AGG_FP32) return fail(AGG_E_ARG, "logits have dtype %d, not bf16 or fp32", logits_dtype);
  if (score != AGG_SCORE_SOFTMAX && score != AGG_SCORE_SIGMOID) return fail(AGG_E_ARG, "unknown score %d", score);
  if (groups < 1 || groups > AGG_MAX_GROUPS || experts % groups)
    return fail(AGG_E_ARG, "%d groups: 1 to %d that divide %d experts are wanted", groups, AGG_MAX_GROUPS, experts);
  if (top_groups < 1 || top_groups > groups) return fail(AGG_E_ARG, "top_groups %d not in [1, %d]", top_groups, groups);
  if (top_k < 1 || top_k > AGG_MAX_TOP_K || top_k > top_groups * (experts / groups))
    return fail(AGG_E_ARG, "top_k %d: 1 to %d, and no more than the experts of the kept groups", top_k, AGG_MAX_TOP_K);
  if (!std::isfinite(scale)) return fail(AGG_E_ARG, "scale is not finite");
  if (ld < experts) return fail(AGG_E_ARG, "a row stride of %lld is below the %d experts", (long long)ld, experts);
  if (tokens > kMostRows) return fail(AGG_E_UNSUPPORTED, "tokens beyond 2^30");
  if (tokens == 0) return AGG_OK;
  if (!logits || !ids || !weights) return fail(AGG_E_ARG, "logits, ids or weights is NULL");
  return AGG_OK;
}

extern "C" int agg_check_plan_args(int64_t tokens, int top_k, const int32_t* ids, int first, int n_local,
                                   const int32_t* offsets, const int32_t* slot_token, const int32_t* token_slot,
                                   const int32_t* work) {
  clear_error();
  if (tokens < 0) return fail(AGG_E_ARG, "negative size");
  if (top_k < 1 || top_k > AGG_MAX_TOP_K) return fail(AGG_E_ARG, "top_k %d not in [1, %d]", top_k, AGG_MAX_TOP_K);
  if (first < 0) return fail(AGG_E_ARG, "first %d is negative", first);
  if (n_local < 1 || n_local > AGG_MAX_EXPERTS) return fail(AGG_E_ARG, "n_local %d not in [1, %d]", n_local, AGG_MAX_EXPERTS);
  if (tokens * top_k > kMostRows || (tokens * top_k / AGG_PLAN_PAIRS + 1) * (n_local + 1) >= (int64_t(1) << 31))
    return fail(AGG_E_UNSUPPORTED, "%lld pairs are too many", (long long)(tokens * top_k));
  if (!offsets) return fail(AGG_E_ARG, "offsets is NULL");
  if (tokens == 0) return AGG_OK;
  if (!ids || !slot_token || !token_slot || !work) return fail(AGG_E_ARG, "ids, slot_token, token_slot or work is NULL");
  return AGG_OK;
}

extern "C" int agg_check_moe_gemm_args(int64_t slots, int n_experts, int64_t n, int64_t k, int dtype, int gated,
                                       int64_t a_rows, const void* a, int64_t ld_a, const float* a_scale,
                                       const int32_t* slot_token, const void* b, const float* b_scale,
                                       const int32_t* offsets, const void* out) {
  clear_error();
  if (slots < 0 || n < 0 || k < 0 || a_rows < 0) return fail(AGG_E_ARG, "negative size");
  if (n_experts < 1 || n_experts > AGG_MAX_EXPERTS) return fail(AGG_E_ARG, "%d experts, not 1 to %d", n_experts, AGG_MAX_EXPERTS);
  if (dtype != AGG_BF16 && dtype != AGG_FP8_E4M3) return fail(AGG_E_ARG, "unknown dtype %d", dtype);
  const int eb = dtype == AGG_FP8_E4M3 ? 1 : 2;
  if ((k * eb) % 16) return fail(AGG_E_ARG, "k * %d bytes = %lld is not a multiple of 16", eb, (long long)(k * eb));
  if ((n * eb) % 16 || n % 8) return fail(AGG_E_ARG, "n %lld: rows of b and out are multiples of 16 bytes", (long long)n);
  if (slots > kMostRows || a_rows > kMostRows || n > kMostRows || k > kMostRows) return fail(AGG_E_UNSUPPORTED, "dimension beyond 2^30");
  if (k * n * (gated ? 2 : 1) * eb >= (int64_t(1) << 31)) return fail(AGG_E_UNSUPPORTED, "one expert's weight is 2 GiB or more");
  if (slots == 0 || n == 0) return AGG_OK;
  CHECK(need(offsets, "offsets"));
  CHECK(need(out, "out"));
  if (k == 0) return fail(AGG_E_ARG, "k is 0");
  CHECK(need(a, "a"));
  CHECK(need(b, "b"));
  CHECK(check_stride(ld_a, k, eb, "a"));
  if (a_rows < 1) return fail(AGG_E_ARG, "a has no rows");
  if (!slot_token && a_rows < slots) return fail(AGG_E_ARG, "a has %lld rows for %lld slots", (long long)a_rows, (long long)slots);
  if ((slot_token ? a_rows : 256) * ld_a * eb >= (int64_t(1) << 31))
    return fail(AGG_E_UNSUPPORTED, "rows of a taken through slot_token span 2 GiB or more (or 256 rows do)");
  if (dtype == AGG_FP8_E4M3) {
    if (!a_scale) return fail(AGG_E_ARG, "a_scale is NULL");
    CHECK(need(b_scale, "b_scale"));
  }
  return AGG_OK;
}

extern "C" int agg_check_combine_args(int64_t tokens, int top_k, int64_t n, int64_t slots, const void* y,
                                      const int32_t* token_slot, const float* weights, int out_dtype,
                                      const void* out) {
  clear_error();
  if (tokens < 0 || n < 0 || slots < 0) return fail(AGG_E_ARG, "negative size");
  if (top_k < 1 || top_k > AGG_MAX_TOP_K) return fail(AGG_E_ARG, "top_k %d not in [1, %d]", top_k, AGG_MAX_TOP_K);
  if (out_dtype != AGG_BF16 && out_dtype != AGG_FP32) return fail(AGG_E_ARG, "out has dtype %d, not bf16 or fp32", out_dtype);
  if (n % 8) return fail(AGG_E_ARG, "n %lld is not a multiple of 8", (long long)n);
  if (tokens > kMostRows || n > kMostRows || slots > kMostRows) return fail(AGG_E_UNSUPPORTED, "dimension beyond 2^30");
  if (tokens == 0 || n == 0) return AGG_OK;
  if (!token_slot || !weights) return fail(AGG_E_ARG, "token_slot or weights is NULL");
  if (slots > 0) CHECK(need(y, "y"));
  CHECK(need(out, "out"));
  return AGG_OK;
}

extern "C" int agg_moe_gemm_shape(int dtype, int64_t slots, int n_experts, int64_t n, int64_t k, int gated,
                                  int* ksplit, int* bm, int* bn) {
  clear_error();
  if (!ksplit || !bm || !bn) return fail(AGG_E_ARG, "agg_moe_gemm_shape: NULL output");
  const ExpertShape s = choose_expert_shape(dtype, slots, std::max(n_experts, 1), n, k, gated, 256);
  *ksplit = s.stream ? s.ksplit : 0;
  *bm = s.stream ? 0 : s.tile.bm;
  *bn = s.stream ? 0 : s.tile.bn;
  return AGG_OK;
}
