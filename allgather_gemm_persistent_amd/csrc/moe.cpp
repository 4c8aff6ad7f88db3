// The mixture-of-experts operators' host side that needs no GPU: argument checks and the choice of
// the experts' kernel.
#include <algorithm>
#include <cmath>

#include "plan.h"

namespace agg {

namespace {

// Microseconds of a tile over all of K: a start and a rate per two bytes of K.
struct TileTime {
  double start, rate;
  double at(double k2) const { return start + rate * k2; }
};

double ceil_div(double a, double b) { return std::ceil(a / b); }

}  // namespace

// The kernel whose time is expected to be the least. The times are fits to measured calls (8 experts of
// 8192 x 7168 and 3584 x 8192, 8 of 1024 x 4096, 30 of 1000 x 1032, 32 of 2048 x 1536, 60 of 256 x
// 2816; 1 to 400 rows an expert, bf16 and fp8). Against every kernel forced, the choice is within 10% of
// the fastest in 68 of 84 such calls and in 36 of 40 random ones; it takes 4.9% and 3.3% longer on
// average and at worst 1.51 times as long (32 experts of 2048 x 1536 bf16, 192 rows each). What the fits
// stand for, at 8 experts of 8192 x 7168 bf16, us:
//   rows an expert      4    16    48    96   192   384
//   streaming         152   159   329   620  1128  2139
//   256 x 256 tiles   175   174   175   184   211   404
//   128 x 128         202   207   217   226   377   615
//   64 x 64           297   309   325   520   710  1277
// and at 30 of 1000 x 1032, 16 rows: streaming 26, 64 x 64 19, 256 x 256 22.
ExpertShape choose_expert_shape(int dtype, int64_t slots, int n_experts, int64_t n, int64_t k, int gated, int units) {
  ExpertShape r{false, 0, 1, {64, 64}};
  const bool fp8 = dtype == AGG_FP8_E4M3;
  const int64_t cols = gated ? 2 * n : n;
  // rows an expert holds if the slots are spread evenly over the experts that can hold any; they scatter
  // around that
  const int64_t busy = std::max<int64_t>(1, std::min<int64_t>(n_experts, slots));
  const double rows = double(slots) / double(busy), spread = std::sqrt(rows);
  const double k2 = double(k) * (fp8 ? 0.5 : 1.0);             // K in units of two bytes
  const double bytes = double(busy) * double(k) * double(cols) * (fp8 ? 1.0 : 2.0);
  const double u = units;

  // Streaming: the weights at 6.2 TB/s, or a compute unit's 160 pieces of rows a microsecond; read again
  // for every 32 rows of the fullest expert. Strips fewer than 3/4 of the units: K in parts of 16 blocks
  // of 32 or more, as many as fill the units.
  const int64_t width = fp8 ? 256 : 128;
  const int64_t strips = (n + width - 1) / width, groups = busy * strips;
  int64_t parts = 1;
  if (groups * 4 < int64_t(units) * 3 && int64_t(n_experts) * strips <= kMoeCounters) {
    parts = std::min<int64_t>({units / groups, (k + 511) / 512, 16});
    parts = std::max<int64_t>(1, std::min(parts, kMoeWsBytes / std::max<int64_t>(1, slots * cols * 4)));
  }
  const double passes = ceil_div(2 * rows + 2 * spread, 32);   // (the fullest of unevenly liked experts)
  const double stream = passes * std::max(bytes / 6.2e6 + 3, ceil_div(double(groups * parts), u) *
                                                                 (5.7 + double(k) * (gated ? 2 : 1) / (160.0 * double(parts))));

  // Tiles: waves of the grid times a tile's microseconds, or the weights at 5.4 TB/s. The 256-row shapes
  // have whole tiles and, for an expert's last 64 or 128 rows, low ones.
  struct Shape { TileShape s; TileTime whole, half, quarter; };
  const double g = gated ? 1.25 : 1.0;                         // narrow tiles: gate and up pieces apart
  const Shape shapes[] = {
      {{256, 256}, fp8 ? TileTime{22, 0.0247} : TileTime{14, 0.0235}, fp8 ? TileTime{14, 0.016} : TileTime{10, 0.016},
       fp8 ? TileTime{12.5, 0.0107} : TileTime{9, 0.0128}},
      {{256, 224}, {13, 0.0206 * (gated ? 1.15 : 1.0)}, {10, 0.015 * g}, {9, 0.0125 * g}},
      {{128, 128}, {5, fp8 ? 0.0135 : 0.0118}, {}, {}},
      {{128, 64}, {3, fp8 ? 0.0072 * g : 0.0068 * g}, {}, {}},
      {{64, 64}, {2.5, fp8 ? 0.0066 * g : 0.0068 * g}, {}, {}}};
  double best = 1e300;
  for (const Shape& t : shapes) {
    // (in fp8 a tile of 256 x 224 takes as long as one of 256 x 256: 1015 and 834 us at 16384 even rows of
    // 8 experts of 8192 x 7168; a forced tile alone takes it)
    if (fp8 && t.s.bn == 224) continue;
    const double across = double((cols + t.s.bn - 1) / t.s.bn) * double(busy) / 3.0;
    double whole = 0, half = 0, quarter = 0;                   // tiles, over rows - spread, rows, rows + spread
    for (double d : {-spread, 0.0, spread}) {
      const double held = std::max(1.0, std::ceil(rows + d)), full = std::floor(held / t.s.bm), rest = held - full * t.s.bm;
      whole += full * across;
      if (rest == 0) continue;
      if (t.s.bm < 256 || rest > 128) whole += across;
      else if (rest > 64) half += across;
      else quarter += across;
    }
    const double tw = t.whole.at(k2), th = t.half.at(k2), tq = t.quarter.at(k2);
    // (a long launch is bound by power: a partly filled last wave costs its share, not a whole one)
    const double waves = whole > 2 * u && t.s.bm > 64 ? whole / u + 0.15 : ceil_div(whole, u), low = half + quarter;
    double cost = waves * tw;
    // (64 x 64 tiles run two to a compute unit: later ones save most of their start)
    if (t.s.bm == 64) cost -= (waves - 1) * std::min(2.5, 0.45 * tw);
    if (low > 0) {
      // the workgroups that are a whole tile short take up to two low ones, all take the others
      const double tl = (half * th + quarter * tq) / low, spare = waves * u - whole;
      const double turns = spare > 0 ? std::min(2.0, ceil_div(low, spare)) : 0.0;
      const double others = std::max(0.0, ceil_div(low - turns * spare, u));
      cost = std::max(cost, std::max(waves - 1, 0.0) * tw + turns * tl) + others * tl;
      cost = std::max({cost, half > 0 ? th : 0.0, quarter > 0 ? tq : 0.0});
    }
    cost = std::max(cost, bytes / 5.4e6 + 3);
    if (cost < best) {
      best = cost;
      r.tile = t.s;
    }
  }
  if (stream < best) {
    r.stream = true;
    r.strips = int(strips);
    r.ksplit = int(parts);
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
constexpr int64_t kMostStride = int64_t(1) << 31;

#define CHECK(expr)                  \
  do {                               \
    if (int rc_ = (expr)) return rc_; \
  } while (0)

// elements from one row to the next: at least `cols`, and rows that start on 16 bytes
int check_stride(int64_t ld, int64_t cols, int elem, const char* what) {
  if (ld < cols) return fail(AGG_E_ARG, "%s: a row stride of %lld is below the %lld columns", what, (long long)ld, (long long)cols);
  if (ld > kMostStride) return fail(AGG_E_UNSUPPORTED, "%s: a row stride of %lld is beyond 2^31", what, (long long)ld);
  if ((ld * elem) % 16) return fail(AGG_E_ARG, "%s: a row stride of %lld bytes is not a multiple of 16", what, (long long)(ld * elem));
  return AGG_OK;
}

// what moe_gemm takes of its sizes
int check_moe_sizes(int64_t slots, int n_experts, int64_t n, int64_t k, int dtype, int gated, int64_t a_rows) {
  if (slots < 0 || n < 0 || k < 0 || a_rows < 0) return fail(AGG_E_ARG, "negative size");
  if (n_experts < 1 || n_experts > AGG_MAX_EXPERTS) return fail(AGG_E_ARG, "%d experts, not 1 to %d", n_experts, AGG_MAX_EXPERTS);
  if (dtype != AGG_BF16 && dtype != AGG_FP8_E4M3) return fail(AGG_E_ARG, "unknown dtype %d", dtype);
  const int eb = dtype == AGG_FP8_E4M3 ? 1 : 2;
  if ((k * eb) % 16) return fail(AGG_E_ARG, "k * %d bytes = %lld is not a multiple of 16", eb, (long long)(k * eb));
  if ((n * eb) % 16 || n % 8) return fail(AGG_E_ARG, "n %lld: rows of b and out are multiples of 16 bytes", (long long)n);
  if (slots > kMostRows || a_rows > kMostRows || n > kMostRows || k > kMostRows) return fail(AGG_E_UNSUPPORTED, "dimension beyond 2^30");
  if (k * n * (gated ? 2 : 1) * eb >= (int64_t(1) << 31)) return fail(AGG_E_UNSUPPORTED, "one expert's weight is 2 GiB or more");
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
  if (ld_out > kMostStride) return fail(AGG_E_UNSUPPORTED, "out: a row stride of %lld is beyond 2^31", (long long)ld_out);
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
  if (tokens > kMostRows || ld > kMostStride) return fail(AGG_E_UNSUPPORTED, "tokens beyond 2^30 or a row stride beyond 2^31");
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
  if (tokens > kMostRows || tokens * top_k > kMostRows || (tokens * top_k / AGG_PLAN_PAIRS + 1) * (n_local + 1) >= (int64_t(1) << 31))
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
  CHECK(check_moe_sizes(slots, n_experts, n, k, dtype, gated, a_rows));
  const int eb = dtype == AGG_FP8_E4M3 ? 1 : 2;
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
  CHECK(check_moe_sizes(slots, n_experts, n, k, dtype, gated, 0));
  // (a product without columns has no strips to divide the units among)
  const ExpertShape s = choose_expert_shape(dtype, slots, n_experts, std::max<int64_t>(n, 1), k, gated, 256);
  *ksplit = s.stream ? s.ksplit : 0;
  *bm = s.stream ? 0 : s.tile.bm;
  *bn = s.stream ? 0 : s.tile.bn;
  return AGG_OK;
}
