// The product with an epilogue: what of its host side needs no GPU.
#include <algorithm>

#include "plan.h"

using namespace agg;

namespace {

constexpr int64_t kMostRows = int64_t(1) << 30;
constexpr int64_t kMostStride = int64_t(1) << 31;

#define CHECK(expr)                  \
  do {                               \
    if (int rc_ = (expr)) return rc_; \
  } while (0)

int need(const void* p, const char* what, uintptr_t align = 16) {
  if (!p) return fail(AGG_E_ARG, "%s is NULL", what);
  if (reinterpret_cast<uintptr_t>(p) & (align - 1)) return fail(AGG_E_ARG, "%s is not %d-byte aligned", what, int(align));
  return AGG_OK;
}

// elements from one row to the next: at least `cols`, and rows that start on 16 bytes
int check_rows(const void* p, int64_t ld, int64_t cols, int elem, const char* what) {
  CHECK(need(p, what));
  if (ld < cols) return fail(AGG_E_ARG, "%s: a row stride of %lld is below the %lld columns", what, (long long)ld, (long long)cols);
  if (ld > kMostStride) return fail(AGG_E_UNSUPPORTED, "%s: a row stride of %lld is beyond 2^31", what, (long long)ld);
  if ((ld * elem) % 16) return fail(AGG_E_ARG, "%s: a row stride of %lld bytes is not a multiple of 16", what, (long long)(ld * elem));
  return AGG_OK;
}

int check_sizes(int64_t m, int64_t n, int64_t k, int dtype) {
  if (m < 0 || n < 0 || k < 0) return fail(AGG_E_ARG, "negative size");
  if (dtype != AGG_BF16 && dtype != AGG_FP8_E4M3) return fail(AGG_E_ARG, "unknown dtype %d", dtype);
  const int eb = dtype == AGG_FP8_E4M3 ? 1 : 2;
  if (m > kMostRows || n > kMostRows || k > kMostRows) return fail(AGG_E_UNSUPPORTED, "dimension beyond 2^30");
  if ((k * eb) % 16) return fail(AGG_E_ARG, "k * %d bytes = %lld is not a multiple of 16", eb, (long long)(k * eb));
  if ((n * eb) % 16 || n % 8) return fail(AGG_E_ARG, "n %lld: rows of b and out are multiples of 16 bytes", (long long)n);
  if (k * n * eb >= (int64_t(1) << 31)) return fail(AGG_E_UNSUPPORTED, "b is 2 GiB or more");
  return AGG_OK;
}

int float_size(int dtype) { return dtype == AGG_FP32 ? 4 : dtype == AGG_BF16 ? 2 : 0; }

}  // namespace

extern "C" int agg_check_linear_args(int64_t m, int64_t n, int64_t k, int dtype, const void* a, int64_t ld_a,
                                     const float* a_scale, const void* b, const float* b_scale, const void* bias, int act,
                                     int residual_dtype, const void* residual, int64_t ld_residual, int out_dtype,
                                     const void* out, int64_t ld_out) {
  clear_error();
  CHECK(check_sizes(m, n, k, dtype));
  const int eb = dtype == AGG_FP8_E4M3 ? 1 : 2;
  if (act < AGG_ACT_NONE || act > AGG_ACT_GELU_TANH) return fail(AGG_E_ARG, "unknown activation %d", act);
  if (!float_size(out_dtype)) return fail(AGG_E_ARG, "out has dtype %d, not bf16 or fp32", out_dtype);
  if (residual && !float_size(residual_dtype)) return fail(AGG_E_ARG, "residual has dtype %d, not bf16 or fp32", residual_dtype);
  if (m == 0 || n == 0) return AGG_OK;
  if (k == 0) return fail(AGG_E_ARG, "k is 0");
  CHECK(check_rows(a, ld_a, k, eb, "a"));
  if (256 * ld_a * eb >= (int64_t(1) << 31)) return fail(AGG_E_UNSUPPORTED, "256 rows of a span 2 GiB or more");
  CHECK(need(b, "b"));
  if (dtype == AGG_FP8_E4M3) {
    CHECK(need(a_scale, "a_scale", 4));
    CHECK(need(b_scale, "b_scale"));
  }
  if (bias) CHECK(need(bias, "bias"));
  if (residual) CHECK(check_rows(residual, ld_residual, n, float_size(residual_dtype), "residual"));
  CHECK(check_rows(out, ld_out, n, float_size(out_dtype), "out"));
  if (out == residual && (residual_dtype != out_dtype || (ld_out != ld_residual && m > 1)))
    return fail(AGG_E_ARG, "out is the residual at another type or stride");
  return AGG_OK;
}

extern "C" int agg_linear_shape(int dtype, int64_t m, int64_t n, int64_t k, int* ksplit, int* bm, int* bn) {
  clear_error();
  if (!ksplit || !bm || !bn) return fail(AGG_E_ARG, "agg_linear_shape: NULL output");
  CHECK(check_sizes(m, n, k, dtype));
  // (a product without columns has no strips to divide the units among)
  const ExpertShape s = choose_expert_shape(dtype, m, 1, std::max<int64_t>(n, 1), k, 0, 256, true);
  *ksplit = s.stream ? s.ksplit : 0;
  *bm = s.stream ? 0 : s.tile.bm;
  *bn = s.stream ? 0 : s.tile.bn;
  return AGG_OK;
}
