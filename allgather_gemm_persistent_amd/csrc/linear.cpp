// The product with an epilogue: what of its host side needs no GPU.
#include <algorithm>
#include <cmath>

#include "plan.h"

namespace agg {

LinearShape split_linear(int dtype, int64_t m, int64_t n, int64_t k, TileShape tile, int parts) {
  const int64_t slices = (k * (dtype == AGG_FP8_E4M3 ? 1 : 2) + 63) / 64, pairs = (slices + 1) / 2;
  const int64_t tiles = (m + tile.bm - 1) / tile.bm * ((n + tile.bn - 1) / tile.bn);
  int64_t p = std::max<int64_t>(1, std::min<int64_t>(parts, pairs));
  if (tile.bm * tile.bn > kMaxSplitTileArea || tiles > kMoeCounters) p = 1;
  if (p > 1) p = std::min<int64_t>(p, std::max<int64_t>(1, kLinearWsBytes / std::max<int64_t>(1, m * n * 4)));
  const int64_t each = (pairs + p - 1) / p;                    // slice pairs of a part
  p = std::max<int64_t>(1, (pairs + each - 1) / std::max<int64_t>(each, 1));
  return LinearShape{false, 0, int(p), int(p > 1 ? 2 * each : slices), tile};
}

// The kernel whose time is expected to be the least, us. The times are fits to measured calls of 1 to 4096 rows, bf16 and
// fp8; what they stand for, us (parts of K in brackets; the choice is within 8% of the fastest in 29 of 34 such calls):
//   rows x columns x K bf16    streaming   64 x 64        128 x 64      128 x 128     256 x 256
//   16 x 1024 x 8192            11.4 (16)  26.0, 11.9 (8)
//   48 x 8192 x 8192            52         34.3, 30.4 (2)  39.9, 31.0 (2) 55.3, 32.3 (4)
//   128 x 2048 x 8192           72         33.8, 17.7 (4)  41.9, 22.9 (4) 58.0, 31.9 (4)  99.0
//   128 x 8192 x 8192                      38.8, 46.2 (2)  50.0, 40.4 (2) 63.6, 42.4 (4) 104.8
//   512 x 8192 x 8192                     125.4           116.7           80.0          154.4
//   4096 x 8192 x 8192                    984             753            570            412
LinearShape choose_linear_shape(int dtype, int64_t m, int64_t n, int64_t k, int units) {
  const bool fp8 = dtype == AGG_FP8_E4M3;
  const int eb = fp8 ? 1 : 2;
  const double u = units, k2 = double(k) * eb / 2, bytes = double(k) * double(n) * eb;
  auto ceil_div = [](double a, double b) { return std::ceil(a / b); };

  // Streaming: as moe_gemm's of one expert
  const int64_t width = fp8 ? 256 : 128, strips = (n + width - 1) / width;
  int64_t parts = 1;
  if (strips * 4 < int64_t(units) * 3 && strips <= kMoeCounters) {
    parts = std::min<int64_t>({units / std::max<int64_t>(strips, 1), (k + 511) / 512, 16});
    parts = std::max<int64_t>(1, std::min(parts, kMoeWsBytes / std::max<int64_t>(1, m * n * 4)));
  }
  const double stream = ceil_div(double(m), 32) * std::max(bytes / 6.2e6 + 3, ceil_div(double(strips * parts), u) *
                                                           (5.7 + double(k) / (160.0 * double(parts))));
  LinearShape best{true, int(strips), int(parts), 0, {0, 0}};
  double least = stream;

  // Tiles: a start and a rate per two bytes of K, which grows as more compute units read beside each other. A split K adds
  // the parts' way through the workspace and the last part's sum, at what one compute unit reads; it pays only where the
  // parts have a unit each
  struct Shape { TileShape s; double start, alone, crowded; };
  const Shape shapes[] = {{{256, 256}, fp8 ? 22.0 : 14, fp8 ? 0.0247 : 0.0235, fp8 ? 0.0247 : 0.0235},
                          {{256, 224}, 13, 0.0206, 0.0240},
                          {{128, 128}, 5, fp8 ? 0.0068 : 0.0064, fp8 ? 0.0125 : 0.0092},
                          {{128, 64}, 3, fp8 ? 0.0065 : 0.0045, fp8 ? 0.0105 : 0.0072},
                          {{64, 64}, 2.5, fp8 ? 0.0055 : 0.0038, fp8 ? 0.0095 : 0.0044}};
  for (const Shape& t : shapes) {
    // (in fp8 a tile of 256 x 224 takes as long as one of 256 x 256)
    if (fp8 && t.s.bn == 224) continue;
    const double tiles = ceil_div(double(m), t.s.bm) * ceil_div(double(n), t.s.bn);
    for (int p = 1; p <= kMaxKSplit && (p == 1 || tiles * p <= u); ++p) {
      const LinearShape x = split_linear(dtype, m, n, k, t.s, p);
      if (x.ksplit != p) continue;
      const double rate = t.alone + (t.crowded - t.alone) * std::min(1.0, tiles * p / (0.6 * u));
      // (64 x 64 tiles: two on a unit, which read beside each other)
      const double waves = t.s.bm > 64 ? (tiles > 2 * u ? tiles / u + 0.15 : ceil_div(tiles * p, u)) : std::max(1.0, 1.12 * tiles * p / u);
      double cost = t.s.bm > 64 ? waves * (t.start + rate * k2 / p) : t.start + waves * rate * k2 / p;
      cost = std::max(cost, bytes / 5.4e6 + 3);
      if (p > 1) cost += 3.5 + p * double(t.s.bm * t.s.bn) * 4 / 55e3 + 8.0 * p * double(m) * double(n) / 4e6;
      if (cost < least) {
        least = cost;
        best = x;
      }
    }
  }
  return best;
}

}  // namespace agg

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
  const LinearShape s = choose_linear_shape(dtype, m, std::max<int64_t>(n, 1), k, 256);
  *ksplit = s.ksplit;
  *bm = s.stream ? 0 : s.tile.bm;
  *bn = s.stream ? 0 : s.tile.bn;
  return AGG_OK;
}
