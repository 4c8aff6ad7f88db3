// The attention operators' host side that needs no GPU: argument checks.
#include <algorithm>
#include <cmath>

#include "plan.h"

namespace agg {

// compute units that paged_attn counts on: up to 512 workgroups, so that a row's parts (two a workgroup at most) are joined
// in two steps of 32, and the counters (eight a workgroup and two) suffice
constexpr int kAttnUnits = 256;
static_assert(16 * kAttnUnits + 2 <= kWsCounters, "paged_attn's counters");

AttnShape choose_attn_shape(const agg_kv_cache& cache, int64_t rows, int q_heads, int64_t seq_pages, int64_t window,
                            int units) {
  const int group = q_heads / cache.kv_heads, dim = cache.head_dim;
  // as many of a head's queries at once as there are (a head's keys and values are read again for more), up to what the
  // registers nearly hold: 33 to 64 of 128 channels in bf16 spill 27 to 38 registers, 17 and more of 256 channels 73. Half as
  // many at once and a second reading spill none and cost where reading counts: 32 rows of 8000 tokens on 2 heads 65 -> 85 us
  // (48 queries of 128), 128 -> 179 (24 of 256); they gain where joins do: 4 rows of 2000 on one head 42 -> 18, 47 -> 31
  const int most = dim > 128 ? 2 : 4;
  AttnShape s;
  s.row_tiles = group <= 16 ? 1 : group <= 32 || most == 2 ? 2 : 4;
  // the grid: what the compute units hold at once
  s.grid = std::min(units, kAttnUnits) * (s.row_tiles == 1 && dim <= 128 ? 2 : 1);
  const int queries = std::min(group, 16 * s.row_tiles);
  s.slot_bytes = (queries * (dim + 4) * 4 + 15) / 16 * 16;
  const int64_t splits = (group + 16 * s.row_tiles - 1) / (16 * s.row_tiles), room = seq_pages * cache.page_size;
  s.row_most = ((window > 0 && window < room ? window : room) / 32 + 2) * cache.kv_heads * splits;
  // Results wait in the workspace where a row is split: at most four for every workgroup, and fewer than half as many
  // as there are tiles, since a part of a split row has four tiles or more but for the last
  const int64_t slots = std::min<int64_t>(4 * s.grid, std::max<int64_t>(1, rows * s.row_most / 2));
  s.ws_bytes = slots * s.slot_bytes;
  return s;
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

int check_cache(const agg_kv_cache* c) {
  if (!c) return fail(AGG_E_ARG, "cache is NULL");
  if (c->dtype != AGG_BF16 && c->dtype != AGG_FP8_E4M3) return fail(AGG_E_ARG, "the cache has dtype %d, not bf16 or fp8", c->dtype);
  const bool fp8 = c->dtype == AGG_FP8_E4M3;
  const int eb = fp8 ? 1 : 2;
  if (c->page_size < 16 || c->page_size > AGG_MAX_PAGE || c->page_size % 16)
    return fail(AGG_E_ARG, "page_size %d is not a multiple of 16 up to %d", c->page_size, AGG_MAX_PAGE);
  if (c->head_dim < 16 || c->head_dim > AGG_MAX_HEAD_DIM || c->head_dim % 16)
    return fail(AGG_E_ARG, "head_dim %d is not a multiple of 16 up to %d", c->head_dim, AGG_MAX_HEAD_DIM);
  if (c->kv_heads < 1 || c->kv_heads > AGG_MAX_HEADS) return fail(AGG_E_ARG, "%d heads, not 1 to %d", c->kv_heads, AGG_MAX_HEADS);
  if (c->pages < 0) return fail(AGG_E_ARG, "negative size");
  if (c->pages > kMostRows) return fail(AGG_E_UNSUPPORTED, "%lld pages are too many", (long long)c->pages);
  if (c->pages == 0) return AGG_OK;
  CHECK(need(c->k, "k of the cache"));
  CHECK(need(c->v, "v of the cache"));
  if (fp8) {
    CHECK(need(c->k_scale, "k_scale"));
    CHECK(need(c->v_scale, "v_scale"));
  }
  struct {
    int64_t ld, count;
    const char* what;
  } const strides[] = {{c->ld_page, c->pages, "ld_page"}, {c->ld_token, c->page_size, "ld_token"}, {c->ld_head, c->kv_heads, "ld_head"}};
  for (const auto& s : strides) {
    if (s.count == 1) continue;              // (never taken)
    if (s.ld < c->head_dim) return fail(AGG_E_ARG, "the cache's %s %lld is below head_dim", s.what, (long long)s.ld);
    if ((s.ld * eb) % 16) return fail(AGG_E_ARG, "the cache's %s of %lld bytes is not a multiple of 16", s.what, (long long)(s.ld * eb));
    // (a product with 2^30 pages stays inside 63 bits of bytes)
    if (s.ld > kMostStride) return fail(AGG_E_UNSUPPORTED, "the cache's %s %lld is beyond 2^31", s.what, (long long)s.ld);
  }
  // (16 tokens lie in one buffer descriptor)
  if (c->ld_token * eb > (int64_t(1) << 26)) return fail(AGG_E_UNSUPPORTED, "the cache's ld_token is beyond 2^26 bytes");
  return AGG_OK;
}

// (positions are 32-bit)
int check_table_size(const agg_kv_cache* c, int64_t seq_pages) {
  if (seq_pages > kMostRows || seq_pages * c->page_size > kMostRows)
    return fail(AGG_E_UNSUPPORTED, "a table's row of %lld pages is beyond 2^30 positions", (long long)seq_pages);
  return AGG_OK;
}

int check_table(const agg_kv_cache* c, const int32_t* table, int64_t seqs, int64_t seq_pages, int64_t ld_table) {
  if (seqs < 0 || seq_pages < 0) return fail(AGG_E_ARG, "negative size");
  if (seqs > kMostRows) return fail(AGG_E_UNSUPPORTED, "%lld sequences are beyond 2^30", (long long)seqs);
  CHECK(check_table_size(c, seq_pages));
  if (seqs == 0 || seq_pages == 0) return AGG_OK;
  if (seqs > 1 && ld_table < seq_pages) return fail(AGG_E_ARG, "ld_table %lld is below the %lld pages", (long long)ld_table, (long long)seq_pages);
  if (ld_table > kMostStride) return fail(AGG_E_UNSUPPORTED, "ld_table is beyond 2^31");
  return need(table, "table", 4);
}

// what paged_attn divides its work by
int check_attn_sizes(const agg_kv_cache* c, int64_t rows, int q_heads, int64_t seq_pages, int64_t window) {
  if (rows < 0 || window < 0 || seq_pages < 0) return fail(AGG_E_ARG, "negative size");
  CHECK(check_cache(c));
  if (q_heads < 1 || q_heads > AGG_MAX_HEADS || q_heads % c->kv_heads)
    return fail(AGG_E_ARG, "%d heads of queries: a multiple of the cache's %d up to %d is wanted", q_heads, c->kv_heads, AGG_MAX_HEADS);
  if (rows > kMostRows / 1024) return fail(AGG_E_UNSUPPORTED, "rows beyond 2^20");
  CHECK(check_table_size(c, seq_pages));
  // (the tiles of a row are counted in 31 bits)
  const int64_t room = seq_pages * c->page_size, splits = (q_heads / c->kv_heads + 15) / 16;
  if (((window > 0 && window < room ? window : room) / 32 + 2) * c->kv_heads * splits >= (int64_t(1) << 31))
    return fail(AGG_E_UNSUPPORTED, "%lld positions of %d heads are beyond 2^36", (long long)room, q_heads);
  return AGG_OK;
}

}  // namespace

extern "C" int agg_check_kv_write_args(const agg_kv_cache* cache, int64_t tokens, int q_heads, const void* q, int64_t ld_q,
                                       const void* q_out, int64_t ld_q_out, const void* k, int64_t ld_k, const void* v,
                                       int64_t ld_v, const float* rope, int64_t rope_rows, int rope_dim,
                                       int rope_pairs, const int32_t* positions, const int32_t* table, int64_t seqs,
                                       int64_t seq_pages, int64_t ld_table) {
  clear_error();
  if (tokens < 0 || rope_rows < 0) return fail(AGG_E_ARG, "negative size");
  CHECK(check_cache(cache));
  if (q_heads < 0 || q_heads > AGG_MAX_HEADS) return fail(AGG_E_ARG, "%d heads of queries, not 0 to %d", q_heads, AGG_MAX_HEADS);
  if (rope_dim < 0 || rope_dim > cache->head_dim || rope_dim % 16)
    return fail(AGG_E_ARG, "rope_dim %d is not a multiple of 16 up to head_dim %d", rope_dim, cache->head_dim);
  if (!rope != (rope_dim == 0)) return fail(AGG_E_ARG, "rope and rope_dim go together");
  if (rope_pairs != 0 && rope_pairs != 1) return fail(AGG_E_ARG, "rope_pairs is %d, not 0 or 1", rope_pairs);
  if (tokens > kMostRows || rope_rows > kMostRows) return fail(AGG_E_UNSUPPORTED, "tokens or rope_rows beyond 2^30");
  CHECK(check_table(cache, table, seqs, seq_pages, ld_table));
  if (tokens == 0) return AGG_OK;
  const int64_t d = cache->head_dim;
  CHECK(check_rows(k, ld_k, cache->kv_heads * d, 2, "k"));
  CHECK(check_rows(v, ld_v, cache->kv_heads * d, 2, "v"));
  if (q_heads > 0) {
    CHECK(check_rows(q, ld_q, q_heads * d, 2, "q"));
    CHECK(check_rows(q_out, ld_q_out, q_heads * d, 2, "q_out"));
    if (q == q_out && ld_q != ld_q_out && tokens > 1) return fail(AGG_E_ARG, "q_out is q at another stride");
  }
  if (rope) CHECK(need(rope, "rope"));
  return need(positions, "positions", 4);
}

extern "C" int agg_check_kv_read_args(const agg_kv_cache* cache, int64_t tokens, const int32_t* positions,
                                      const int32_t* table, int64_t seqs, int64_t seq_pages, int64_t ld_table,
                                      int out_dtype, const void* k_out, int64_t ld_k, const void* v_out, int64_t ld_v) {
  clear_error();
  if (tokens < 0) return fail(AGG_E_ARG, "negative size");
  CHECK(check_cache(cache));
  if (out_dtype != AGG_BF16 && out_dtype != AGG_FP32) return fail(AGG_E_ARG, "out has dtype %d, not bf16 or fp32", out_dtype);
  if (tokens > kMostRows) return fail(AGG_E_UNSUPPORTED, "tokens beyond 2^30");
  CHECK(check_table(cache, table, seqs, seq_pages, ld_table));
  if (tokens == 0) return AGG_OK;
  const int64_t cols = int64_t(cache->kv_heads) * cache->head_dim;
  const int eb = out_dtype == AGG_FP32 ? 4 : 2;
  CHECK(check_rows(k_out, ld_k, cols, eb, "k_out"));
  CHECK(check_rows(v_out, ld_v, cols, eb, "v_out"));
  return need(positions, "positions", 4);
}

extern "C" int agg_check_paged_attn_args(const agg_kv_cache* cache, int64_t rows, int q_heads, const void* q,
                                         int64_t ld_q, float scale, const int32_t* lens, const int32_t* table,
                                         int64_t seqs, int64_t seq_pages, int64_t ld_table, int64_t window,
                                         int out_dtype, const void* out, int64_t ld_out) {
  clear_error();
  CHECK(check_attn_sizes(cache, rows, q_heads, seq_pages, window));
  if (!std::isfinite(scale) || !std::isfinite(scale * 1.442695041f)) return fail(AGG_E_ARG, "scale is not finite");
  if (out_dtype != AGG_BF16 && out_dtype != AGG_FP32) return fail(AGG_E_ARG, "out has dtype %d, not bf16 or fp32", out_dtype);
  CHECK(check_table(cache, table, seqs, seq_pages, ld_table));
  if (rows == 0) return AGG_OK;
  const int64_t cols = int64_t(q_heads) * cache->head_dim;
  CHECK(check_rows(q, ld_q, cols, 2, "q"));
  CHECK(check_rows(out, ld_out, cols, out_dtype == AGG_FP32 ? 4 : 2, "out"));
  return need(lens, "lens", 4);
}

extern "C" int agg_paged_attn_workspace(const agg_kv_cache* cache, int64_t rows, int q_heads, int64_t seq_pages,
                                        int64_t window, int64_t* bytes) {
  clear_error();
  if (!bytes) return fail(AGG_E_ARG, "agg_paged_attn_workspace: NULL output");
  CHECK(check_attn_sizes(cache, rows, q_heads, seq_pages, window));
  *bytes = rows == 0 ? 0 : choose_attn_shape(*cache, rows, q_heads, seq_pages, window, 256).ws_bytes;
  return AGG_OK;
}
