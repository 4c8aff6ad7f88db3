// The C entry points of the attention operators: checks, then one launch on the caller's stream.
#include "attn.h"
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

// an array of words that may be missing
int check_words(const void* p, const char* what) {
  return reinterpret_cast<uintptr_t>(p) & 3 ? fail(AGG_E_ARG, "%s is not 4-byte aligned", what) : AGG_OK;
}

constexpr int kAttnLeast = 4;   // 32-token tiles: one for each wave
constexpr int64_t kAttnRows = 2048;   // of a launch

// (a dimension of one element may come with any stride: none is taken)
agg_kv_cache without_idle_strides(const agg_kv_cache& c) {
  agg_kv_cache r = c;
  if (r.pages == 1) r.ld_page = 0;
  if (r.kv_heads == 1) r.ld_head = 0;
  return r;
}

}  // namespace

extern "C" int kv_write(agg_ctx* ctx, const agg_kv_cache* cache, int64_t tokens, int q_heads, const void* q, int64_t ld_q,
                        void* q_out, int64_t ld_q_out, const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                        const float* rope, int64_t rope_rows, int rope_dim, int rope_pairs, const int32_t* positions,
                        const int32_t* token_seq, const int32_t* table, int64_t seqs, int64_t seq_pages,
                        int64_t ld_table, agg_stream stream) {
  if (int rc = agg_check_kv_write_args(cache, tokens, q_heads, q, ld_q, q_out, ld_q_out, k, ld_k, v, ld_v, rope, rope_rows,
                                       rope_dim, rope_pairs, positions, table, seqs, seq_pages, ld_table))
    return rc;
  if (int rc = tokens > 0 ? check_words(token_seq, "token_seq") : AGG_OK) return rc;
  if (int rc = enter(ctx)) return rc;
  // (no sequence, page or table: no token has a place)
  if (tokens == 0 || seqs == 0 || seq_pages == 0 || cache->pages == 0) return AGG_OK;
  const KvWriteArgs a{without_idle_strides(*cache), {positions, token_seq, table, seqs, seq_pages, ld_table, 0},
                      static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
                      static_cast<uint16_t*>(q_out), ld_q, ld_q_out, ld_k, ld_v, rope, tokens, rope_rows, q_heads,
                      rope_dim, rope_pairs};
  HIP_TRY(launch_kv_write(a, ctx_units(ctx), S(stream)));
  return AGG_OK;
}

extern "C" int kv_read(agg_ctx* ctx, const agg_kv_cache* cache, int64_t tokens, const int32_t* positions,
                       const int32_t* token_seq, const int32_t* table, int64_t seqs, int64_t seq_pages, int64_t ld_table,
                       int out_dtype, void* k_out, int64_t ld_k, void* v_out, int64_t ld_v, agg_stream stream) {
  if (int rc = agg_check_kv_read_args(cache, tokens, positions, table, seqs, seq_pages, ld_table, out_dtype, k_out, ld_k,
                                      v_out, ld_v))
    return rc;
  if (int rc = tokens > 0 ? check_words(token_seq, "token_seq") : AGG_OK) return rc;
  if (int rc = enter(ctx)) return rc;
  if (tokens == 0) return AGG_OK;
  const KvReadArgs a{without_idle_strides(*cache), {positions, token_seq, table, seqs, seq_pages, ld_table, 0}, k_out, v_out,
                     ld_k, ld_v, tokens, out_dtype == AGG_FP32};
  HIP_TRY(launch_kv_read(a, ctx_units(ctx), S(stream)));
  return AGG_OK;
}

extern "C" int paged_attn(agg_ctx* ctx, const agg_kv_cache* cache, int64_t rows, int q_heads, const void* q, int64_t ld_q,
                          float scale, const int32_t* lens, const int32_t* row_seq, const int32_t* table, int64_t seqs,
                          int64_t seq_pages, int64_t ld_table, int64_t window, int out_dtype, void* out, int64_t ld_out,
                          float* lse, agg_stream stream) {
  if (int rc = agg_check_paged_attn_args(cache, rows, q_heads, q, ld_q, scale, lens, table, seqs, seq_pages, ld_table,
                                         window, out_dtype, out, ld_out))
    return rc;
  if (rows > 0) {
    if (int rc = check_words(row_seq, "row_seq")) return rc;
    if (int rc = check_words(lse, "lse")) return rc;
  }
  if (int rc = enter(ctx)) return rc;
  if (rows == 0) return AGG_OK;
  const AttnShape shape = choose_attn_shape(*cache, rows, q_heads, seq_pages, window, ctx_units(ctx));
  AttnArgs a{without_idle_strides(*cache), static_cast<const uint16_t*>(q), out, lse, lens, row_seq, table, seqs,
             seq_pages, ld_table, rows, 0, ld_q, ld_out, window, scale * 1.442695041f, q_heads, q_heads / cache->kv_heads,
             shape.row_tiles, out_dtype == AGG_FP32, kAttnLeast, nullptr, shape.ws_bytes, shape.slot_bytes, nullptr, 0, 0};
  // runs of 16 tokens to pages: with 2^s <= d < 2^(s+1) and magic = ceil(2^(31+s) / d), magic * d is less than d above
  // 2^(31+s), so x * magic >> (31+s) is x / d while x * 2^(s+1) stays below 2^(31+s)
  const uint32_t d = uint32_t(cache->page_size) / 16;
  int s = 0;
  while (d >> (s + 1)) ++s;
  a.page_magic = uint32_t(((uint64_t(1) << (31 + s)) + d - 1) / d);
  a.page_shift = uint32_t(31 + s);
  if (int rc = ctx_moe_workspace(ctx, stream, size_t(a.ws_bytes), &a.ws, &a.counts)) return rc;
  // (a launch counts its tiles in 31 bits; and a workgroup finds a unit's row by walking up to a 256th of the launch's rows, so
  // that time would grow with the square of them: 64 heads on 8, rows of 16 tokens, in one launch 241 us for 2048, 1668 for 8192,
  // 17245 for 32768; in launches of 2048 982 and 3914)
  const int64_t most = ((int64_t(1) << 31) - 1) / shape.row_most, at_once = most < kAttnRows ? most : kAttnRows;
  for (int64_t r = 0; r < rows; r += at_once) {
    AttnArgs p = a;
    p.rows = rows - r < at_once ? rows - r : at_once;
    p.first_row = r;
    p.q += r * ld_q;
    p.out = static_cast<char*>(out) + r * ld_out * (a.out_fp32 ? 4 : 2);
    if (lse) p.lse += r * q_heads;
    p.lens += r;
    if (row_seq) p.row_seq += r;
    HIP_TRY(launch_attn(p, shape.grid, S(stream)));
  }
  return AGG_OK;
}
