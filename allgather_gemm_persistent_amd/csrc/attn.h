// Device-side interface of the attention operators: launch functions (defined in kv.hip and attn.hip)
// and their argument blocks.
#pragma once

#include "kernels.h"

namespace agg {

// Where the tokens of a call lie in a cache.
struct PlaceArgs {
  const int32_t* positions;
  const int32_t* token_seq;   // or null: token t is sequence first + t
  const int32_t* table;       // seqs x seq_pages
  int64_t seqs, seq_pages, ld_table, first;
};

struct KvWriteArgs {
  agg_kv_cache cache;
  PlaceArgs at;
  const uint16_t *q, *k, *v;  // bfloat16 rows
  uint16_t* q_out;
  int64_t ld_q, ld_q_out, ld_k, ld_v;   // elements
  const float* rope;          // rope_rows x rope_dim, cosines then sines; or null
  int64_t tokens, rope_rows;
  int q_heads, rope_dim, pairs;
};
hipError_t launch_kv_write(const KvWriteArgs& a, int cus, hipStream_t stream);

struct KvReadArgs {
  agg_kv_cache cache;
  PlaceArgs at;
  void *k, *v;                // tokens x (kv_heads * head_dim), bfloat16 or float
  int64_t ld_k, ld_v;         // elements
  int64_t tokens;
  int out_fp32;
};
hipError_t launch_kv_read(const KvReadArgs& a, int cus, hipStream_t stream);

struct AttnArgs {
  agg_kv_cache cache;
  const uint16_t* q;          // rows x (q_heads * head_dim) bfloat16
  void* out;                  // rows x (q_heads * head_dim), bfloat16 or float
  float* lse;                 // rows x q_heads, or null
  const int32_t* lens;
  const int32_t* row_seq;     // or null: row r is sequence first_row + r
  const int32_t* table;       // seqs x seq_pages
  int64_t seqs, seq_pages, ld_table;
  int64_t rows, first_row, ld_q, ld_out;
  int64_t window;             // 0: none
  float scale2;               // scale * log2(e)
  int q_heads, group;         // heads of queries, and how many share a head of the cache
  int row_tiles;              // 16-row tiles of a head's queries a workgroup takes at once (1, 2, 4)
  int out_fp32;
  int least;                  // tiles of a unit at least
  float* ws;                  // slots of slot_bytes for the parts of the rows that are split
  int64_t ws_bytes;
  int slot_bytes;
  uint32_t* counts;           // eight for every workgroup and two, zero before and after
  uint32_t page_magic, page_shift;   // x / (page_size / 16) = x * page_magic >> page_shift for x below 2^27
};
// `grid` workgroups divide the work; rows * kv_heads * (tiles of a row) stays below 2^31.
hipError_t launch_attn(const AttnArgs& a, int grid, hipStream_t stream);

}  // namespace agg
