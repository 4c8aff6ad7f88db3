// The paged cache's row operators, bound by memory: the rotation of queries and keys with the write of
// keys and values (kv_write), and the rows read back (kv_read).
#include <type_traits>

#include "attn.h"
#include "convert.h"

namespace agg {

namespace {

// The place of a token: its page and the position in it; page -1 if it has none.
struct Place {
  int page, off, position;
};

__device__ inline Place place_of(const PlaceArgs& a, const agg_kv_cache& c, int64_t t) {
  const int p = a.positions[t];
  const int s = a.token_seq ? a.token_seq[t] : (int)(a.first + t);
  Place r{-1, 0, p};
  if (p < 0 || s < 0 || s >= a.seqs) return r;
  const uint32_t n = (uint32_t)p / (uint32_t)c.page_size;
  if (n >= a.seq_pages) return r;
  const int page = a.table[s * a.ld_table + n];
  r.off = p - (int)n * c.page_size;
  if (page >= 0 && page < c.pages) r.page = page;
  return r;
}

// the largest over a group of 2^lanes_log2 lanes (1 to 16 of them)
__device__ inline uint32_t group_max(uint32_t m, int lanes_log2) {
  auto with = [&](auto ctrl) {
    const uint32_t b = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, decltype(ctrl)::value, 0xF, 0xF, true);
    m = b > m ? b : m;
  };
  using std::integral_constant;
  if (lanes_log2 > 0) with(integral_constant<int, 0xB1>{});    // lanes 1 0 3 2 of each four
  if (lanes_log2 > 1) with(integral_constant<int, 0x4E>{});    // lanes 2 3 0 1
  if (lanes_log2 > 2) with(integral_constant<int, 0x141>{});   // eight lanes mirrored
  if (lanes_log2 > 3) with(integral_constant<int, 0x140>{});   // sixteen mirrored
  return m;
}

// element `d` of head `h` at a place
__device__ inline int64_t element(const agg_kv_cache& c, const Place& at, int h, int d) {
  return at.page * c.ld_page + at.off * c.ld_token + h * c.ld_head + d;
}

}  // namespace

// How a workgroup's threads stand: groups of 2^lanes_log2 lanes, 2^heads_log2 groups to a token, and the other
// tokens after it. A group takes heads first, first + 2^heads_log2, ... of its token, kAhead at a time with all their loads
// ahead of the first use.
struct Deal {
  int lanes_log2, heads_log2;
};
constexpr int kAhead = 4;

// A row is one head of one token: a query's, a key's or a value's. A lane of its group takes two chunks of 8 channels,
// those that turn together where they do (channel i and i + rope_dim / 2 in chunks rope_dim / 16 apart), so nothing is
// read twice or passed between lanes, and the angles are read once for all of a token's heads. The
// rotation and the largest element of a row are fp32; each stored value is rounded once.
//
// Bound by memory: 8192 tokens of 64 + 8 + 8 heads of 128 into 8 bits (322 MB) take 60 us, 5.4 TB/s, where a large copy
// reaches 5.1; a lane with one chunk of one head, its partner's read beside it, took 100. 16 such tokens: 3.6 us, a
// launch and three round trips to memory (position, page, row).
template <bool FP8>
__global__ void __launch_bounds__(256) kv_write_kernel(const KvWriteArgs a, const Deal deal) {
  const agg_kv_cache& c = a.cache;
  const int D = c.head_dim, lane = threadIdx.x & ((1 << deal.lanes_log2) - 1), group = threadIdx.x >> deal.lanes_log2;
  const int64_t t = (int64_t)blockIdx.x * (256 >> (deal.lanes_log2 + deal.heads_log2)) + (group >> deal.heads_log2);
  if (t >= a.tokens) return;
  const Place at = place_of(a.at, c, t);
  if (at.page < 0 || (a.rope && at.position >= a.rope_rows)) return;
  // this lane's chunks
  const int turning = a.rope_dim / 16;                     // lanes whose channels turn
  const bool in = lane * 16 < D, halves = lane < turning && !a.pairs;
  const int d0 = halves ? lane * 8 : lane * 16, d1 = halves ? d0 + a.rope_dim / 2 : d0 + 8;
  // their angles: halves: 8 of both chunks; pairs: 4 of each
  float cs[8], sn[8];
  if (lane < turning) {
    const float* const p = a.rope + (int64_t)at.position * a.rope_dim + lane * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4 x = reinterpret_cast<const f32x4*>(p)[i], y = reinterpret_cast<const f32x4*>(p + a.rope_dim / 2)[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        cs[4 * i + e] = x[e];
        sn[4 * i + e] = y[e];
      }
    }
  }
  const int heads = a.q_heads + 2 * c.kv_heads, step = 1 << deal.heads_log2;
  for (int h0 = group & (step - 1); h0 < heads; h0 += kAhead * step) {
    u32x4 w[kAhead][2];
    // (past the last head or channel: nothing is read)
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int head = h0 + u * step;
      const uint16_t* const src = head < a.q_heads              ? a.q + t * a.ld_q + (int64_t)head * D
                                  : head < a.q_heads + c.kv_heads ? a.k + t * a.ld_k + (int64_t)(head - a.q_heads) * D
                                                                : a.v + t * a.ld_v + (int64_t)(head - a.q_heads - c.kv_heads) * D;
      w[u][0] = w[u][1] = u32x4{};
      if (in && head < heads) {
        w[u][0] = *reinterpret_cast<const u32x4*>(src + d0);
        w[u][1] = *reinterpret_cast<const u32x4*>(src + d1);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int head = h0 + u * step;
      if (head >= heads) break;
      float x[2][8];
      widen(w[u][0], x[0]);
      widen(w[u][1], x[1]);
      if (lane < turning && head < a.q_heads + c.kv_heads) {
        if (a.pairs) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float &p = x[i >> 2][2 * (i & 3)], &q = x[i >> 2][2 * (i & 3) + 1];
            const float v = p * cs[i] - q * sn[i];
            q = q * cs[i] + p * sn[i];
            p = v;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float v = x[0][i] * cs[i] - x[1][i] * sn[i];
            x[1][i] = x[1][i] * cs[i] + x[0][i] * sn[i];
            x[0][i] = v;
          }
        }
      }
      if (head < a.q_heads) {
        uint16_t* const to = a.q_out + t * a.ld_q_out + (int64_t)head * D;
        if (in) {
          *reinterpret_cast<u32x4*>(to + d0) = narrow(x[0]);
          *reinterpret_cast<u32x4*>(to + d1) = narrow(x[1]);
        }
        continue;
      }
      const bool key = head < a.q_heads + c.kv_heads;
      const int h = key ? head - a.q_heads : head - a.q_heads - c.kv_heads;
      void* const pool = key ? c.k : c.v;
      const int64_t to = element(c, at, h, 0);
      if constexpr (!FP8) {
        if (in) {
          *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(pool) + to + d0) = narrow(x[0]);
          *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(pool) + to + d1) = narrow(x[1]);
        }
      } else {
        // the largest element by its bit pattern: a NaN is larger than every number and is kept
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t b = __builtin_bit_cast(uint32_t, x[i >> 3][i & 7]) & 0x7FFFFFFFu;
          m = b > m ? b : m;
        }
        m = group_max(m, deal.lanes_log2);
        const float top = __builtin_bit_cast(float, m) / 448.0f;
        const float scale = top > 0.0f ? top : 1.0f;        // a row of zeros, or with a NaN: 1
        // One reciprocal a row, and a step that brings each quotient to what the division gives (a product with the
        // reciprocal alone is a unit off now and then, and puts more elements on the other side of a tie). A
        // subnormal scale can be a third below max|x| / 448, an infinite one has no reciprocal, and the 1 of a row
        // with a NaN has nothing to do with the others: these divide and clamp
        if (top >= kNormal && top < __builtin_inff()) {
          const float by = 1.0f / scale;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float& v = x[i >> 3][i & 7];
            const float q = v * by;
            v = __builtin_fmaf(__builtin_fmaf(-q, scale, v), by, q);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i >> 3][i & 7] = clamp_e4m3(x[i >> 3][i & 7] / scale);
        }
        if (in) {
          *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(pool) + to + d0) = narrow_e4m3(x[0]);
          *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(pool) + to + d1) = narrow_e4m3(x[1]);
        }
        if (lane == 0) (key ? c.k_scale : c.v_scale)[((int64_t)at.page * c.kv_heads + h) * c.page_size + at.off] = scale;
      }
    }
  }
}

// A row is one head of one token, of the keys or of the values; a lane of its group takes two chunks of 8 channels.
// Bound by memory: 65536 tokens of 8 heads of 64 bf16 (269 MB) take 55 us, 4.9 TB/s (one chunk a lane: 60), 4951 of 8
// heads of 128 from 8 bits (31 MB) 8.4.
template <bool FP8, bool OUT32>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvReadArgs a, const Deal deal) {
  const agg_kv_cache& c = a.cache;
  const int D = c.head_dim, lane = threadIdx.x & ((1 << deal.lanes_log2) - 1), group = threadIdx.x >> deal.lanes_log2;
  const int64_t t = (int64_t)blockIdx.x * (256 >> (deal.lanes_log2 + deal.heads_log2)) + (group >> deal.heads_log2);
  const int d = lane * 16;
  if (t >= a.tokens || d >= D) return;
  const Place at = place_of(a.at, c, t);
  const int heads = 2 * c.kv_heads, step = 1 << deal.heads_log2;
  for (int h0 = group & (step - 1); h0 < heads; h0 += kAhead * step) {
    u32x4 w[kAhead][FP8 ? 1 : 2];
    float scale[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int head = h0 + u * step;
      const bool key = head < c.kv_heads;
      const int h = key ? head : head - c.kv_heads;
      scale[u] = 0.0f;
#pragma unroll
      for (int i = 0; i < (FP8 ? 1 : 2); ++i) w[u][i] = u32x4{};
      if (head < heads && at.page >= 0) {
        const int64_t from = element(c, at, h, d);
        const void* const pool = key ? c.k : c.v;
        if constexpr (FP8) {
          w[u][0] = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(pool) + from);
          scale[u] = (key ? c.k_scale : c.v_scale)[((int64_t)at.page * c.kv_heads + h) * c.page_size + at.off];
        } else {
          w[u][0] = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(pool) + from)[0];
          w[u][1] = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(pool) + from)[1];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int head = h0 + u * step;
      if (head >= heads) break;
      const bool key = head < c.kv_heads;
      const int h = key ? head : head - c.kv_heads;
      const int64_t to = t * (key ? a.ld_k : a.ld_v) + (int64_t)h * D + d;
      void* const out = key ? a.k : a.v;
      if constexpr (!FP8 && !OUT32) {
        reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + to)[0] = w[u][0];
        reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + to)[1] = w[u][1];
        continue;
      }
      float x[2][8];
      if constexpr (FP8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[u][0][i], false);
          const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[u][0][i], true);
          float* const p = &x[i >> 1][4 * (i & 1)];
          p[0] = lo[0] * scale[u];
          p[1] = lo[1] * scale[u];
          p[2] = hi[0] * scale[u];
          p[3] = hi[1] * scale[u];
        }
      } else {
        widen(w[u][0], x[0]);
        widen(w[u][FP8 ? 0 : 1], x[1]);
      }
      if constexpr (OUT32) {
        f32x4* const p = reinterpret_cast<f32x4*>(static_cast<float*>(out) + to);
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = f32x4{x[i >> 1][4 * (i & 1)], x[i >> 1][4 * (i & 1) + 1], x[i >> 1][4 * (i & 1) + 2], x[i >> 1][4 * (i & 1) + 3]};
      } else {
        reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + to)[0] = narrow(x[0]);
        reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + to)[1] = narrow(x[1]);
      }
    }
  }
}

namespace {

// The deal of `heads` rows a token of `d` channels: a group takes several heads where tokens enough are left to fill the
// GPU (their places and angles are then read less often).
Deal deal_of(int64_t tokens, int heads, int d, int cus) {
  Deal r{0, 0};
  while ((16 << r.lanes_log2) < d) ++r.lanes_log2;
  const int groups_log2 = 8 - r.lanes_log2;
  while (r.heads_log2 < groups_log2 && (1 << r.heads_log2) < heads &&
         ((kAhead << r.heads_log2) < heads || (tokens << (r.lanes_log2 + r.heads_log2)) < int64_t(cus) * 1024))
    ++r.heads_log2;
  return r;
}

unsigned blocks_of(int64_t tokens, const Deal& d) {
  const int64_t each = 256 >> (d.lanes_log2 + d.heads_log2);
  return (unsigned)((tokens + each - 1) / each);
}

// (a launch holds fewer than 2^32 threads)
constexpr int64_t kMostTokens = int64_t(1) << 23;

PlaceArgs after(const PlaceArgs& a, int64_t t) {
  PlaceArgs r = a;
  r.positions += t;
  if (r.token_seq) r.token_seq += t;
  r.first += t;
  return r;
}

}  // namespace

hipError_t launch_kv_write(const KvWriteArgs& all, int cus, hipStream_t stream) {
  for (int64_t t = 0; t < all.tokens; t += kMostTokens) {
    KvWriteArgs a = all;
    a.tokens = all.tokens - t < kMostTokens ? all.tokens - t : kMostTokens;
    a.at = after(all.at, t);
    a.q += t * a.ld_q;
    a.q_out += t * a.ld_q_out;
    a.k += t * a.ld_k;
    a.v += t * a.ld_v;
    const Deal d = deal_of(a.tokens, a.q_heads + 2 * a.cache.kv_heads, a.cache.head_dim, cus);
    const dim3 grid(blocks_of(a.tokens, d)), block(256);
    if (a.cache.dtype == AGG_FP8_E4M3) hipLaunchKernelGGL(kv_write_kernel<true>, grid, block, 0, stream, a, d);
    else hipLaunchKernelGGL(kv_write_kernel<false>, grid, block, 0, stream, a, d);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

hipError_t launch_kv_read(const KvReadArgs& all, int cus, hipStream_t stream) {
  for (int64_t t = 0; t < all.tokens; t += kMostTokens) {
    KvReadArgs a = all;
    a.tokens = all.tokens - t < kMostTokens ? all.tokens - t : kMostTokens;
    a.at = after(all.at, t);
    a.k = static_cast<char*>(all.k) + t * a.ld_k * (a.out_fp32 ? 4 : 2);
    a.v = static_cast<char*>(all.v) + t * a.ld_v * (a.out_fp32 ? 4 : 2);
    const Deal d = deal_of(a.tokens, 2 * a.cache.kv_heads, a.cache.head_dim, cus);
    const dim3 grid(blocks_of(a.tokens, d)), block(256);
    if (a.cache.dtype == AGG_FP8_E4M3) {
      if (a.out_fp32) hipLaunchKernelGGL((kv_read_kernel<true, true>), grid, block, 0, stream, a, d);
      else hipLaunchKernelGGL((kv_read_kernel<true, false>), grid, block, 0, stream, a, d);
    } else {
      if (a.out_fp32) hipLaunchKernelGGL((kv_read_kernel<false, true>), grid, block, 0, stream, a, d);
      else hipLaunchKernelGGL((kv_read_kernel<false, false>), grid, block, 0, stream, a, d);
    }
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace agg
