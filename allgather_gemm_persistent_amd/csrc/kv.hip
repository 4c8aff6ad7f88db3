// The paged cache's row operators, bound by memory: the rotation of queries and keys with the write of
// keys and values (kv_write), and the rows read back (kv_read).
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
  const int s = a.token_seq ? a.token_seq[t] : (int)t;
  Place r{-1, 0, p};
  if (p < 0 || s < 0 || s >= a.seqs) return r;
  const uint32_t n = (uint32_t)p / (uint32_t)c.page_size;
  if (n >= a.seq_pages) return r;
  const int page = a.table[s * a.ld_table + n];
  r.off = p - (int)n * c.page_size;
  if (page >= 0 && page < c.pages) r.page = page;
  return r;
}

// element `d` of head `h` at a place
__device__ inline int64_t element(const agg_kv_cache& c, const Place& at, int h, int d) {
  return at.page * c.ld_page + at.off * c.ld_token + h * c.ld_head + d;
}

}  // namespace

// A row is one head of one token: a query's, a key's or a value's. It is taken by a group of 2^group_log2
// lanes of a wave, a chunk of 8 channels each. A channel that turns has its partner in the same
// chunk (pairs) or in the chunk rope_dim / 16 further (halves), which the lane reads as well: from
// the cache that its neighbour's read fills. Sums of the rotation and the largest element of a row are fp32;
// each stored value is rounded once.
template <bool FP8>
__global__ void __launch_bounds__(256) kv_write_kernel(const KvWriteArgs a, int64_t first, uint32_t rows,
                                                       int group_log2) {
  const int lane = threadIdx.x & ((1 << group_log2) - 1);
  const uint32_t per_block = 256u >> group_log2;
  const agg_kv_cache& c = a.cache;
  const uint32_t heads = (uint32_t)(a.q_heads + 2 * c.kv_heads);
  const int d = lane * 8;
  const bool in = d < c.head_dim;
  for (uint32_t r = blockIdx.x * per_block + (threadIdx.x >> group_log2); r < rows; r += gridDim.x * per_block) {
    const int64_t t = first + r / heads;
    const int head = (int)(r % heads);
    const Place at = place_of(a.at, c, t);
    if (at.page < 0 || (a.rope && at.position >= a.rope_rows)) continue;
    // 0: a query, 1: a key, 2: a value
    const int kind = head < a.q_heads ? 0 : head < a.q_heads + c.kv_heads ? 1 : 2;
    const int h = kind == 0 ? head : kind == 1 ? head - a.q_heads : head - a.q_heads - c.kv_heads;
    const uint16_t* const src = (kind == 0 ? a.q + t * a.ld_q : kind == 1 ? a.k + t * a.ld_k : a.v + t * a.ld_v) +
                                (int64_t)h * c.head_dim;
    float x[8] = {};
    if (in) widen(*reinterpret_cast<const u32x4*>(src + d), x);
    if (kind < 2 && d < a.rope_dim) {
      const float* const cosines = a.rope + (int64_t)at.position * a.rope_dim;
      const float* const sines = cosines + a.rope_dim / 2;
      if (a.pairs) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float cs = cosines[d / 2 + i], sn = sines[d / 2 + i], u = x[2 * i], w = x[2 * i + 1];
          x[2 * i] = u * cs - w * sn;
          x[2 * i + 1] = w * cs + u * sn;
        }
      } else {
        const int half = a.rope_dim / 2;
        const bool low = d < half;
        const int angle = low ? d : d - half;
        float other[8];
        widen(*reinterpret_cast<const u32x4*>(src + (low ? d + half : d - half)), other);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float cs = cosines[angle + i], sn = sines[angle + i];
          x[i] = low ? x[i] * cs - other[i] * sn : x[i] * cs + other[i] * sn;
        }
      }
    }
    if (kind == 0) {
      if (in) *reinterpret_cast<u32x4*>(a.q_out + t * a.ld_q_out + (int64_t)h * c.head_dim + d) = narrow(x);
      continue;
    }
    void* const pool = kind == 1 ? c.k : c.v;
    const int64_t to = element(c, at, h, d);
    if constexpr (!FP8) {
      if (in) *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(pool) + to) = narrow(x);
    } else {
      // the largest element by its bit pattern: a NaN is larger than every number and is kept
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t b = __builtin_bit_cast(uint32_t, x[i]) & 0x7FFFFFFFu;
        m = b > m ? b : m;
      }
      for (int s = 1 << group_log2 >> 1; s > 0; s >>= 1) {
        const uint32_t b = (uint32_t)__shfl_xor((int)m, s);
        m = b > m ? b : m;
      }
      const float top = __builtin_bit_cast(float, m) / 448.0f;
      const float scale = top > 0.0f ? top : 1.0f;          // a row of zeros, or with a NaN: 1
      // (one reciprocal a row: it and the division differ by a unit of fp32 at most, far below e4m3's. A
      // scale so small that the reciprocal overflows divides; a subnormal one can be a third below
      // max|x| / 448, and the 1 of a row with a NaN has nothing to do with the others: these clamp)
      const bool small = !(scale >= kNormal);
      const float by = 1.0f / scale;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = small ? x[i] / scale : x[i] * by;
        if (!(top >= kNormal)) x[i] = clamp_e4m3(x[i]);
      }
      if (in) *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(pool) + to) = narrow_e4m3(x);
      if (lane == 0)
        (kind == 1 ? c.k_scale : c.v_scale)[((int64_t)at.page * c.kv_heads + h) * c.page_size + at.off] = scale;
    }
  }
}

// A row is one head of one token, of the keys or of the values; a lane takes a chunk of 8 channels.
template <bool FP8, bool OUT32>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvReadArgs a, int64_t first, uint32_t rows,
                                                      int group_log2) {
  const int lane = threadIdx.x & ((1 << group_log2) - 1);
  const uint32_t per_block = 256u >> group_log2;
  const agg_kv_cache& c = a.cache;
  const uint32_t heads = (uint32_t)(2 * c.kv_heads);
  const int d = lane * 8;
  if (d >= c.head_dim) return;
  for (uint32_t r = blockIdx.x * per_block + (threadIdx.x >> group_log2); r < rows; r += gridDim.x * per_block) {
    const int64_t t = first + r / heads;
    const int head = (int)(r % heads);
    const bool key = head < c.kv_heads;
    const int h = key ? head : head - c.kv_heads;
    const Place at = place_of(a.at, c, t);
    float x[8] = {};
    if (at.page >= 0) {
      const void* const pool = key ? c.k : c.v;
      const int64_t from = element(c, at, h, d);
      if constexpr (FP8) {
        const u32x2 p = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(pool) + from);
        const float scale = (key ? c.k_scale : c.v_scale)[((int64_t)at.page * c.kv_heads + h) * c.page_size + at.off];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)p[i], false);
          const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)p[i], true);
          x[4 * i] = lo[0] * scale;
          x[4 * i + 1] = lo[1] * scale;
          x[4 * i + 2] = hi[0] * scale;
          x[4 * i + 3] = hi[1] * scale;
        }
      } else {
        widen(*reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(pool) + from), x);
      }
    }
    const int64_t to = t * (key ? a.ld_k : a.ld_v) + (int64_t)h * c.head_dim + d;
    void* const out = key ? a.k : a.v;
    if constexpr (OUT32) {
      f32x4* const p = reinterpret_cast<f32x4*>(static_cast<float*>(out) + to);
      p[0] = f32x4{x[0], x[1], x[2], x[3]};
      p[1] = f32x4{x[4], x[5], x[6], x[7]};
    } else {
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + to) = narrow(x);
    }
  }
}

namespace {

// lanes of a row of `d` channels, as a power of two
int group_of(int d) {
  int g = 1;
  while ((8 << g) < d) ++g;
  return g;
}

// `go(first token, rows, blocks)` for every launch: a launch counts its rows in 32 bits
template <typename F>
hipError_t in_launches(int64_t tokens, int64_t heads, int group_log2, int cus, F go) {
  const int64_t most = (int64_t(1) << 30) / heads;
  for (int64_t t = 0; t < tokens; t += most) {
    const int64_t rows = (tokens - t < most ? tokens - t : most) * heads;
    const int64_t per_block = 256 >> group_log2, blocks = (rows + per_block - 1) / per_block;
    const int64_t grid = blocks < int64_t(cus) * 64 ? blocks : int64_t(cus) * 64;
    go(t, (uint32_t)rows, (unsigned)grid);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_kv_write(const KvWriteArgs& a, int cus, hipStream_t stream) {
  const int g = group_of(a.cache.head_dim);
  return in_launches(a.tokens, a.q_heads + 2 * a.cache.kv_heads, g, cus, [&](int64_t t, uint32_t rows, unsigned grid) {
    if (a.cache.dtype == AGG_FP8_E4M3) hipLaunchKernelGGL(kv_write_kernel<true>, dim3(grid), dim3(256), 0, stream, a, t, rows, g);
    else hipLaunchKernelGGL(kv_write_kernel<false>, dim3(grid), dim3(256), 0, stream, a, t, rows, g);
  });
}

hipError_t launch_kv_read(const KvReadArgs& a, int cus, hipStream_t stream) {
  const int g = group_of(a.cache.head_dim);
  return in_launches(a.tokens, 2 * a.cache.kv_heads, g, cus, [&](int64_t t, uint32_t rows, unsigned grid) {
    const dim3 gr(grid), bl(256);
    if (a.cache.dtype == AGG_FP8_E4M3) {
      if (a.out_fp32) hipLaunchKernelGGL((kv_read_kernel<true, true>), gr, bl, 0, stream, a, t, rows, g);
      else hipLaunchKernelGGL((kv_read_kernel<true, false>), gr, bl, 0, stream, a, t, rows, g);
    } else {
      if (a.out_fp32) hipLaunchKernelGGL((kv_read_kernel<false, true>), gr, bl, 0, stream, a, t, rows, g);
      else hipLaunchKernelGGL((kv_read_kernel<false, false>), gr, bl, 0, stream, a, t, rows, g);
    }
  });
}

}  // namespace agg
