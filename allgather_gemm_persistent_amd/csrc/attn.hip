// Attention of new tokens over a paged cache (paged_attn): out = sum_i softmax(x)_i v_i, x_i = scale q . k_i,
// for every row (a new token) and head of queries.
#include <type_traits>

#include "attn.h"
#include "convert.h"

namespace agg {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kAttnWaves = 4;
constexpr int kTile = 32;                      // tokens a wave takes at once: two runs of 16
constexpr int kBufferFlags = 0x00020000;       // word 3 of a raw buffer resource
constexpr uint32_t kOutOfRange = 0x80000000u;  // an offset past every descriptor
constexpr float kLn2 = 0.693147181f;

__device__ inline f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}

__device__ inline uint32_t pack2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}
__device__ inline float low_half(uint32_t p) { return __builtin_bit_cast(float, p << 16); }
__device__ inline float high_half(uint32_t p) { return __builtin_bit_cast(float, p & 0xFFFF0000u); }

// two e4m3 of a word as two bf16 (exact)
template <bool HIGH>
__device__ inline uint32_t widen8(uint32_t p) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p, 1.0f, HIGH));
}

}  // namespace

// One workgroup per row, head of the cache and 16 * RT of the queries that share it; its four waves take runs
// of the length and join their results.
//
// A wave takes 32 tokens at a time through the matrix units, transposed, so that nothing passes between
// lanes on the way: S^T = K Q^T with the tokens as rows and the (up to 16) queries as columns puts into lane
// l the products of query l % 16 with tokens 4 (l / 16) + i of both runs of 16, which is the order in which the
// second product O^T = V^T P^T wants its weights in that lane if token 4 (l / 16) + i of run u is called
// contraction index 8 (l / 16) + 4 u + i. V is read row by row (a lane holds VE channels of 8 tokens) and turned by
// byte permutes inside the lane: fragment m holds channel m of every lane's chunk.
//
// Softmax in one pass: a lane holds the running maximum and sum (in powers of 2) of its query, over its own
// tokens the sum, over all the maximum. The weights enter the second product as a bf16 and the bf16 of what that
// leaves, so they carry 16 bits; the matrix units are far from busy (32 tokens of 128 channels are 8 KiB of K
// and of V, and 24 matrix instructions).
template <bool FP8, int DP, int RT>
__global__ void __launch_bounds__(kAttnWaves * 64) attn_kernel(const AttnArgs a) {
  constexpr int EL = FP8 ? 1 : 2;
  constexpr int KS = DP / 32;                  // contraction steps of the first product
  constexpr int VE = DP / 16;                  // channels of V a lane holds
  constexpr int KL = DP * EL / 64;             // 16-byte loads of a token's keys by a lane
  constexpr int VW = VE * EL / 4;              // words of a token's values in a lane
  constexpr int PO = DP + 4;                   // padded row of the partial results
  __shared__ __attribute__((aligned(16))) float s_o[kAttnWaves][16][PO];
  __shared__ float s_m[kAttnWaves][16], s_l[kAttnWaves][16];

  const agg_kv_cache& cache = a.cache;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int D = cache.head_dim, pg = cache.page_size;
  // the item
  const int splits = (a.group + 16 * RT - 1) / (16 * RT);
  const int item = blockIdx.x;
  const int part = item % splits, head = item / splits % cache.kv_heads;
  const int64_t row = item / splits / cache.kv_heads;
  const int q0 = part * 16 * RT;               // first query of the head's group
  const int held = a.group - q0 < 16 * RT ? a.group - q0 : 16 * RT;

  // its tokens [lo, hi)
  const int seq = __builtin_amdgcn_readfirstlane(a.row_seq ? a.row_seq[row] : (int)row);
  const int room = (int)(a.seq_pages * pg);
  int hi = __builtin_amdgcn_readfirstlane(a.lens[row]);
  hi = seq < 0 || seq >= a.seqs || hi < 0 ? 0 : hi < room ? hi : room;
  const int lo = a.window > 0 && hi > a.window ? (int)(hi - a.window) : 0;
  const int32_t* const table = a.table + (hi > 0 ? seq * a.ld_table : 0);

  // this wave's runs of 32 tokens
  const int first = lo / kTile, tiles = hi > lo ? (hi + kTile - 1) / kTile - first : 0;
  const int t_lo = first + tiles * wave / kAttnWaves, t_hi = first + tiles * (wave + 1) / kAttnWaves;

  // Q: column c, steps of 32 channels; lane's 8 of step s as K's lane has them
  u32x4 qf[RT][KS];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d = FP8 ? (s >> 1) * 64 + g * 16 + (s & 1) * 8 : s * 32 + g * 8;
      const int j = r * 16 + c;
      qf[r][s] = u32x4{};
      if (j < held && d < D)
        qf[r][s] = *reinterpret_cast<const u32x4*>(a.q + row * a.ld_q + (int64_t)(head * a.group + q0 + j) * D + d);
    }

  f32x4 o[RT][VE];
  float m[RT], l[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.0f;
#pragma unroll
    for (int e = 0; e < VE; ++e) o[r][e] = f32x4{};
  }

  // offsets of this lane in a run of 16 tokens
  const uint32_t token_bytes = (uint32_t)(cache.ld_token * EL);
  uint32_t koff[KL];
#pragma unroll
  for (int i = 0; i < KL; ++i) {
    const int d = FP8 ? i * 64 + g * 16 : i * 32 + g * 8;
    koff[i] = d < D ? (uint32_t)c * token_bytes + (uint32_t)(d * EL) : kOutOfRange;
  }
  // (256 channels of bf16: two loads of 16 bytes, 128 channels apart)
  constexpr int VL = VW > 4 ? VW / 4 : 1, VC = VE / VL;
  uint32_t voff[VL];
#pragma unroll
  for (int i = 0; i < VL; ++i) {
    const int d = i * 16 * VC + c * VC;
    voff[i] = d < D ? (uint32_t)(d * EL) : kOutOfRange;
  }

  // the page of each run of 16 tokens, and the place in it: 64 runs in the lanes at a time
  int pages = -1, inside = 0, block = -1;
  auto look_up = [&](int run) {
    if (run >> 6 == block) return;
    block = run >> 6;
    const uint32_t token = ((uint32_t)block * 64 + (uint32_t)lane) * 16;
    const uint32_t n = token / (uint32_t)pg;
    pages = -1;
    if ((int)token < hi) {
      const int p = table[n];
      if (p >= 0 && p < cache.pages) pages = p;
    }
    inside = (int)(token - n * (uint32_t)pg);
  };
  struct Run {
    int page, inside;
    int held;                                  // of its 16 tokens, from the first
  };
  auto run_of = [&](int run) {
    look_up(run);
    Run r{__builtin_amdgcn_readlane(pages, run & 63), __builtin_amdgcn_readlane(inside, run & 63), hi - run * 16};
    r.held = r.page < 0 || r.held < 0 ? 0 : r.held < 16 ? r.held : 16;
    return r;
  };
  auto descriptor = [&](const void* pool, const Run& r) {
    const int64_t at = r.held ? (int64_t)r.page * cache.ld_page + (int64_t)r.inside * cache.ld_token +
                                    (int64_t)head * cache.ld_head : 0;
    return __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(static_cast<const uint8_t*>(pool)) + at * EL, 0,
        r.held ? (int)((uint32_t)(r.held - 1) * token_bytes + (uint32_t)(D * EL)) : 0, kBufferFlags);
  };

  struct Keys {
    u32x4 k[2][KL];
    f32x4 scale[2];
    int held[2];
  };
  struct Values {
    uint32_t v[2][4][VW];
    f32x4 scale[2];
  };
  auto load_keys = [&](Keys& x, int tile) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const Run r = run_of(2 * tile + u);
      x.held[u] = r.held;
      const __amdgpu_buffer_rsrc_t d = descriptor(cache.k, r);
#pragma unroll
      for (int i = 0; i < KL; ++i)
        x.k[u][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(d, (int)koff[i], 0, 0));
      if constexpr (FP8) {
        x.scale[u] = f32x4{};
        if (r.held)
          x.scale[u] = *reinterpret_cast<const f32x4*>(
              cache.k_scale + ((int64_t)r.page * cache.kv_heads + head) * pg + r.inside + 4 * g);
      }
    }
  };
  auto load_values = [&](Values& x, int tile) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const Run r = run_of(2 * tile + u);
      const __amdgpu_buffer_rsrc_t d = descriptor(cache.v, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // (a value before the window may be anything, and zero times it a NaN: it is not read)
        const int token = tile * kTile + u * 16 + 4 * g + i;
        const uint32_t skip = token < lo ? kOutOfRange : 0u;
        const uint32_t base = (uint32_t)(4 * g + i) * token_bytes;
#pragma unroll
        for (int p = 0; p < VL; ++p) {
          const int off = (int)((voff[p] + base) | skip | (voff[p] & kOutOfRange));
          if constexpr (VW >= 4) {
            const u32x4 w = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(d, off, 0, 0));
#pragma unroll
            for (int e = 0; e < 4; ++e) x.v[u][i][4 * p + e] = w[e];
          } else if constexpr (VW == 2) {
            const u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(d, off, 0, 0));
            x.v[u][i][0] = w[0];
            x.v[u][i][1] = w[1];
          } else {
            x.v[u][i][0] = __builtin_amdgcn_raw_buffer_load_b32(d, off, 0, 0);
          }
        }
      }
      if constexpr (FP8) {
        x.scale[u] = f32x4{};
        if (r.held)
          x.scale[u] = *reinterpret_cast<const f32x4*>(
              cache.v_scale + ((int64_t)r.page * cache.kv_heads + head) * pg + r.inside + 4 * g);
      }
    }
  };

  Keys kx;
  Values vx;
  if (t_lo < t_hi) {
    load_keys(kx, t_lo);
    load_values(vx, t_lo);
  }
  for (int tile = t_lo; tile < t_hi; ++tile) {
    // ---- S^T, times the scale and in powers of 2
    f32x4 s[RT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        s[r][u] = f32x4{};
#pragma unroll
        for (int st = 0; st < KS; ++st) {
          u32x4 f;
          if constexpr (FP8) {
            const u32x4 w = kx.k[u][st >> 1];
            const uint32_t x = w[(st & 1) * 2], y = w[(st & 1) * 2 + 1];
            f = u32x4{widen8<false>(x), widen8<true>(x), widen8<false>(y), widen8<true>(y)};
          } else {
            f = kx.k[u][st];
          }
          s[r][u] = mfma16(f, qf[r][st], s[r][u]);
        }
      }
    bool in[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        in[u][i] = 4 * g + i < kx.held[u] && tile * kTile + u * 16 + 4 * g + i >= lo;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float top = -INFINITY;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = s[r][u][i] * a.scale2;
          if constexpr (FP8) x *= kx.scale[u][i];
          s[r][u][i] = in[u][i] ? x : -INFINITY;
          top = fmaxf(top, s[r][u][i]);
        }
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float now = fmaxf(m[r], top);
      const float base = now == -INFINITY ? 0.0f : now;   // (nothing so far)
      const float shrink = __builtin_amdgcn_exp2f(m[r] - base);
      m[r] = now;
      l[r] *= shrink;
#pragma unroll
      for (int e = 0; e < VE; ++e) o[r][e] *= shrink;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[r][u][i] = __builtin_amdgcn_exp2f(s[r][u][i] - base);
          l[r] += s[r][u][i];
          if constexpr (FP8) s[r][u][i] = in[u][i] ? s[r][u][i] * vx.scale[u][i] : 0.0f;
        }
    }
    if (tile + 1 < t_hi) load_keys(kx, tile + 1);
    // ---- O^T
    u32x4 hi2[RT], lo2[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float x = s[r][p >> 1][2 * (p & 1)], y = s[r][p >> 1][2 * (p & 1) + 1];
        hi2[r][p] = pack2(x, y);
        lo2[r][p] = pack2(x - low_half(hi2[r][p]), y - high_half(hi2[r][p]));
      }
    // fragments of two channels at a time
    auto turn = [&](const uint32_t (&w)[8], int e) {
      u32x4 f0, f1;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        f0[p] = __builtin_amdgcn_perm(w[2 * p + 1], w[2 * p], 0x05040100u);
        f1[p] = __builtin_amdgcn_perm(w[2 * p + 1], w[2 * p], 0x07060302u);
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        o[r][e] = mfma16(f0, hi2[r], o[r][e]);
        o[r][e] = mfma16(f0, lo2[r], o[r][e]);
        o[r][e + 1] = mfma16(f1, hi2[r], o[r][e + 1]);
        o[r][e + 1] = mfma16(f1, lo2[r], o[r][e + 1]);
      }
    };
#pragma unroll
    for (int e = 0; e < VE; e += 2) {
      uint32_t w[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        if constexpr (FP8) {
          const uint32_t x = vx.v[t >> 2][t & 3][e / 4];
          w[t] = e & 2 ? widen8<true>(x) : widen8<false>(x);
        } else {
          w[t] = vx.v[t >> 2][t & 3][e / 2];
        }
      }
      turn(w, e);
    }
    if (tile + 1 < t_hi) load_values(vx, tile + 1);
  }

  // ---- the waves' results, 16 queries at a time
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    if (r * 16 >= held) break;
    float sum = l[r];
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    __syncthreads();
    if (g == 0) {
      s_m[wave][c] = m[r];
      s_l[wave][c] = sum;
    }
    // row 4 g + i of fragment e is channel e of chunk 4 g + i
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e)
        s_o[wave][c][e / VC * 16 * VC + (4 * g + i) * VC + e % VC] = o[r][e][i];
    __syncthreads();
    for (int x = tid; x < 16 * (DP / 8); x += kAttnWaves * 64) {
      const int j = x / (DP / 8), d = x % (DP / 8) * 8;
      if (r * 16 + j >= held || d >= D) continue;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kAttnWaves; ++w) top = fmaxf(top, s_m[w][j]);
      const float base = top == -INFINITY ? 0.0f : top;
      float total = 0.0f, y[8] = {};
#pragma unroll
      for (int w = 0; w < kAttnWaves; ++w) {
        const float by = __builtin_amdgcn_exp2f(s_m[w][j] - base);
        total += by * s_l[w][j];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] += by * s_o[w][j][d + e];
      }
      const float inv = total > 0.0f ? 1.0f / total : total;   // (a NaN stays one)
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= inv;
      const int qh = head * a.group + q0 + r * 16 + j;
      const int64_t to = row * a.ld_out + (int64_t)qh * D + d;
      if (a.out_fp32) {
        f32x4* const p = reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + to);
        p[0] = f32x4{y[0], y[1], y[2], y[3]};
        p[1] = f32x4{y[4], y[5], y[6], y[7]};
      } else {
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + to) = narrow(y);
      }
      if (a.lse && d == 0) a.lse[row * a.q_heads + qh] = top == -INFINITY ? top : top * kLn2 + logf(total);
    }
  }
}

template <bool FP8, int DP>
static hipError_t launch_attn_dp(const AttnArgs& a, hipStream_t stream) {
  const int splits = (a.group + 16 * a.row_tiles - 1) / (16 * a.row_tiles);
  const dim3 grid((unsigned)(a.rows * a.cache.kv_heads * splits)), block(kAttnWaves * 64);
  if (a.row_tiles == 1) hipLaunchKernelGGL((attn_kernel<FP8, DP, 1>), grid, block, 0, stream, a);
  else if (a.row_tiles == 2) hipLaunchKernelGGL((attn_kernel<FP8, DP, 2>), grid, block, 0, stream, a);
  else if constexpr (DP < 256) hipLaunchKernelGGL((attn_kernel<FP8, DP, 4>), grid, block, 0, stream, a);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

template <bool FP8>
static hipError_t launch_attn_type(const AttnArgs& a, hipStream_t stream) {
  if (a.cache.head_dim <= 64) return launch_attn_dp<FP8, 64>(a, stream);
  if (a.cache.head_dim <= 128) return launch_attn_dp<FP8, 128>(a, stream);
  return launch_attn_dp<FP8, 256>(a, stream);
}

hipError_t launch_attn(const AttnArgs& a, hipStream_t stream) {
  return a.cache.dtype == AGG_FP8_E4M3 ? launch_attn_type<true>(a, stream) : launch_attn_type<false>(a, stream);
}

}  // namespace agg
