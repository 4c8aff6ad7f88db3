// Operators on whole rows, bound by memory: the residual's addition with the RMS norm and its
// 8-bit output (rms_norm, quant_rows), and the experts' weighted sum (moe_combine).
#include "convert.h"
#include "moe.h"

namespace agg {

namespace {

template <int T, typename F>
__device__ inline uint32_t block_reduce(uint32_t v, F op, uint32_t* lds) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = op(v, (uint32_t)__shfl_xor((int)v, d));
  if constexpr (T > 64) {
    constexpr int W = T / 64;
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v = op(v, lds[w]);
  }
  return v;
}

}  // namespace

// One workgroup a row: s = x + residual, y = s * rsqrt(mean(s^2) + eps) * weight (without a weight:
// y = s). A thread holds V chunks of 8 consecutive columns in registers, so every input is read
// once and the two reductions (the sum of squares; for 8 bits with a scale per row the largest
// |y|) cost no second pass. Sums are 32-bit; s is rounded only where residual_out stores it, so y
// does not carry that rounding.
//
// Bound by memory: 4096 x 8192 bf16 with a residual (268 MB) takes 47 us, 5.7 TB/s, and 4951 x 7168 bf16
// to 8 bits (106 MB) 21 us, 5.0 TB/s, where a large copy reaches 5.1. 16 rows of 8192 fp32: 4.1 us, a
// launch and one round trip to memory; there a row goes over 1024 threads.
template <int T, int V, bool XF32, bool OUT8>
__global__ void __launch_bounds__(T) norm_kernel(const NormArgs a) {
  __shared__ uint32_t lds[2][16];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, chunks = (int)(a.cols / 8);
  float s[V][8];
  u32x4 r[V], xb[V], w[V];
  f32x4 xf[V][2];
  // every load of the row goes out before the first use
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = tid + i * T;
    r[i] = w[i] = xb[i] = u32x4{};
    xf[i][0] = xf[i][1] = f32x4{};
    if (c < chunks) {
      if constexpr (XF32) {
        const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(a.x) + row * a.ld_x + c * 8);
        xf[i][0] = p[0];
        xf[i][1] = p[1];
      } else {
        xb[i] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.x) + row * a.ld_x + c * 8);
      }
      if (a.residual) r[i] = *reinterpret_cast<const u32x4*>(a.residual + row * a.ld_r + c * 8);
      if (a.weight) w[i] = *reinterpret_cast<const u32x4*>(a.weight + c * 8);
    }
  }
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = tid + i * T;
    if constexpr (XF32) {
#pragma unroll
      for (int e = 0; e < 8; ++e) s[i][e] = xf[i][e >> 2][e & 3];
    } else {
      widen(xb[i], s[i]);
    }
    if (a.residual) {
      float add[8];
      widen(r[i], add);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[i][e] += add[e];
      if (a.residual_out && c < chunks)
        *reinterpret_cast<u32x4*>(a.residual_out + row * a.ld_ro + c * 8) = narrow(s[i]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sq += s[i][e] * s[i][e];
  }
  if (a.weight) {
    sq = __builtin_bit_cast(float, block_reduce<T>(__builtin_bit_cast(uint32_t, sq), [](uint32_t x, uint32_t y) {
      return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y));
    }, lds[0]));
    const float inv = rsqrtf(sq / (float)a.cols + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float wv[8];
      widen(w[i], wv);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[i][e] = s[i][e] * inv * wv[e];
    }
  }
  if constexpr (OUT8) {
    float scale = a.scale;
    bool clamp = true;
    if (a.scales) {
      // the largest |y| by its bit pattern: a NaN is larger than every number and is kept
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t b = __builtin_bit_cast(uint32_t, s[i][e]) & 0x7FFFFFFFu;
          m = b > m ? b : m;
        }
      m = block_reduce<T>(m, [](uint32_t x, uint32_t y) { return x > y ? x : y; }, lds[1]);
      const float top = __builtin_bit_cast(float, m) / 448.0f;
      scale = top > 0.0f ? top : 1.0f;      // a row of zeros, or with a NaN: 1
      clamp = !(top >= kNormal);
      if (tid == 0) a.scales[row] = scale;
    }
    // one reciprocal a row instead of a division an element (27 -> 21 us at 4951 x 7168, where the
    // divisions cost more than the memory): y * (1 / scale) and y / scale differ by a unit of fp32 at
    // most, far below e4m3's. Scales so small that the reciprocal overflows divide. With a scale of the
    // row's own, |y| / scale is at most 448 but for a few units, which the conversion rounds away (up to
    // 464); but a subnormal one, a multiple of 2^-149, can be a third below max|y| / 448, and the 1 of a
    // row with a NaN has nothing to do with the other elements: these, and a given scale, need the clamp
    const bool small = !(scale >= kNormal);
    const float by = 1.0f / scale;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * T;
      if (c >= chunks) continue;
      float q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = s[i][e] * by;
      if (small) {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = s[i][e] / scale;
      }
      if (clamp) {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = clamp_e4m3(q[e]);
      }
      *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.out) + row * a.ld_out + c * 8) = narrow_e4m3(q);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * T;
      if (c < chunks)
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + row * a.ld_out + c * 8) = narrow(s[i]);
    }
  }
}

template <int T, int V>
static hipError_t launch_norm_tv(const NormArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)a.rows), block(T);
  if (a.x_fp32) {
    if (a.out_fp8) hipLaunchKernelGGL((norm_kernel<T, V, true, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((norm_kernel<T, V, true, false>), grid, block, 0, stream, a);
  } else {
    if (a.out_fp8) hipLaunchKernelGGL((norm_kernel<T, V, false, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((norm_kernel<T, V, false, false>), grid, block, 0, stream, a);
  }
  return hipGetLastError();
}

hipError_t launch_norm(const NormArgs& all, int cus, hipStream_t stream) {
  NormArgs a = all;
  // (a launch holds fewer than 2^32 threads: more rows go in further ones)
  constexpr int64_t kMost = 1 << 21;
  for (; a.rows > kMost; a.rows -= kMost) {
    NormArgs p = a;
    p.rows = kMost;
    if (hipError_t e = launch_norm(p, cus, stream)) return e;
    a.x = static_cast<const char*>(a.x) + kMost * a.ld_x * (a.x_fp32 ? 4 : 2);
    if (a.residual) a.residual += kMost * a.ld_r;
    if (a.residual_out) a.residual_out += kMost * a.ld_ro;
    a.out = static_cast<char*>(a.out) + kMost * a.ld_out * (a.out_fp8 ? 1 : 2);
    if (a.scales) a.scales += kMost;
  }
  const int64_t chunks = a.cols / 8;
  if (chunks <= 64) return launch_norm_tv<64, 1>(a, stream);
  if (chunks <= 128) return launch_norm_tv<64, 2>(a, stream);
  if (chunks <= 256) return launch_norm_tv<256, 1>(a, stream);
  if (chunks <= 512) return launch_norm_tv<256, 2>(a, stream);
  // a row over 1024 threads for fewer rows than compute units: 3.1 us and 3.2 at 16 x 8192 bf16 with a
  // residual, but 20.9 and 20.2 at 2048 rows. (Short rows the other way: 2048 x 512 takes 3.2 us with 64
  // threads a row, 3.7 with 256)
  if (chunks <= 1024) return a.rows <= cus ? launch_norm_tv<1024, 1>(a, stream) : launch_norm_tv<256, 4>(a, stream);
  if (chunks <= 2048) return launch_norm_tv<1024, 2>(a, stream);
  if (chunks <= 4096) return launch_norm_tv<1024, 4>(a, stream);
  return hipErrorInvalidValue;
}

// out[t] = sum_j weights[t, j] * y[token_slot[t, j]], j ascending, in 32 bits; a pair without a slot
// adds nothing. A thread takes 8 columns of a token; its rows of y are loaded four at a time, so a
// token's whole top 4 is on its way at once. The order of the sum is the choices', whatever the slots'.
// Bound by memory: 5120 tokens of 2 x 8192 bf16 (252 MB) take 39 us, 6.4 TB/s (y was just written: a part
// of it comes from the caches).
template <bool OUT32>
__global__ void __launch_bounds__(256) combine_kernel(const CombineArgs a) {
  const int64_t t = blockIdx.y;
  const int64_t col = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (col >= a.n) return;
  float sum[8] = {};
  for (int j0 = 0; j0 < a.top_k; j0 += 4) {
    u32x4 v[4];
    float w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      v[u] = u32x4{};
      w[u] = 0.0f;
      if (j0 + u < a.top_k) {
        const int64_t slot = a.token_slot[t * a.top_k + j0 + u];
        if (slot >= 0 && slot < a.slots) {
          w[u] = a.weights[t * a.top_k + j0 + u];
          v[u] = *reinterpret_cast<const u32x4*>(a.y + slot * a.n + col);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float f[8];
      widen(v[u], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += w[u] * f[e];
    }
  }
  if constexpr (OUT32) {
    f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + t * a.n + col);
    p[0] = f32x4{sum[0], sum[1], sum[2], sum[3]};
    p[1] = f32x4{sum[4], sum[5], sum[6], sum[7]};
  } else {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + t * a.n + col) = narrow(sum);
  }
}

hipError_t launch_combine(const CombineArgs& a, hipStream_t stream) {
  // (grid.y is limited to 65535 blocks: more tokens go in further launches)
  for (int64_t t0 = 0; t0 < a.tokens; t0 += 65535) {
    CombineArgs p = a;
    p.tokens = a.tokens - t0 < 65535 ? a.tokens - t0 : 65535;
    p.token_slot = a.token_slot + t0 * a.top_k;
    p.weights = a.weights + t0 * a.top_k;
    p.out = static_cast<uint8_t*>(a.out) + t0 * a.n * (a.out_fp32 ? 4 : 2);
    const dim3 grid((unsigned)((a.n + 2047) / 2048), (unsigned)p.tokens);
    if (a.out_fp32) hipLaunchKernelGGL(combine_kernel<true>, grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL(combine_kernel<false>, grid, dim3(256), 0, stream, p);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace agg
