// The experts' products (moe_gemm): out[s] = A[slot_token[s]] @ B[e] for the slots s of expert e,
// e = 0 .. n_experts - 1, with the slots of one expert side by side.
//
// Two kernels. Many rows an expert: the persistent MFMA kernel of gemm_kernel.h over the tiles of
// all experts (kEpiExperts), bound by the matrix units. Few rows an expert: expert_stream_kernel
// below, bound by reading every weight once.
#include "gemm_kernel.h"
#include "moe.h"

namespace agg {

typedef long i64x1;

__device__ inline f32x4 mfma16(const u32x4& b, const u32x4& a, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c,
                                                 0, 0, 0);
}
__device__ inline f32x4 mfma16(const u32x2& b, const u32x2& a, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(__builtin_bit_cast(i64x1, b), __builtin_bit_cast(i64x1, a), c,
                                                    0, 0, 0);
}

// Few rows an expert: a workgroup of 8 waves holds a strip of B's columns (128 bf16 or 256 fp8) of
// one expert and all of K, each wave every eighth block of 32 K rows; rows are taken 16 * RB at a
// time (B is read again for more).
//
// B goes from memory to registers, without LDS: lane l loads 16 bytes (CW columns) of each of the 8
// K rows 8 * (l / 16) .. + 7 of a block at column chunk l % 16, so one instruction reads 256 bytes
// in a row from 4 rows. The MFMA wants 8 consecutive K of one column in a lane; those are the 8
// loaded rows at a fixed column of the lane's chunk, so the transposition stays inside the lane:
// byte permutes (32 for 8 KiB of bf16, 64 of fp8, far below what the memory leaves time for).
// Fragment c of the wave then holds column c of every lane's chunk, i.e. MFMA c computes columns
// 16-byte-chunk * CW + c. Two blocks per wave are loaded ahead, 16 waves a CU: 256 KiB in flight.
// The 8 partial sums meet in LDS in wave order, so the result does not depend on timing.
constexpr int kStreamWaves = 8;

template <int RB, bool FP8>
__global__ void __launch_bounds__(kStreamWaves * 64) expert_stream_kernel(const StreamArgs a) {
  constexpr int CW = FP8 ? 16 : 8;           // columns of a lane's 16 bytes
  constexpr int SC = 16 * CW;                // columns of a strip
  constexpr int EL = FP8 ? 1 : 2;
  constexpr int HC = 128;                    // columns summed per pass over LDS
  constexpr int PC = HC + 4;                 // padded row of a pass
  using Frag = std::conditional_t<FP8, u32x2, u32x4>;
  __shared__ __attribute__((aligned(16))) float part[kStreamWaves][16][PC];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = lane & 15, kq = lane >> 4;
  const int expert = blockIdx.y;
  const int lo = __builtin_amdgcn_readfirstlane((int)expert_bound(a.x, expert));
  const int end = __builtin_amdgcn_readfirstlane((int)expert_bound(a.x, expert + 1));
  if (lo >= end) return;
  const int N = (int)a.N, K = (int)a.K, NO = a.x.gated ? N / 2 : N;
  const int strip = blockIdx.x;

  // this lane's chunk of B's columns; gated: the strip holds SC/2 gate columns (chunks 0..7) and
  // their up columns (chunks 8..15)
  int col, col_end;
  if (a.x.gated) {
    col = strip * (SC / 2) + (g & 7) * CW;
    col_end = NO;
    if (col < col_end && g >= 8) { col += NO; col_end = N; }
  } else {
    col = strip * SC + g * CW;
    col_end = N;
  }
  const uint32_t row_bytes = (uint32_t)N * EL;
  const uint32_t b0 = col < col_end ? (uint32_t)col * EL : kOutOfRange;
  const __amdgpu_buffer_rsrc_t db = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(a.b) + (int64_t)expert * N * K * EL, 0, (int)((int64_t)N * K * EL), kBufferFlags);
  const int blocks = (K + 31) / 32;

  for (int r0 = lo; r0 < end; r0 += 16 * RB) {
    uint32_t a0[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int s = r0 + r * 16 + g;
      a0[r] = kOutOfRange;
      if (s < end) {
        const int64_t ar = a.x.slot_token ? (int64_t)a.x.slot_token[s] : (int64_t)s - r0;
        if (ar >= 0 && (!a.x.slot_token || ar < a.x.a_rows)) a0[r] = (uint32_t)ar * (uint32_t)a.x.a_stride;
      }
    }
    const int held = end - r0 < 16 * RB ? end - r0 : 16 * RB;
    const int64_t rows = a.x.slot_token ? a.x.a_rows : (int64_t)held;
    const __amdgpu_buffer_rsrc_t da = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(a.a) + (a.x.slot_token ? 0 : (int64_t)r0 * a.x.a_stride), 0,
        (int)((rows - 1) * a.x.a_stride + (int64_t)K * EL), kBufferFlags);

    f32x4 acc[CW][RB];
#pragma unroll
    for (int c = 0; c < CW; ++c)
#pragma unroll
      for (int r = 0; r < RB; ++r) acc[c][r] = f32x4{};

    struct Block {
      u32x4 b[8];
      Frag a[RB];
    };
    // block kb of 32 K rows; past the end of K every lane's offset is out of range (reads zeros):
    // K is a multiple of 8, so a lane's 8 rows lie inside K or outside it together
    auto load = [&](Block& x, int kb) {
      const int k0 = kb * 32 + kq * 8;
      const uint32_t out = k0 < K ? 0u : kOutOfRange;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x.b[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                     db, (int)((b0 + (uint32_t)(k0 + i) * row_bytes) | out | (b0 & kOutOfRange)), 0, 2));
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        const int off = (int)((a0[r] + (uint32_t)k0 * EL) | out | (a0[r] & kOutOfRange));
        if constexpr (FP8) x.a[r] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(da, off, 0, 0));
        else x.a[r] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(da, off, 0, 0));
      }
    };
    auto compute = [&](const Block& x) {
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        if constexpr (!FP8) {
          // dword d holds columns 2d (low half) and 2d + 1
          u32x4 f0, f1;
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            f0[p] = __builtin_amdgcn_perm(x.b[2 * p + 1][d], x.b[2 * p][d], 0x05040100u);
            f1[p] = __builtin_amdgcn_perm(x.b[2 * p + 1][d], x.b[2 * p][d], 0x07060302u);
          }
#pragma unroll
          for (int r = 0; r < RB; ++r) {
            acc[2 * d][r] = mfma16(f0, x.a[r], acc[2 * d][r]);
            acc[2 * d + 1][r] = mfma16(f1, x.a[r], acc[2 * d + 1][r]);
          }
        } else {
          // dword d holds columns 4d .. 4d + 3: a 4 x 4 byte transposition of rows 0..3 and of 4..7
          u32x2 f[4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t q0 = x.b[4 * h][d], q1 = x.b[4 * h + 1][d], q2 = x.b[4 * h + 2][d], q3 = x.b[4 * h + 3][d];
            const uint32_t t0 = __builtin_amdgcn_perm(q1, q0, 0x05010400u), t1 = __builtin_amdgcn_perm(q1, q0, 0x07030602u);
            const uint32_t u0 = __builtin_amdgcn_perm(q3, q2, 0x05010400u), u1 = __builtin_amdgcn_perm(q3, q2, 0x07030602u);
            f[0][h] = __builtin_amdgcn_perm(u0, t0, 0x05040100u);
            f[1][h] = __builtin_amdgcn_perm(u0, t0, 0x07060302u);
            f[2][h] = __builtin_amdgcn_perm(u1, t1, 0x05040100u);
            f[3][h] = __builtin_amdgcn_perm(u1, t1, 0x07060302u);
          }
#pragma unroll
          for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[4 * d + c][r] = mfma16(f[c], x.a[r], acc[4 * d + c][r]);
        }
      }
    };
    Block x0, x1, x2;
    int kb = wave;
    load(x0, kb);
    load(x1, kb + kStreamWaves);
    for (; kb < blocks; kb += 3 * kStreamWaves) {
      load(x2, kb + 2 * kStreamWaves);
      compute(x0);
      load(x0, kb + 3 * kStreamWaves);
      compute(x1);
      load(x1, kb + 4 * kStreamWaves);
      compute(x2);
    }

    // ---- the waves' partial sums, HC columns and 16 rows a pass: lane l holds, of row l % 16,
    // columns (4 * (l / 16) + i) * CW + c
#pragma unroll
    for (int r = 0; r < RB; ++r) {
#pragma unroll
      for (int h = 0; h < SC / HC; ++h) {
        // (fp8: pass h takes columns h * 8 .. + 7 of every chunk, bf16: all 8)
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 8; c += 4)
            *reinterpret_cast<f32x4*>(&part[wave][g][(4 * kq + i) * 8 + c]) =
                f32x4{acc[h * 8 + c][r][i], acc[h * 8 + c + 1][r][i], acc[h * 8 + c + 2][r][i], acc[h * 8 + c + 3][r][i]};
        __syncthreads();
        auto total = [&](int row, int c4) {
          f32x4 v = *reinterpret_cast<const f32x4*>(&part[0][row][c4]);
#pragma unroll
          for (int w = 1; w < kStreamWaves; ++w) v += *reinterpret_cast<const f32x4*>(&part[w][row][c4]);
          return v;
        };
        // pass column c4 is column h * 8 + c4 % 8 of chunk c4 / 8
        const int row = tid >> 5, c4 = (tid & 31) * 4;
        const int64_t s = (int64_t)r0 + r * 16 + row;
        float rs = 1.0f;
        if (FP8 && s < end) {
          const int64_t ar = a.x.slot_token ? (int64_t)a.x.slot_token[s] : s;
          rs = (ar >= 0 && ar < a.x.a_rows) ? a.x.a_scale[ar] : 0.0f;
        }
        const int chunk = c4 >> 3, in = h * 8 + (c4 & 7);
        auto store = [&](int n, const f32x4& v) {
          u32x2 packed;
          packed[0] = bf16x2_rne(v[0], v[1]);
          packed[1] = bf16x2_rne(v[2], v[3]);
          *reinterpret_cast<u32x2*>(a.c + s * NO + n) = packed;
        };
        if (!a.x.gated) {
          const int n = strip * SC + chunk * CW + in;
          if (s < end && n < N) {
            f32x4 v = total(row, c4);
            if (FP8) v *= *reinterpret_cast<const f32x4*>(a.x.b_scale + (int64_t)expert * N + n) * rs;
            store(n, v);
          }
        } else if (chunk < 8) {
          const int n = strip * (SC / 2) + chunk * CW + in;
          if (s < end && n < NO) {
            f32x4 gt = total(row, c4), up = total(row, c4 + 64);
            if (FP8) {
              gt *= *reinterpret_cast<const f32x4*>(a.x.b_scale + (int64_t)expert * N + n) * rs;
              up *= *reinterpret_cast<const f32x4*>(a.x.b_scale + (int64_t)expert * N + NO + n) * rs;
            }
            store(n, f32x4{silu(gt[0]) * up[0], silu(gt[1]) * up[1], silu(gt[2]) * up[2], silu(gt[3]) * up[3]});
          }
        }
      }
    }
  }
}

template <int BM, int BN, int DT>
static hipError_t launch_tiles(const GemmArgs& args, int grid, hipStream_t stream) {
  hipLaunchKernelGGL((gemm_kernel<BM, BN, DT, kEpiExperts>), dim3(grid), dim3(kThreads), 0, stream, args);
  return hipGetLastError();
}

template <int DT>
static hipError_t launch_tiles_shape(const GemmArgs& args, int bm, int bn, int grid, hipStream_t s) {
  if (bm == 256 && bn == 256) return launch_tiles<256, 256, DT>(args, grid, s);
  if (bm == 256 && bn == 224) return launch_tiles<256, 224, DT>(args, grid, s);
  if (bm == 128 && bn == 128) return launch_tiles<128, 128, DT>(args, grid, s);
  if (bm == 128 && bn == 64) return launch_tiles<128, 64, DT>(args, grid, s);
  if (bm == 64 && bn == 64) return launch_tiles<64, 64, DT>(args, grid, s);
  return hipErrorInvalidValue;
}

hipError_t launch_expert_tiles(const GemmArgs& args, int bm, int bn, int dtype, int grid, hipStream_t stream) {
  if (dtype == AGG_BF16) return launch_tiles_shape<AGG_BF16>(args, bm, bn, grid, stream);
  return launch_tiles_shape<AGG_FP8_E4M3>(args, bm, bn, grid, stream);
}

template <int RB, bool FP8>
static hipError_t launch_stream(const StreamArgs& args, hipStream_t stream) {
  const int64_t cols = FP8 ? 256 : 128;
  const int64_t strips = (args.N + cols - 1) / cols;
  hipLaunchKernelGGL((expert_stream_kernel<RB, FP8>), dim3((unsigned)strips, (unsigned)args.x.n_experts),
                     dim3(kStreamWaves * 64), 0, stream, args);
  return hipGetLastError();
}

hipError_t launch_expert_stream(const StreamArgs& args, int row_blocks, int dtype, hipStream_t stream) {
  if (dtype == AGG_FP8_E4M3)
    return row_blocks == 1 ? launch_stream<1, true>(args, stream) : launch_stream<2, true>(args, stream);
  if (row_blocks == 1) return launch_stream<1, false>(args, stream);
  return row_blocks == 2 ? launch_stream<2, false>(args, stream) : launch_stream<4, false>(args, stream);
}

}  // namespace agg
