// The product with an epilogue (linear): out = act(A B + bias) + residual. The kernels are those of the experts' products
// with one expert that holds every row: tiles on the matrix units (gemm_kernel.h, kEpiLinear) where the rows are many,
// bound by the matrix units; the weight streamed through registers (stream_kernel.h) where they are few, bound by
// reading it once.
//
// rows x columns x K, with a bf16 residual or a bias:
//   16 x 10240 x 8192 bf16, streamed                     31.9 us    5.3 TB/s
//   128 x 8192 x 8192 fp8, 128 x 64 tiles, K in two      25.6 us    2.7 TB/s (34 where nothing of the weight is cached)
//   4096 x 8192 x 8192 bf16, 256 x 256 tiles             406 - 414 us    1328 - 1354 TFLOP/s
//   777 x 1000 x 1032 bf16, GELU, 64 x 64 tiles          10.8 us    latency: 17 slices of K in turn
// Between some 32 and 256 rows neither bound is near. Rows of B that are a multiple of 1024 bytes apart cost most (32 rows,
// fp8, 128 x 64 tiles, nothing of the weight cached: 8192 columns 27.2 us, 8128 21.9, 6144, on fewer compute units, 27.2;
// one part of K 41 and 30), whichever XCD takes which columns, whatever A's stride or the loads' cache policy, and more in
// flight does not help (a ring of five slice pairs instead of four: 34.2 -> 34.7 us at 128 rows). B's loads non-temporal
// gain 2 to 8% there, but lose 20% where the last level holds the weight. Wider tiles need K in more parts, whose
// sums pass through memory (128 rows: 128 x 128, four parts: 33.9; 64 x 64, whole: 40.4).
#include "stream_kernel.h"

namespace agg {

template <int BM, int BN, int DT>
static hipError_t launch_tiles(const GemmArgs& args, int grid, hipStream_t stream) {
  hipLaunchKernelGGL((gemm_kernel<BM, BN, DT, kEpiLinear>), dim3(grid), dim3(kThreads), 0, stream, args);
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

hipError_t launch_linear_tiles(const GemmArgs& args, int bm, int bn, int dtype, int grid, hipStream_t stream) {
  if (dtype == AGG_BF16) return launch_tiles_shape<AGG_BF16>(args, bm, bn, grid, stream);
  return launch_tiles_shape<AGG_FP8_E4M3>(args, bm, bn, grid, stream);
}

hipError_t launch_linear_stream(const StreamArgs& args, int dtype, hipStream_t stream) {
  const dim3 grid((unsigned)(args.strips * args.ksplit)), block(kStreamWaves * 64);
  if (dtype == AGG_FP8_E4M3) hipLaunchKernelGGL((expert_stream_kernel<true, false, true>), grid, block, 0, stream, args);
  else hipLaunchKernelGGL((expert_stream_kernel<false, false, true>), grid, block, 0, stream, args);
  return hipGetLastError();
}

}  // namespace agg
