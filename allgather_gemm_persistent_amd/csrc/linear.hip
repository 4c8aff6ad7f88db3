// The product with an epilogue (linear): out = act(A B + bias) + residual. The kernels are those of the experts' products
// with one expert that holds every row: tiles on the matrix units (gemm_kernel.h, kEpiLinear) where the rows are many,
// bound by the matrix units; the weight streamed through registers (stream_kernel.h) where they are few, bound by
// reading it once.
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
