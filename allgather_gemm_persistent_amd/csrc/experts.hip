// The experts' products (moe_gemm): out[s] = A[slot_token[s]] @ B[e] for the slots s of expert e,
// e = 0 .. n_experts - 1, with the slots of one expert side by side.
//
// Two kernels. Many rows an expert: the persistent MFMA kernel of gemm_kernel.h over the tiles of
// all experts (kEpiExperts), bound by the matrix units. Few rows an expert: the streaming
// kernel of stream_kernel.h, bound by reading every weight once.
#include "stream_kernel.h"

namespace agg {

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

hipError_t launch_expert_stream(const StreamArgs& args, int dtype, hipStream_t stream) {
  const dim3 grid((unsigned)(args.strips * args.ksplit), (unsigned)args.x.n_experts), block(kStreamWaves * 64);
  if (dtype == AGG_FP8_E4M3) {
    if (args.x.gated) hipLaunchKernelGGL((expert_stream_kernel<true, true, false>), grid, block, 0, stream, args);
    else hipLaunchKernelGGL((expert_stream_kernel<true, false, false>), grid, block, 0, stream, args);
  } else {
    if (args.x.gated) hipLaunchKernelGGL((expert_stream_kernel<false, true, false>), grid, block, 0, stream, args);
    else hipLaunchKernelGGL((expert_stream_kernel<false, false, false>), grid, block, 0, stream, args);
  }
  return hipGetLastError();
}

}  // namespace agg
