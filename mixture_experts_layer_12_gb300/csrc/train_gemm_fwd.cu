// train_gemm_fwd.cu -- train_gemm.cuh's products of the forward pass.
#include "train_gemm.cuh"

namespace moe {

cudaError_t launch_train_gemm_fwd(int op, const CUtensorMap& tm_a, const CUtensorMap& tm_b,
                                  const CUtensorMap& tm_a64, const TrainGemmArgs& a, int64_t max_tiles,
                                  cudaStream_t st) {
  if (op == kTrainFwdGelu) return train_launch<kTrainFwdGelu>(tm_a, tm_b, tm_a64, a, max_tiles, st);
  if (op == kTrainFwdSwiGLU) return train_launch<kTrainFwdSwiGLU>(tm_a, tm_b, tm_a64, a, max_tiles, st);
  if (op == kTrainPlainBf16) return train_launch<kTrainPlainBf16>(tm_a, tm_b, tm_a64, a, max_tiles, st);
  return train_launch<kTrainPlain>(tm_a, tm_b, tm_a64, a, max_tiles, st);
}

cudaError_t train_gemm_fwd_set_attributes() {
  cudaError_t e = train_set_attributes<kTrainFwdGelu>();
  if (e == cudaSuccess) e = train_set_attributes<kTrainFwdSwiGLU>();
  if (e == cudaSuccess) e = train_set_attributes<kTrainPlain>();
  if (e == cudaSuccess) e = train_set_attributes<kTrainPlainBf16>();
  return e;
}

}  // namespace moe
