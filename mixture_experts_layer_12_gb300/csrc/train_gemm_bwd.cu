// train_gemm_bwd.cu -- train_gemm.cuh's products with transposed weights.
#include "train_gemm.cuh"

namespace moe {

cudaError_t launch_train_gemm_bwd(int op, const CUtensorMap& tm_a, const CUtensorMap& tm_b,
                                  const CUtensorMap& tm_a64, const TrainGemmArgs& a, int64_t max_tiles,
                                  cudaStream_t st) {
  if (op == kTrainBwdGelu) return train_launch<kTrainBwdGelu>(tm_a, tm_b, tm_a64, a, max_tiles, st);
  if (op == kTrainBwdSwiGLU) return train_launch<kTrainBwdSwiGLU>(tm_a, tm_b, tm_a64, a, max_tiles, st);
  if (op == kTrainRowsF32) return train_launch<kTrainRowsF32>(tm_a, tm_b, tm_a64, a, max_tiles, st);
  return train_launch<kTrainRows>(tm_a, tm_b, tm_a64, a, max_tiles, st);
}

cudaError_t train_gemm_bwd_set_attributes() {
  cudaError_t e = train_set_attributes<kTrainBwdGelu>();
  if (e == cudaSuccess) e = train_set_attributes<kTrainBwdSwiGLU>();
  if (e == cudaSuccess) e = train_set_attributes<kTrainRows>();
  if (e == cudaSuccess) e = train_set_attributes<kTrainRowsF32>();
  return e;
}

}  // namespace moe
