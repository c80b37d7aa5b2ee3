// train_gemm_wgrad.cu -- train_gemm.cuh's weight gradients, and the choice of
// the kernel for a product.
#include "train_gemm.cuh"

namespace moe {

cudaError_t launch_train_gemm_fwd(int op, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                  const TrainGemmArgs&, int64_t, cudaStream_t);
cudaError_t launch_train_gemm_bwd(int op, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                  const TrainGemmArgs&, int64_t, cudaStream_t);
cudaError_t train_gemm_fwd_set_attributes();
cudaError_t train_gemm_bwd_set_attributes();

cudaError_t launch_train_gemm(int op, const CUtensorMap& tm_a, const CUtensorMap& tm_b,
                              const CUtensorMap& tm_a64, const TrainGemmArgs& a, int64_t max_tiles,
                              cudaStream_t st) {
  switch (op) {
    case kTrainFwdGelu:
    case kTrainFwdSwiGLU:
    case kTrainPlain:
    case kTrainPlainBf16: return launch_train_gemm_fwd(op, tm_a, tm_b, tm_a64, a, max_tiles, st);
    case kTrainBwdGelu:
    case kTrainBwdSwiGLU:
    case kTrainRows:
    case kTrainRowsF32: return launch_train_gemm_bwd(op, tm_a, tm_b, tm_a64, a, max_tiles, st);
    case kTrainWgrad: return train_launch<kTrainWgrad>(tm_a, tm_b, tm_a64, a, max_tiles, st);
    default: return train_launch<kTrainWgradF32>(tm_a, tm_b, tm_a64, a, max_tiles, st);
  }
}

cudaError_t train_gemm_set_attributes() {
  cudaError_t e = train_gemm_fwd_set_attributes();
  if (e == cudaSuccess) e = train_gemm_bwd_set_attributes();
  if (e == cudaSuccess) e = train_set_attributes<kTrainWgrad>();
  if (e == cudaSuccess) e = train_set_attributes<kTrainWgradF32>();
  return e;
}

}  // namespace moe
