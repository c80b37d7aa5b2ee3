// decode_ffn_bf16.cu -- the weight stream of the decode operators for bf16 weights
// (decode_ffn.cuh); a translation unit of its own so that they compile side by side.
#include "decode_ffn.cuh"

namespace moe {

cudaError_t launch_decode_ffn_bf16(const DecFfnMaps& m, const DecFfnArgs& a, int ctas, cudaStream_t st) {
  return ffn_rows<0>(m, a, ctas, st);
}
cudaError_t decode_ffn_bf16_set_attributes() { return ffn_attrs<0>(); }

}  // namespace moe
