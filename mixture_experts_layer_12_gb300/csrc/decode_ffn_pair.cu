// decode_ffn_pair.cu -- the weight stream of the decode operators for gated
// bf16 experts whose gate's and up projection's chunks alternate
// (decode_ffn.cuh); a translation unit of its own so that they compile side by side.
#include "decode_ffn.cuh"

namespace moe {

cudaError_t launch_decode_ffn_pair(const DecFfnMaps& m, const DecFfnArgs& a, int ctas, cudaStream_t st) {
  return ffn_rows<kDecPair>(m, a, ctas, st);
}
cudaError_t decode_ffn_pair_set_attributes() { return ffn_attrs<kDecPair>(); }

}  // namespace moe
