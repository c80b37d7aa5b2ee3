// decode_ffn_q4_64.cu -- the weight stream of the decode operators for 4-bit weights with a scale per 64 rows
// (decode_ffn.cuh); a translation unit of its own so that they compile side by side.
#include "decode_ffn.cuh"

namespace moe {

cudaError_t launch_decode_ffn_q4_64(const DecFfnMaps& m, const DecFfnArgs& a, int ctas, cudaStream_t st) {
  return ffn_rows<64>(m, a, ctas, st);
}
cudaError_t decode_ffn_q4_64_set_attributes() { return ffn_attrs<64>(); }

}  // namespace moe
