// train_internal.h -- launch interfaces between the training entry points
// (train_api.cu) and their kernels.  Not part of the public interface.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_internal.h"

namespace moe {

// ---- expert row segments as the backward pass lays them out.
// Compact rows (dispatch order): segment e holds rows [offsets[e],
// offsets[e+1]).  Padded rows: segment e starts at a multiple of 16 and its
// rows are followed by zero rows up to the next multiple of 16, so that a
// product that sums over a segment's rows in steps of 16 (the K of one
// tcgen05.mma) never reads a neighbour's rows.
constexpr int kSegPad = 16;
inline size_t padded_rows_cap(size_t rows, int E) {
  const size_t hit = rows < (size_t)E ? rows : (size_t)E;  // segments that hold rows
  return (rows + hit * (kSegPad - 1) + kSegPad - 1) / kSegPad * kSegPad;
}

// What a kernel knows of the segments: from `offsets` on the device, or
// (offsets null) `E` chunks of `chunk` rows of the `rows` there are, laid out
// without padding (chunk % 16 == 0).  Offsets that run backwards or past
// `rows` or overlap are cut so that no row is outside [0, rows) and no padded row
// outside the padded buffers, and set MOE_DEV_BAD_ID in the call's status.
struct SegArgs {
  const int32_t* offsets;  // [E+1] or null
  int E;
  int rows;        // row capacity of compact buffers
  int rows_pad;    // row capacity of padded buffers
  int chunk;
};

// ---- the products of training (train_gemm.cuh).
enum TrainOp {
  kTrainFwdGelu = 0,    // z = A W1[e] kept, out = GELU(z)
  kTrainFwdSwiGLU = 1,  // z = A [W_gate | W_up] kept, out = SiLU(z_gate) * z_up
  kTrainBwdGelu = 2,    // g = A W2[e]^T; dz, w h and <g, h> from the kept z
  kTrainBwdSwiGLU = 3,
  kTrainRows = 4,       // out = A W[e]^T
  kTrainPlain = 5,      // out32 = A W[e]
  kTrainWgrad = 6,      // out[e] = A_e^T B_e over a segment's rows
  kTrainWgradF32 = 7,   // the same in fp32
  kTrainRowsF32 = 8,    // out32 = A W[e]^T
  kTrainPlainBf16 = 9   // out = A W[e]
};

struct TrainGemmArgs {
  SegArgs seg;
  int M;        // Wgrad: rows of out (columns of A)
  int N;        // output columns (FwdSwiGLU, Bwd*: F)
  int K;        // reduction length (not Wgrad)
  int splits;   // Plain, RowsF32: parts of K, each a [rows, N] of out32
  int ksplit;   // stages of 64 in each of them (the last may have fewer)
  uint16_t* out;
  int ld_out;   // columns from one row of `out` to the next (not Wgrad)
  float* out32;
  // kept pre-activations, compact rows: bf16 [rows, halves * N], or int8
  // codes of that shape with scales [rows, halves * ceil(N / 32)]
  int keep_bits;
  void* z;
  uint8_t* z_scales;
  // Bwd: gate weight of compact row r is w[perm[r]] (w null: 1); dz [., halves
  // * N] and hw [., N] padded rows, ld_dz and ld_hw columns apart; part [rows, units] the sums of g * h over
  // 64 columns (null: not wanted)
  const float* w;
  const int32_t* perm;
  int n_w;      // entries of w
  uint16_t* dz;
  uint16_t* hw;
  int ld_dz, ld_hw;
  float* part;
  int units;
  const int* merge_status;  // a status word to take over, or null
  int* status;
  uint64_t wait_limit_ns;
};
// Operand boxes: A of row products {64, 128} and {64, 64} (tm_a64), of Wgrad
// {64, 64}; B of Fwd and Plain W [E, K, N] {64, 64, 1}, of Bwd and Rows W
// [E, N, K] {64, 128, 1}, of Wgrad {64, 64} (2D, as A).  Wgrad's third map is its
// output [E, M, N], box of 64 bytes x 32 rows, 64-byte swizzle.  max_tiles
// bounds the number of 256 x 256 tiles.
cudaError_t launch_train_gemm(int op, const CUtensorMap& tm_a, const CUtensorMap& tm_b,
                              const CUtensorMap& tm_a64, const TrainGemmArgs& a, int64_t max_tiles,
                              cudaStream_t st);
cudaError_t train_gemm_set_attributes();

// ---- rows and elements (train_rows.cu).
// dst[padded row] = src[perm ? perm[r] / k : r] for the rows r of every
// segment, zeros behind each (compact: dst[r], nothing behind); two (src, dst)
// pairs at once (src1 may be null).
struct GatherArgs {
  SegArgs seg;
  bool compact;
  const int32_t* perm;
  int T, H, k;
  int ld;  // columns from one row of dst to the next
  const uint16_t* src[2];
  uint16_t* dst[2];
};
cudaError_t launch_train_gather(const GatherArgs& a, int sms, cudaStream_t st);

// out[t] = (add ? add[t] : 0) + sum_j (w ? w[t, j] : 1) * rows[slot[t, j]]
//          + (dl ? sum_j dl[t, j] * wt[ids[t, j]] : 0)
// (fp32, in that order, j ascending), rounded to bf16 once; rows in bf16 or fp32
// (both null: none), wt [E, H] bf16.  add (fp32) and w go with rows in fp32 only,
// which may be `splits` parts of T * k rows each, summed in their order.  With
// `range` (offsets of E segments) slot[t, 0] is t for the rows t inside the
// segments, and the others are not written.
struct RowsSumArgs {
  const uint16_t* rows;
  const float* rows32;
  int splits;
  const int32_t* range;
  const float* w;
  const int32_t* slot;
  const float* add;
  int T, H, k;
  uint16_t* out;
  const float* dl;
  const int32_t* ids;
  const uint16_t* wt;
  int E;
};
cudaError_t launch_rows_sum(const RowsSumArgs& a, cudaStream_t st);

struct CombineBackwardArgs {
  const uint16_t* dy;
  const uint16_t* Y;
  const float* w;
  const int32_t* slot;
  int T, H, k;
  uint16_t* dY;
  float* dw;
};
cudaError_t launch_combine_backward(const CombineBackwardArgs& a, cudaStream_t st);

cudaError_t launch_quantize_a8(int64_t rows, int cols, const uint16_t* x, int8_t* codes,
                               uint8_t* scales, int sms, cudaStream_t st);
cudaError_t launch_dequantize_a8(int64_t rows, int cols, const int8_t* codes, const uint8_t* scales,
                                 uint16_t* out, int sms, cudaStream_t st);

// The gate's gradient: dlogits as two bf16 numbers (the second is what the
// first one's rounding left), dl [T, 2 ep], and sums of 16 tokens' dlogits.
constexpr int kGateTokens = 16;
struct GateBackwardArgs {
  int T, E, k, ep;
  int gating;
  const int32_t* ids;
  const float* weights;
  const float* probs;  // [T, E], MOE_GATE_SOFTMAX_TOPK only
  const float* dw;     // [T, k], or null: sums of part[slot[t, j]][0 .. units)
  const float* part;
  const int32_t* slot;
  int rows, units;
  uint16_t* dl;
  float* dlk;          // [T, k], the chosen experts' dlogits in fp32, or null
  float* db_part;      // [ceil(T / 16), E]
  // W_router [H, E] on the way: transposed into wt [E, H] bf16, or (wt null)
  // twice side by side into w2 [H, 2 ep], zeros between
  const uint16_t* w_router;
  int H;
  uint16_t* wt;
  uint16_t* w2;
};
cudaError_t launch_gate_backward(const GateBackwardArgs& a, cudaStream_t st);

// dw_router[h, e] = sum over S of part[s, h, e] + part[s, h, ep + e];
// db[e] = sum of the token blocks' sums (null: not wanted).
struct RouterReduceArgs {
  int H, E, ep, S;
  const float* part;   // [S, H, 2 ep]
  uint16_t* dw_router;
  const float* db_part;
  int n_db;
  float* db;
};
cudaError_t launch_router_reduce(const RouterReduceArgs& a, cudaStream_t st);

// probs[t] = softmax(sum over S of logits[s, t] + bias) over E of ldl columns
cudaError_t launch_router_softmax(const float* logits, int S, int ldl, const float* bias, int T, int E,
                                  float* probs, cudaStream_t st);

}  // namespace moe
