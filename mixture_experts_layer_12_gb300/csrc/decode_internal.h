// decode_internal.h -- launch interfaces between the decode entry points
// (decode_api.cu) and their kernels.  Not part of the public interface.
#pragma once

#include "moe_decode.h"
#include "moe_internal.h"

namespace moe {

// A run of rows that share one expert's weights: at most kDecRows rows,
// consecutive in dispatch order.
struct DecEntry {
  int32_t expert;
  int32_t row0;
  int32_t n;
  int32_t pad;
};

constexpr int kDecRows = 64;               // rows of an entry at most
constexpr int kDecMaxCtas = 152;           // CTAs of the streaming kernel
// entries: at most one per expert or segment, plus the row blocks that long
// ones are cut into
constexpr int kDecMaxEntries = kMaxExperts + MOED_MAX_ROWS / 8;

// Control block at the start of a workspace, cleared by the first kernel of
// every call.  bytes: [status 64 | grid barriers 64 | item counters | n_entries].
constexpr size_t kDecBarrierOffset = 64;
constexpr size_t kDecItemOffset = 128;    // kDecMaxCtas ints (<= 152 * 4 = 608 bytes)
constexpr size_t kDecCountOffset = 960;     // number of entries, rows of the longest
constexpr size_t kDecEntryOffset = 1024;    // entries
constexpr int kDecCtrlInts = 240;           // ints zeroed: everything before n_entries

// ---- kernel 1 of the layer: routing and dispatch by one cluster of 8 CTAs
struct DecRouteArgs {
  const uint16_t* x;   // [T, H]
  const uint16_t* w;   // [H, E]
  const float* bias;   // [E] or null
  int T, H, E, k;
  int capacity;        // -1: unlimited
  int gating;
  int32_t* ids;
  float* weights;
  int32_t* counts;
  int32_t* offsets;
  int32_t* perm;
  int32_t* slot;
  int* ctrl;           // control block
  DecEntry* entries;
  int row_block;       // rows of an entry at most
};
cudaError_t launch_decode_route(const DecRouteArgs& a, cudaStream_t st);

// ---- kernel 1 of the grouped products: entries from segment offsets
struct DecPrepArgs {
  const int32_t* seg_offsets;
  int n_segments, rows, E;
  int* ctrl;
  DecEntry* entries;
  int max_entries;     // room in `entries`
  int row_block;       // rows of an entry at most
};
cudaError_t launch_decode_prep(const DecPrepArgs& a, cudaStream_t st);

// ---- kernel 2: the weight stream (decode_ffn.cuh)
constexpr int kDecNone = 0;    // y = x W (grouped products)
constexpr int kDecGelu = 1;    // the layer, GELU experts
constexpr int kDecSwiGLU = 2;  // the layer, gated experts
struct DecFfnArgs {
  const int* ctrl;
  const DecEntry* entries;
  int max_entries;       // host bound on the number of entries
  unsigned* barrier;     // 3 grid barriers
  uint32_t arrivals;     // CTAs that they wait for: all (the self-test: one more than there are)
  unsigned* item_counts;
  float* parts;          // [CTAs][2][row_cap][128] partial tiles of the first product's split items (kDecPair: two)
  float* parts2;         // the second product's: the first's are still being read
  int row_cap;           // rows of an entry at most, rounded up to 8
  float* yfull;          // layer: [T*k, H] fp32 expert outputs of whole items
  uint16_t* h;           // layer: [T*k, F]
  const uint16_t* s1;    // 4-bit: scales
  const uint16_t* s2;
  int blocked1, blocked2;  // the tensor maps have column blocks (see DecFfnMaps)
  const uint16_t* x;
  const int32_t* perm;   // layer
  const int32_t* slot;   // layer
  const float* gate;     // layer
  uint16_t* y;
  int T, k;
  int act;               // kDec*
  int group;             // 4-bit: rows per scale; 0: bf16; kDecPair
  int K1, N1;            // first product: x [., K1] -> N1 columns of h (or y)
  int nb1, kc1;          // its column blocks and K chunks
  int least1, least2;    // chunks worth a CTA of their own
  int K2, N2, nb2, kc2;  // second product (layer)
  int* status;
  uint64_t wait_limit_ns;
};
// W [E, K, N] (4 bits: words [E, K/8, N]) with 128-byte swizzle.  Where the
// columns divide into blocks of 128 bytes (64 bf16, 32 words), gate and up
// separately: dimensions [E, blocks, K, block], a box of one expert, as many
// blocks as a 128- (gated: 64-) column half takes and one chunk's rows.
// Elsewhere: dimensions [E, K, N], a box of one block.  (kDecPair: the box is 128 columns.)
struct DecFfnMaps {
  CUtensorMap w1, w2;
};
constexpr int kDecBN = 128;    // columns of an item's weight tile
constexpr int kDecKC16 = 64;   // K rows of a chunk, bf16 weights
constexpr int kDecKC4 = 256;   // K rows of a chunk, 4-bit weights
// a `group` that says: bf16, gated, chunks of the gate and of the up projection in turn
constexpr int kDecPair = -1;
// one translation unit per weight type (bf16, the same in pairs; 4 bits with a scale
// per 32, 64 or 128 rows)
#define DECODE_FFN_UNIT(name)                                                                    \
  cudaError_t launch_decode_ffn_##name(const DecFfnMaps& m, const DecFfnArgs& a, int ctas,       \
                                       cudaStream_t st);                                         \
  cudaError_t decode_ffn_##name##_set_attributes();
DECODE_FFN_UNIT(bf16)
DECODE_FFN_UNIT(pair)
DECODE_FFN_UNIT(q4_32)
DECODE_FFN_UNIT(q4_64)
DECODE_FFN_UNIT(q4_128)
#undef DECODE_FFN_UNIT
cudaError_t decode_route_set_attributes();

// ---- 4-bit weights
cudaError_t launch_quantize_q4(int E, int K, int N, int group, const uint16_t* w, uint32_t* codes,
                               uint16_t* scales, cudaStream_t st);
cudaError_t launch_dequantize_q4(int E, int K, int N, int group, const uint32_t* codes,
                                 const uint16_t* scales, uint16_t* w, cudaStream_t st);

}  // namespace moe
