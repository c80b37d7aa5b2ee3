// train_gemm.cuh -- the products of a training step on the 5th-generation
// tensor cores, grouped by expert.
//
// For the rows r of expert e (A_e = its rows of A):
//   Fwd    z = A_e W1[e], kept in bf16 or 8 bits; h = act(z)
//   Bwd    g = A_e W2[e]^T with A the rows' dy; from the kept z:
//          dz = w g act'(z), w h, and <g, h> (the gate weight's gradient)
//   Rows   out = A_e W[e]^T                     (dxp = dz W1^T)
//   Wgrad  out[e] = A_e^T B_e                   (dW2 = (w h)^T dy, dW1 = xp^T dz)
//   Plain  out = A_e W[e], fp32 or bf16          (Y = h W2, the router's logits)
//
// One design serves all (as the forward's expert GEMM): CTA pairs run the
// 2-SM tcgen05.mma (M = 256, N = 256, K = 16, fp32 in TMEM), each CTA holding
// 128 rows of A and 128 columns of B per 64-deep stage, five or six stages fed by
// one TMA thread, one MMA thread in the leader, and an epilogue double-buffered
// against the next tile.  8192 rows of 8 experts of 4096 x 14336: 600-625 us each
// of the six products while the card is cool, 1.54-1.60 PFLOP/s (back to back under
// the power cap 1.35: the four of a backward and their row copies 2840-2910 us);
// without any epilogue 2-5% less: the rest
// is the main loop, 0.38 us a stage where the MMAs alone would take 0.27, with
// shared memory filled and read at its rate meanwhile (a quarter less to read out
// of L2, A shared by two pairs through multicast, changed nothing).  What differs
// is the operands' major and the epilogue:
//   * transposed weights are K-major operands of the same bytes: W2 [E, F, H]
//     read as [N = F rows, K = H] needs no transposed copy;
//   * Wgrad's operands are both MN-major ([K = rows, M] and [K = rows, N]):
//     row-major activations as they are.  Its K is an expert's row count, any
//     number: rows are padded to 16 with zeros (SegTable), the box of a stage
//     may reach past them, but only the K steps of the expert's own 16-row
//     groups are issued, so a neighbour's infinities or NaN stay its own;
//   * the Bwd epilogue never writes g: it reads the kept z, one 32-column
//     chunk ahead, and leaves the two operands that the remaining products
//     need.  <g, h> makes dw without the experts' output Y, which therefore is
//     not kept: dw = dy . (h W2) = (dy W2^T) . h.
// Two epilogue warps per TMEM lane quadrant share a tile's columns: the Bwd
// epilogue reads and writes 8 to 16 bytes a column and is the longer half of a
// tile with K below 2000.
// Every mbarrier wait is bounded (MOE_DEV_TIMEOUT on expiry).
#pragma once

#include <atomic>

#include "train_seg.cuh"

namespace moe {
namespace {

constexpr int TBM = 128;            // rows per CTA
constexpr int TPAIR_M = 2 * TBM;    // rows per pair tile
constexpr int TBN = 256;            // columns per pair tile
constexpr int TBK = 64;
constexpr int TSTAGES = 6;          // at most (TrainTraits)
constexpr int TACC = 2;
constexpr int T_OP_BYTES = 128 * TBK * 2;  // a CTA's half of either operand: 16 KB
constexpr int T_BOX = 64 * TBK * 2;        // one 64-column MN-major box: 8 KB
constexpr int T_STAGE_BYTES = 2 * T_OP_BYTES;
constexpr int T_MMA_WARP = 1;
constexpr int T_EPI_WARP0 = 2;
constexpr int T_EPI_WARPS = 8;  // two per TMEM lane quadrant (warp % 4)
constexpr int T_THREADS = 32 * (T_EPI_WARP0 + T_EPI_WARPS);
constexpr int T_TMEM_COLS = TACC * TBN;
constexpr uint16_t T_PAIR_MASK = 0x3;

struct TrainCtrl {
  uint64_t full[TSTAGES];
  uint64_t empty[TSTAGES];
  uint64_t tfull[TACC];
  uint64_t tempty[TACC];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int tile_start[kMaxExperts + 1];
  SegTable seg;
};
constexpr int T_TURN = 2048;  // 32 rows x 64 bytes between a warp's threads and memory

template <int OP>
struct TrainTraits {
  static constexpr bool FWD = OP == kTrainFwdGelu || OP == kTrainFwdSwiGLU;
  static constexpr bool BWD = OP == kTrainBwdGelu || OP == kTrainBwdSwiGLU;
  static constexpr bool GATED = OP == kTrainFwdSwiGLU || OP == kTrainBwdSwiGLU;
  static constexpr bool PAIRED = OP == kTrainFwdSwiGLU;  // a tile holds 128 gate and 128 up columns
  static constexpr bool WGRAD = OP == kTrainWgrad || OP == kTrainWgradF32;
  static constexpr bool A_MN = WGRAD;
  static constexpr bool B_MN = !(BWD || OP == kTrainRows || OP == kTrainRowsF32);
  static constexpr bool A_PADDED = !(FWD || OP == kTrainPlain || OP == kTrainPlainBf16);
  static constexpr bool SPLIT = OP == kTrainPlain || OP == kTrainRowsF32;
  static constexpr bool OUT32 = OP == kTrainPlain || OP == kTrainWgradF32 || OP == kTrainRowsF32;
  static constexpr int BN_OUT = PAIRED ? TBN / 2 : TBN;
  // the epilogue's buffers per warp (FWD: z and h, BWD: z turned into dz, and
  // w h, Wgrad: a ring), and the stages that fit beside them
  static constexpr int HALVES = GATED ? 2 : 1;
  static constexpr int BUFS = FWD || BWD ? HALVES + 1 : WGRAD ? 3 : 1;
  static constexpr int STAGES = FWD || BWD || WGRAD ? 5 : TSTAGES;
  static constexpr size_t SMEM =
      1024 + (size_t)STAGES * T_STAGE_BYTES + T_EPI_WARPS * BUFS * T_TURN + sizeof(TrainCtrl);
  static_assert(SMEM <= 232448, "shared memory of one CTA");
};

struct TrainTile {
  int e, nb;
  int base;    // the tile's first row within the segment (Wgrad: row of out)
  int kb;      // stages
  int ks, k0;  // part of K, its first stage
  int k16;     // Wgrad: K steps of 16 in all
  bool half;   // M = 128 tile: 64 rows per CTA
  bool nhalf;  // N = 128 tile
};

// Tiles run segment-major, row-block fastest, so that pairs at work at the
// same time share the columns of B through L2.  An M block with at most 128
// rows runs as an M = 128 MMA (TMEM lanes 0-63: the CTA's 64 rows, columns
// 0..127; lanes 64-127: the same rows, columns 128..255), else an N block
// with at most 128 columns as N = 128.  With paired gate and up columns such an
// M block's CTA loads 64 gate and 64 up columns of the same outputs, so that both
// land in the same lanes; N blocks stay whole.
template <int OP>
__device__ __forceinline__ TrainTile train_tile(const TrainCtrl& c, const TrainGemmArgs& p, int tile,
                                                int& e) {
  using TT = TrainTraits<OP>;
  while (tile >= c.tile_start[e + 1]) ++e;
  const int local = tile - c.tile_start[e];
  const int m = TT::WGRAD ? p.M : c.seg.rows[e];
  const int mbs = (m + TPAIR_M - 1) / TPAIR_M;
  const int mb = local % mbs;
  TrainTile t;
  t.e = e;
  t.nb = local / mbs;
  t.ks = 0;
  t.k0 = 0;
  if constexpr (TT::SPLIT) {
    t.ks = t.nb % p.splits;
    t.nb /= p.splits;
    t.k0 = t.ks * p.ksplit;
  }
  t.base = mb * TPAIR_M;
  if constexpr (TT::WGRAD) {
    t.k16 = (c.seg.rows[e] + 15) / 16;
    t.kb = (t.k16 + 3) / 4;
  } else {
    t.k16 = 0;
    t.kb = (p.K + TBK - 1) / TBK;
    if constexpr (TT::SPLIT) t.kb = min(p.ksplit, t.kb - t.k0);
  }
  t.half = m - t.base <= TPAIR_M / 2;
  t.nhalf = !TT::PAIRED && !t.half && p.N - t.nb * TBN <= TBN / 2;
  return t;
}

__device__ __forceinline__ bool train_wait_drain(uint64_t* bar, uint32_t parity, uint64_t limit_ns,
                                                 int* status) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait(a, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(a, parity)) {
    if (global_timer_ns() - t0 > limit_ns) {
      record_status(status, MOE_DEV_TIMEOUT);
      return false;
    }
  }
  return true;
}

// The epilogues' instructions bound the products with short K (a gated Bwd tile
// of 256 x 256 took 22 us of them beside 11 of MMAs with K = 2048), so they use
// the special-function unit's own exponential and reciprocal.
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// erfc(|z| / sqrt 2) and exp(-z^2 / 2): Abramowitz & Stegun, Handbook of
// Mathematical Functions, formula 7.1.26 (|error| <= 1.5e-7); the exponential
// it needs is the normal density's.
__device__ __forceinline__ float train_erfc(float z, float& ex) {
  const float t = rcp_fast(fmaf(0.3275911f * 0.70710678118654752440f, fabsf(z), 1.0f));
  const float poly =
      t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f),
               0.254829592f);
  ex = exp2_fast(z * z * -0.72134752044448170368f);  // -z^2 / (2 ln 2)
  return poly * ex;
}
// GELU(z) = z Phi(z), Phi(z) = (1 + erf(z / sqrt 2)) / 2, without cancellation
__device__ __forceinline__ float train_gelu(float z) {
  float ex;
  const float c = 0.5f * train_erfc(z, ex);
  return z * (z >= 0.0f ? 1.0f - c : c);
}
// GELU and GELU'(z) = Phi(z) + z exp(-z^2 / 2) / sqrt(2 pi); an infinite z
// has a density of 0, not 0 times infinity
__device__ __forceinline__ void train_gelu_grad(float z, float& h, float& d) {
  float ex;
  const float c = 0.5f * train_erfc(z, ex);
  const float phi = z >= 0.0f ? 1.0f - c : c;
  h = z * phi;
  d = ex == 0.0f ? phi : fmaf(z * ex, 0.39894228040143267794f, phi);
}
// 1 / (1 + exp(-a)): exp overflows to infinity below -88, its reciprocal is 0
__device__ __forceinline__ float train_sigmoid(float a) {
  return rcp_fast(1.0f + exp2_fast(a * -1.44269504088896340736f));
}

// A warp's 32 rows x 32 columns between threads (one row each, as TMEM gives
// them) and memory (where 4 lanes together read or write a row's 64 bytes, or 32
// of 8-bit codes): 2 KB of shared memory, rows of four 16-byte pieces whose
// places are turned so that neither side meets a bank twice.  Straight from the
// threads a warp's access met 32 rows at once, 16 bytes each: the weight
// gradients of 64 experts of 2048 x 2816 took 325 us, so 240.  Outputs of one
// chunk are put down in buffers of their own and leave together: with one
// buffer and ten warp barriers a chunk, a gated Bwd tile took 22 us.
struct Turn {
  uint32_t base;  // shared-memory address of the warp's buffer
  int lane;
  __device__ __forceinline__ uint32_t own(int j) const {  // piece j of this thread's row
    return base + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4);
  }
  __device__ __forceinline__ uint32_t at(int row, int j) const {
    return base + row * 64 + ((j ^ ((row >> 1) & 3)) << 4);
  }
  __device__ __forceinline__ Turn buffer(int b) const { return Turn{base + (uint32_t)(b * T_TURN), lane}; }
};
__device__ __forceinline__ void sts16(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts8(uint32_t a, const uint2& v) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 train_pack8(const float* f) {
  uint4 pk;
  pk.x = pack_bf16x2(f[0], f[1]);
  pk.y = pack_bf16x2(f[2], f[3]);
  pk.z = pack_bf16x2(f[4], f[5]);
  pk.w = pack_bf16x2(f[6], f[7]);
  return pk;
}
__device__ __forceinline__ void train_unpack8(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}

// Where a warp's 32 rows of an output are: this lane's piece of its first row,
// and how many of the rows exist.  Addresses are made once per tile: as index
// arithmetic of every access they were a third of the epilogue's instructions.
struct RowsOut {
  uint8_t* p;    // row lane / 4, piece lane % 4 of the first chunk
  size_t step;   // 8 rows
  int left;      // rows from lane / 4 on
};
template <int PIECE, typename T>
__device__ __forceinline__ RowsOut rows_out(T* base, size_t row0, size_t cols, size_t col, int lane, int n_rows) {
  RowsOut o;
  o.p = reinterpret_cast<uint8_t*>(base + (row0 + (lane >> 2)) * cols + col) + (lane & 3) * PIECE;
  o.step = 8 * cols * sizeof(T);
  o.left = n_rows - (lane >> 2);
  return o;
}

// A buffer to memory, after a warp barrier, `off` bytes from its first chunk: the
// pieces that exist (`ok`) of the rows that do; rows from n_full on as zeros.
__device__ __forceinline__ void turn_out(const Turn& t, const RowsOut& o, size_t off, bool ok, int n_full) {
  uint8_t* p = o.p + off;
  const int full_left = n_full - (t.lane >> 2);
  if (__all_sync(0xffffffffu, min(o.left, full_left) > 24)) {  // 32 rows
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = lds16(t.at(i * 8 + (t.lane >> 2), t.lane & 3));
      if (ok) *reinterpret_cast<uint4*>(p) = v;
      p += o.step;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 v = lds16(t.at(i * 8 + (t.lane >> 2), t.lane & 3));
      if (i * 8 >= full_left) v = make_uint4(0u, 0u, 0u, 0u);
      if (ok && i * 8 < o.left) *reinterpret_cast<uint4*>(p) = v;
      p += o.step;
    }
  }
}
// Codes: 8-byte pieces, as rows start on 8 bytes only.
__device__ __forceinline__ void turn_out_codes(const Turn& t, const RowsOut& o, size_t off, bool ok) {
  uint8_t* p = o.p + off;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint2 v = lds8(t.at(i * 8 + (t.lane >> 2), t.lane & 3));
    if (ok && i * 8 < o.left) *reinterpret_cast<uint2*>(p) = v;
    p += o.step;
  }
}
// A buffer to memory by a TMA store (its pieces lie as the 64-byte swizzle lays
// them; what is outside the tensor is left out): the ring's next buffer is free
// once at most BUFS - 1 earlier stores still read theirs, as every buffer that is
// filled is stored.
__device__ __forceinline__ void turn_tma(const Turn& t, const CUtensorMap* m, int c0, int c1, int c2) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (t.lane == 0) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(t.base), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}
template <int N>
__device__ __forceinline__ void turn_tma_wait(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
  __syncwarp();
}

// 32 fp32 values of every thread's row, 16 at a time.
__device__ __forceinline__ void turn_store_f32(const Turn& t, const uint32_t (&v)[32], const RowsOut& o,
                                               size_t off, int valid) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int g = 0; g < 4; ++g)
      sts16(t.own(g), make_uint4(v[16 * h + 4 * g], v[16 * h + 4 * g + 1], v[16 * h + 4 * g + 2],
                                 v[16 * h + 4 * g + 3]));
    __syncwarp();
    turn_out(t, o, off + 64 * h, 16 * h + (t.lane & 3) * 4 < valid, 32);
    __syncwarp();
  }
}

// This thread's 32 columns of z (those below `valid` exist) into buffer t as
// bf16, or as codes with the group's scale byte as the result.
__device__ __forceinline__ uint32_t train_keep(const TrainGemmArgs& p, const Turn& t, int valid,
                                               const uint32_t (&v)[32]) {
  if (p.keep_bits == 16) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[8 * g + i]);
      sts16(t.own(g), train_pack8(f));
    }
    return 0u;
  }
  uint32_t m = 0;
  if (valid == 32) {
#pragma unroll
    for (int i = 0; i < 32; ++i) m = max(m, v[i] & 0x7fffffffu);
  } else {  // gate columns past the last one are up columns
#pragma unroll
    for (int i = 0; i < 32; ++i) m = max(m, i < valid ? v[i] & 0x7fffffffu : 0u);
  }
  const uint32_t b = a8_scale_byte(m);
  const float inv = a8_inverse(b);
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[g * 8 + i]);
    sts8(t.own(g), a8_codes8(f, inv, b));
  }
  return b;
}
// Kept z of a warp's rows: in memory as rows of `halves` N columns, and a scale
// byte per half and 32 columns.
struct KeptOut {
  RowsOut z;
  uint8_t* scales;  // of this lane's row, first chunk, or null
};
__device__ __forceinline__ KeptOut kept_out(const TrainGemmArgs& p, int halves, size_t row0, int hf, int col,
                                            int lane, int n_rows) {
  KeptOut k;
  const size_t pitch = (size_t)halves * p.N, at = (size_t)hf * p.N + col;
  k.scales = nullptr;
  if (p.keep_bits == 16) {
    k.z = rows_out<16>(static_cast<uint16_t*>(p.z), row0, pitch, at, lane, n_rows);
  } else {
    k.z = rows_out<8>(static_cast<int8_t*>(p.z), row0, pitch, at, lane, n_rows);
    if (lane < n_rows)
      k.scales = p.z_scales + ((row0 + lane) * halves + hf) * (size_t)((p.N + 31) / 32) + (col >> 5);
  }
  return k;
}
// ... from the buffer, chunk ch of the part, scale byte b.
__device__ __forceinline__ void train_kept_out(const TrainGemmArgs& p, const Turn& t, const KeptOut& k, int ch,
                                               bool ok, uint32_t b) {
  if (p.keep_bits == 16) {
    turn_out(t, k.z, (size_t)ch * 64, ok, 32);
    return;
  }
  turn_out_codes(t, k.z, (size_t)ch * 32, ok);
  if (k.scales) k.scales[ch] = (uint8_t)b;
}

// 32 kept columns of a warp's rows on their way from memory: four pieces of
// other threads' rows, 16 bytes of bf16 or 8 of codes with the group's scale.
// Rows past the last one are read as the last one (nothing of them is stored, or
// zeros are), columns past the last one are zeros.
struct KeptIn {
  const uint8_t* z;       // this lane's piece of the segment's row row0, first chunk
  const uint8_t* scales;
  uint32_t row[4];        // rows of this lane's four pieces, from row0
};
struct KeptChunk {
  uint4 w[4];
};
__device__ __forceinline__ KeptIn kept_in(const TrainGemmArgs& p, int halves, size_t row0, int hf, int col,
                                          int lane, int n_rows) {
  KeptIn k;
  const size_t at = row0 * halves * p.N + (size_t)hf * p.N + col + (lane & 3) * 8;
  k.z = static_cast<const uint8_t*>(p.z) + at * (p.keep_bits / 8);
  k.scales = p.z_scales + (row0 * halves + hf) * (size_t)((p.N + 31) / 32) + (col >> 5);
#pragma unroll
  for (int i = 0; i < 4; ++i) k.row[i] = (uint32_t)min(i * 8 + (lane >> 2), n_rows - 1);
  return k;
}
__device__ __forceinline__ void train_load_kept(const TrainGemmArgs& p, const KeptIn& k, int halves, int ch,
                                                bool ok, KeptChunk& c) {
  if (p.keep_bits == 16) {
    const uint32_t pitch = (uint32_t)(halves * 2) * (uint32_t)p.N;
    const uint8_t* z = k.z + (size_t)ch * 64;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c.w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (ok) c.w[i] = __ldg(reinterpret_cast<const uint4*>(z + (uint64_t)k.row[i] * pitch));
    }
  } else {
    const uint32_t pitch = (uint32_t)halves * (uint32_t)p.N;
    const uint32_t groups = (uint32_t)halves * (uint32_t)((p.N + 31) / 32);
    const uint8_t* z = k.z + (size_t)ch * 32;
    const uint8_t* s = k.scales + ch;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint2 u = make_uint2(0u, 0u);
      if (ok) u = __ldg(reinterpret_cast<const uint2*>(z + (uint64_t)k.row[i] * pitch));
      c.w[i].x = u.x;
      c.w[i].y = u.y;
      c.w[i].z = __ldg(s + (uint64_t)k.row[i] * groups);
    }
  }
}
// 8 codes as bf16 times a power of two, exactly: a code c is (128 + its low seven
// bits) - (128, or 256 if it is negative), both bf16 with a code's bits in the
// mantissa.
__device__ __forceinline__ uint4 a8_bf16x8(uint2 q, uint32_t b) {
  const uint32_t sb = b == 255u ? 0x7fc0u : b == 0u ? 0x0040u : b << 7;
  const uint32_t s2 = sb | sb << 16;
  const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&s2);
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = __byte_perm(i < 2 ? q.x : q.y, 0x43434343u, i & 1 ? 0x4342 : 0x4140);
    const uint32_t lo = w & 0xff7fff7fu, hi = w & 0xff80ff80u;
    const __nv_bfloat162 v = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&lo),
                                             *reinterpret_cast<const __nv_bfloat162*>(&hi)), s);
    r[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// ... and into buffer t as bf16.
__device__ __forceinline__ void train_kept_in(const TrainGemmArgs& p, const Turn& t, const KeptChunk& k) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 v = k.w[i];
    if (p.keep_bits == 8) v = a8_bf16x8(make_uint2(v.x, v.y), v.z);
    sts16(t.at(i * 8 + (t.lane >> 2), t.lane & 3), v);
  }
}

// 32 lanes x 32 bits, 8 consecutive columns per thread.
__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

template <int OP>
__global__ void __launch_bounds__(T_THREADS, 1)
    train_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                      const __grid_constant__ CUtensorMap tm_a64, const TrainGemmArgs p) {
  using TT = TrainTraits<OP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  constexpr int STAGES = TT::STAGES;
  uint8_t* sB = smem + STAGES * T_OP_BYTES;
  uint8_t* sTurn = smem + STAGES * T_STAGE_BYTES;  // 1024-byte aligned, buffers of 2 KB
  TrainCtrl& c = *reinterpret_cast<TrainCtrl*>(sTurn + T_EPI_WARPS * TT::BUFS * T_TURN);
  constexpr uint32_t IDESC = idesc_bf16_f32(TPAIR_M, TBN, TT::A_MN, TT::B_MN);
  constexpr uint32_t IDESC_HALF = idesc_bf16_f32(TPAIR_M / 2, TBN, TT::A_MN, TT::B_MN);
  constexpr uint32_t IDESC_NHALF = idesc_bf16_f32(TPAIR_M, TBN / 2, TT::A_MN, TT::B_MN);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();  // 0 = leader of the pair
  const int pair = blockIdx.x >> 1;
  const int n_pairs = gridDim.x >> 1;
  const int NB = (p.N + TT::BN_OUT - 1) / TT::BN_OUT;
  pdl_launch_dependents();
  // barriers before the earlier kernels have ended; TMEM after them, or a CTA of an
  // earlier kernel on this SM that has yet to allocate its own would wait for
  // this one, and this one for it
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&c.full[i], 2);
      mbar_init(&c.empty[i], 1);
    }
    for (int i = 0; i < TACC; ++i) {
      mbar_init(&c.tfull[i], 1);
      mbar_init(&c.tempty[i], 2 * T_EPI_WARPS);
    }
    mbar_init(&c.drain, 1);
    c.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  pdl_wait();  // offsets, operands and output buffers belong to earlier kernels
  if (warp == T_MMA_WARP) {
    tmem_alloc_pair(&c.tmem_base, T_TMEM_COLS);
    tmem_relinquish_pair();
  }
  if (warp == 0) {
    seg_scan(p.seg, c.seg, c.tile_start, lane, pair == 0 && rank == 0 ? p.status : nullptr, [&](int n) {
      const int m = TT::WGRAD ? p.M : n;
      return (m + TPAIR_M - 1) / TPAIR_M * NB * (TT::SPLIT ? p.splits : 1);
    });
  }
  if (p.merge_status && blockIdx.x == 0 && threadIdx.x == 32) {
    const int s = *p.merge_status;
    if (s) record_status(p.status, s);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the leader's barriers exist before the peer signals them
  tc_fence_after();
  const int n_tiles = c.tile_start[p.seg.E];
  const uint32_t tmem = c.tmem_base;
  const WaitCtl wc{&c.abort_flag, p.status, p.wait_limit_ns};

  if (warp == 0) {
    // ------------------------------------------------ producer (one thread)
    if (lane == 0) {
      const uint32_t full0 = dsmem_map(smem_u32(&c.full[0]), 0);  // leader's barriers
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      int e = 0;
      bool ok = true;
      for (int tile = pair; tile < n_tiles && ok; tile += n_pairs) {
        const TrainTile t = train_tile<OP>(c, p, tile, e);
        const int off = TT::A_PADDED ? c.seg.pad_off[t.e] : c.seg.row_off[t.e];
        // this CTA's first row of A's M and column of B's N
        const int arow = t.base + rank * (t.half ? TBM / 2 : TBM);
        const int bcol = TT::PAIRED  ? t.nb * TT::BN_OUT + (t.half ? rank * 64 : rank * p.N)
                         : t.nhalf   ? t.nb * TBN + rank * (TBN / 4)
                                     : t.nb * TBN + rank * (TBN / 2);
        const int bcol2 = TT::PAIRED && t.half ? bcol + p.N : bcol + 64;  // of the second box
        const uint32_t a_bytes = t.half ? T_OP_BYTES / 2 : T_OP_BYTES;
        const int b_boxes = t.nhalf ? 1 : 2;  // MN-major: 64-column boxes
        const uint32_t bytes = a_bytes + (TT::B_MN ? b_boxes * T_BOX : T_OP_BYTES);
        for (int kb = 0; kb < t.kb; ++kb) {
          if (!mbar_wait(&c.empty[stage], phase ^ 1u, wc)) {
            ok = false;
            break;
          }
          const uint32_t full_cl = full0 + (uint32_t)(stage * sizeof(uint64_t));
          uint8_t* a = sA + stage * T_OP_BYTES;
          uint8_t* b = sB + stage * T_OP_BYTES;
          mbar_arrive_expect_tx_cluster(full_cl, bytes);
          if constexpr (TT::WGRAD) {
            const int krow = off + kb * TBK;
            tma_load_2d_pair(a, &tm_a, full_cl, arow, krow);
            if (!t.half) tma_load_2d_pair(a + T_BOX, &tm_a, full_cl, arow + 64, krow);
            tma_load_2d_pair(b, &tm_b, full_cl, bcol, krow);
            if (!t.nhalf) tma_load_2d_pair(b + T_BOX, &tm_b, full_cl, bcol2, krow);
          } else {
            // rows past the segment's end are computed but never stored
            const int k0 = (t.k0 + kb) * TBK;
            tma_load_2d_pair(a, t.half ? &tm_a64 : &tm_a, full_cl, k0, off + arow);
            if constexpr (TT::B_MN) {
              tma_load_3d_pair(b, &tm_b, full_cl, bcol, k0, t.e);
              if (!t.nhalf) tma_load_3d_pair(b + T_BOX, &tm_b, full_cl, bcol2, k0, t.e);
            } else {
              tma_load_3d_pair(b, &tm_b, full_cl, k0, bcol, t.e);
            }
          }
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // the bytes of the last armed stages of both CTAs have landed before
      // shared memory is released (at once on the normal path)
      if (rank == 0) {
        for (int m = max(0, issued - STAGES); m < issued; ++m)
          train_wait_drain(&c.full[m % STAGES], (uint32_t)((m / STAGES) & 1), p.wait_limit_ns, p.status);
      }
    }
    __syncwarp();
  } else if (warp == T_MMA_WARP) {
    // ------------------------------------------------ MMA issuer (leader)
    if (rank == 0 && lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      int e = 0;
      for (int tile = pair; tile < n_tiles && ok; tile += n_pairs) {
        const TrainTile t = train_tile<OP>(c, p, tile, e);
        if (t.kb == 0) continue;  // an expert without rows: the epilogue writes zeros
        const uint32_t idesc = t.half ? IDESC_HALF : t.nhalf ? IDESC_NHALF : IDESC;
        if (!mbar_wait(&c.tempty[acc], acc_phase ^ 1u, wc)) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(acc * TBN);
        for (int kb = 0; kb < t.kb; ++kb) {
          if (!mbar_wait(&c.full[stage], phase, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + stage * T_OP_BYTES);
          const uint32_t b0 = smem_u32(sB + stage * T_OP_BYTES);
          const int steps = TT::WGRAD ? min(4, t.k16 - 4 * kb) : 4;
#pragma unroll
          for (int j = 0; j < TBK / 16; ++j) {
            if (TT::WGRAD && j >= steps) break;
            // K-major: 16 elements = 32 bytes inside the swizzle row;
            // MN-major: 16 K rows = two 1024-byte atoms
            const uint64_t ad = TT::A_MN ? sdesc_sw128(a0 + j * 2048, T_BOX, 1024)
                                         : sdesc_sw128(a0 + j * 32, 16, 1024);
            const uint64_t bd = TT::B_MN ? sdesc_sw128(b0 + j * 2048, T_BOX, 1024)
                                         : sdesc_sw128(b0 + j * 32, 16, 1024);
            umma_bf16_pair(d, ad, bd, idesc, (kb | j) != 0 ? 1u : 0u);
          }
          umma_commit_pair_mc(&c.empty[stage], T_PAIR_MASK);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair_mc(&c.tfull[acc], T_PAIR_MASK);
        if (++acc == TACC) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      umma_commit_pair_mc(&c.drain, 0x1);  // all MMAs of this thread have completed
      train_wait_drain(&c.drain, 0, p.wait_limit_ns, p.status);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue warps
    const int q = warp & 3;                     // TMEM lane quadrant this warp may read
    const int wh = (warp - T_EPI_WARP0) >> 2;   // which half of the tile's chunks
    const Turn turn{smem_u32(sTurn + (warp - T_EPI_WARP0) * TT::BUFS * T_TURN), lane};
    const uint32_t tempty0 = dsmem_map(smem_u32(&c.tempty[0]), 0);
    constexpr int HALVES = TT::HALVES;
    int acc = 0;
    uint32_t acc_phase = 0;
    int e = 0;
    // what this warp does of a tile
    struct Part {
      TrainTile t;
      int row0;      // its first row, within the segment (Wgrad: of out)
      int n_seg;     // rows of the segment (Wgrad: of out)
      int n_rows;    // its rows
      int col_base, ch0, ch1;  // first column of the tile's half, its chunks of 32
    };
    const auto part_of = [&](int tile) {
      Part a;
      a.t = train_tile<OP>(c, p, tile, e);
      a.row0 = a.t.base + (a.t.half ? rank * (TBM / 2) + (q & 1) * 32 : rank * TBM + q * 32);
      a.col_base = a.t.nb * TT::BN_OUT + (a.t.half ? (q >> 1) * (TT::BN_OUT / 2) : 0);
      const int n_chunks = (a.t.half || a.t.nhalf ? 4 : 8) / (TT::PAIRED ? 2 : 1);  // both warps'
      a.ch0 = wh * (n_chunks / 2);
      a.ch1 = a.ch0 + n_chunks / 2;
      a.n_seg = TT::WGRAD ? p.M : c.seg.rows[a.t.e];
      a.n_rows = min(max(a.n_seg - a.row0, 0), 32);
      return a;
    };
    [[maybe_unused]] KeptChunk next[HALVES];
    [[maybe_unused]] KeptIn kin[HALVES];
    // this warp's kept rows, and the first chunk of them on its way
    [[maybe_unused]] const auto load_first = [&](const Part& a) {
      if (a.n_rows == 0 || a.col_base + a.ch0 * 32 >= p.N) return;
#pragma unroll
      for (int hf = 0; hf < HALVES; ++hf) {
        kin[hf] = kept_in(p, HALVES, (size_t)c.seg.row_off[a.t.e] + a.row0, hf, a.col_base + a.ch0 * 32, lane,
                          a.n_rows);
        train_load_kept(p, kin[hf], HALVES, 0, a.col_base + a.ch0 * 32 + (lane & 3) * 8 < p.N, next[hf]);
      }
    };
    [[maybe_unused]] int ring = 0;
    Part w = {};
    if (pair < n_tiles) {
      w = part_of(pair);
      if constexpr (TT::BWD) load_first(w);
    }
    for (int tile = pair; tile < n_tiles; tile += n_pairs) {
      const TrainTile t = w.t;
      const int n_rows = w.n_rows;
      [[maybe_unused]] float gw = 0.0f;
      if constexpr (TT::BWD) {
        if (lane < n_rows) {
          gw = 1.0f;
          if (p.w) {
            const int a = __ldg(p.perm + c.seg.row_off[t.e] + w.row0 + lane);
            gw = a >= 0 && a < p.n_w ? __ldg(p.w + a) : 0.0f;
          }
        }
      }
      if (t.kb > 0) {
        int got = 1;
        if (lane == 0) got = mbar_wait(&c.tfull[acc], acc_phase, wc);
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) break;
        tc_fence_after();
      }
      const uint32_t tbase = tmem + (uint32_t)(acc * TBN) + ((uint32_t)(q * 32) << 16);
      const int gcol0 = w.col_base + w.ch0 * 32;
      // chunks of 32 columns that exist, and whether this lane's piece of one does
      const int n_ch = n_rows == 0 ? 0 : min(w.ch1 - w.ch0, (p.N - gcol0 + 31) / 32);

      if constexpr (TT::BWD) {
        const size_t crow0 = (size_t)c.seg.row_off[t.e] + w.row0;
        // padded rows: zeros behind the segment's last one, up to 16 (they share
        // this warp with at least one row of the segment)
        const int n_pad = min(max((w.n_seg + 15) / 16 * 16 - w.row0, 0), 32);
        const size_t prow0 = (size_t)c.seg.pad_off[t.e] + w.row0;
        const Turn b_hw = turn.buffer(HALVES);
        const RowsOut o_dz = rows_out<16>(p.dz, prow0, (size_t)p.ld_dz, gcol0, lane, n_pad);
        const RowsOut o_hw = rows_out<16>(p.hw, prow0, (size_t)p.ld_hw, gcol0, lane, n_pad);
        float* part = p.part && lane < n_rows ? p.part + (crow0 + lane) * (size_t)p.units + (gcol0 >> 6) : nullptr;
        float dot = 0.0f;
#pragma unroll 1
        for (int ch = 0; ch < n_ch; ++ch) {
          const bool piece = gcol0 + ch * 32 + (lane & 3) * 8 < p.N;
#pragma unroll
          for (int hf = 0; hf < HALVES; ++hf) train_kept_in(p, turn.buffer(hf), next[hf]);
          if (ch + 1 < n_ch) {
#pragma unroll
            for (int hf = 0; hf < HALVES; ++hf)
              train_load_kept(p, kin[hf], HALVES, ch + 1, gcol0 + (ch + 1) * 32 + (lane & 3) * 8 < p.N, next[hf]);
          }
          __syncwarp();
          uint32_t v[8], vn[8];
          const uint32_t tcol = tbase + (uint32_t)((w.ch0 + ch) * 32);
          tmem_ld_x8(tcol, v);
          tmem_ld_wait();
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            if (g < 3) tmem_ld_x8(tcol + (uint32_t)(8 * g + 8), vn);
            float z[8], hv[8];
            [[maybe_unused]] float u[8];
            train_unpack8(lds16(turn.own(g)), z);
            if constexpr (TT::GATED) train_unpack8(lds16(turn.buffer(1).own(g)), u);
            // z becomes dz (of the gate), u becomes dz of the up projection
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              // columns past the last one: g and z are 0
              const float gr = __uint_as_float(v[i]);
              const float wg = gw * gr;
              float h;
              if constexpr (TT::GATED) {
                // h = a s(a) u; dh/da = u s (1 + a (1 - s)), dh/du = a s
                const float s = train_sigmoid(z[i]);
                const float as = z[i] * s;
                h = as * u[i];
                z[i] = wg * u[i] * s * fmaf(z[i], 1.0f - s, 1.0f);
                u[i] = wg * as;
              } else {
                float d;
                train_gelu_grad(z[i], h, d);
                z[i] = wg * d;
              }
              dot = fmaf(gr, h, dot);
              hv[i] = gw * h;
            }
            sts16(turn.own(g), train_pack8(z));
            if constexpr (TT::GATED) sts16(turn.buffer(1).own(g), train_pack8(u));
            sts16(b_hw.own(g), train_pack8(hv));
            if (g < 3) {
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = vn[i];
            }
          }
          __syncwarp();
          turn_out(turn, o_dz, (size_t)ch * 64, piece, n_rows);
          if constexpr (TT::GATED) turn_out(turn.buffer(1), o_dz, (size_t)ch * 64 + (size_t)p.N * 2, piece, n_rows);
          turn_out(b_hw, o_hw, (size_t)ch * 64, piece, n_rows);
          if ((ch & 1) || ch + 1 == n_ch) {  // 64 columns, or the last
            if (part) part[ch >> 1] = dot;
            dot = 0.0f;
          }
          __syncwarp();
        }
      } else {
        // Fwd, Rows, Plain, Wgrad
        const bool idle = OP == kTrainWgrad && t.kb == 0;
        if (idle) {
          // an expert without rows: its matrix is one block of memory, of which
          // this tile clears a part in whole lines (36 experts of 2872 x 9480 by
          // tiles, whose rows start inside a sector: 817 us, so 320-342)
          const int64_t all = (int64_t)p.M * p.N / 8;
          const int cnt = c.tile_start[t.e + 1] - c.tile_start[t.e], at = tile - c.tile_start[t.e];
          const int64_t lo = all * at / cnt, hi = all * (at + 1) / cnt;
          uint4* dst = reinterpret_cast<uint4*>(p.out) + (int64_t)t.e * all;
          const int shift = (int)((reinterpret_cast<uintptr_t>(dst) >> 4) & 7);
          for (int64_t i = ((lo + shift) & ~(int64_t)7) - shift + (rank * T_EPI_WARPS + warp - T_EPI_WARP0) * 32 + lane;
               i < hi; i += 2 * T_EPI_WARPS * 32)
            if (i >= lo) dst[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        size_t orow0 = (size_t)c.seg.row_off[t.e] + w.row0;
        if constexpr (TT::SPLIT) orow0 += (size_t)t.ks * p.seg.rows;
        [[maybe_unused]] KeptOut kout[HALVES];
        [[maybe_unused]] RowsOut o;
        if constexpr (!TT::WGRAD) {
          if constexpr (TT::OUT32)
            o = rows_out<16>(p.out32, orow0, (size_t)p.N, gcol0, lane, n_rows);
          else
            o = rows_out<16>(p.out, orow0, (size_t)p.ld_out, gcol0, lane, n_rows);
        }
        if constexpr (TT::FWD) {
#pragma unroll
          for (int hf = 0; hf < HALVES; ++hf) kout[hf] = kept_out(p, HALVES, orow0, hf, gcol0, lane, n_rows);
        }
#pragma unroll 1
        for (int ch = 0; ch < (idle ? 0 : n_ch); ++ch) {
          const int gcol = gcol0 + ch * 32;
          uint32_t v[32];
          [[maybe_unused]] uint32_t uv[32];
          const uint32_t tcol = tbase + (uint32_t)((w.ch0 + ch) * 32);
          tmem_ld_x32(tcol, v);
          // gate columns are the accumulator's first 128 (64 with M = 128), up
          // columns the others
          if constexpr (TT::PAIRED) tmem_ld_x32(tcol + (uint32_t)(t.half ? 64 : 128), uv);
          tmem_ld_wait();
          const int valid = min(32, p.N - gcol);
          if constexpr (TT::WGRAD) {
            // 64 bytes of every row at a time: 32 columns of bf16, 16 of fp32
            constexpr int OUTS = TT::OUT32 ? 2 : 1;
#pragma unroll
            for (int o = 0; o < OUTS; ++o) {
              // one store per buffer of the ring, or the wait would count too few
              if (gcol + 16 * o >= p.N) break;
              turn_tma_wait<TT::BUFS - 1>(lane);
              const Turn out = turn.buffer(ring);
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                if constexpr (TT::OUT32) {
                  const int i = 16 * o + 4 * g;
                  sts16(out.own(g), make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]));
                } else {
                  float f[8];
#pragma unroll
                  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[8 * g + i]);
                  sts16(out.own(g), train_pack8(f));
                }
              }
              turn_tma(out, &tm_a64, gcol + 16 * o, w.row0, t.e);
              ring = ring == TT::BUFS - 1 ? 0 : ring + 1;
            }
          } else if constexpr (TT::OUT32) {
            turn_store_f32(turn, v, o, (size_t)ch * 128, valid);
          } else {
            [[maybe_unused]] uint32_t b0 = 0u, b1 = 0u;
            if constexpr (TT::FWD) b0 = train_keep(p, turn, valid, v);
            if constexpr (TT::PAIRED) b1 = train_keep(p, turn.buffer(1), valid, uv);
            const Turn out = turn.buffer(TT::BUFS - 1);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              float f[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                f[i] = __uint_as_float(v[8 * g + i]);
                if constexpr (OP == kTrainFwdGelu) f[i] = train_gelu(f[i]);
                if constexpr (OP == kTrainFwdSwiGLU)
                  f[i] = f[i] * train_sigmoid(f[i]) * __uint_as_float(uv[8 * g + i]);
              }
              sts16(out.own(g), train_pack8(f));
            }
            __syncwarp();
            const bool piece = (lane & 3) * 8 < valid;
            if constexpr (TT::FWD) train_kept_out(p, turn, kout[0], ch, piece, b0);
            if constexpr (TT::PAIRED) train_kept_out(p, turn.buffer(1), kout[HALVES - 1], ch, piece, b1);
            turn_out(out, o, (size_t)ch * 64, piece, 32);
            __syncwarp();
          }
        }
      }
      // the next tile's part, and its first kept columns while this one's
      // accumulator is handed back
      if (tile + n_pairs < n_tiles) {
        w = part_of(tile + n_pairs);
        if constexpr (TT::BWD) load_first(w);
      }
      if (t.kb > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty0 + (uint32_t)(acc * sizeof(uint64_t)));
        if (++acc == TACC) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
    }
  }

  // A warp's stores have read its buffers (and are complete) before they go.
  if constexpr (TT::WGRAD) {
    if (warp >= T_EPI_WARP0 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  // Both CTAs finish all remote signalling and the leader's MMAs before TMEM
  // is released and before either CTA's shared memory goes away.
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == T_MMA_WARP) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, T_TMEM_COLS);
  }
  cluster_sync_all();
}

template <int OP>
cudaError_t train_set_attributes() {
  return cudaFuncSetAttribute(train_gemm_kernel<OP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)TrainTraits<OP>::SMEM);
}

// Persistent pairs: as many as are resident at once, at most one per tile.
template <int OP>
cudaError_t train_launch(const CUtensorMap& tm_a, const CUtensorMap& tm_b, const CUtensorMap& tm_a64,
                         const TrainGemmArgs& a, int64_t max_tiles, cudaStream_t st) {
  static std::atomic<int> pairs_of[64];
  if (max_tiles <= 0) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(T_THREADS, 1, 1);
  cfg.dynamicSmemBytes = TrainTraits<OP>::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int pairs = dev >= 0 && dev < 64 ? pairs_of[dev].load() : 0;
  if (pairs == 0) {
    e = cudaOccupancyMaxActiveClusters(&pairs, train_gemm_kernel<OP>, &cfg);
    if (e != cudaSuccess) return e;
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    if (dev >= 0 && dev < 64) pairs_of[dev] = pairs;
  }
  if (pairs > max_tiles) pairs = (int)max_tiles;
  cfg.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
  set_pdl_attr(attr[1]);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, train_gemm_kernel<OP>, tm_a, tm_b, tm_a64, a);
}

}  // namespace
}  // namespace moe
