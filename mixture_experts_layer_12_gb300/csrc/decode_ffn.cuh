// decode_ffn.cuh -- second kernel of the decode operators: the expert products
// of a few rows, in one cooperative launch that streams every needed weight
// once.
//
// Per entry (an expert and at most 64 rows of it, in dispatch order):
//   layer:            h = act(x W1[e]);  y[t] = sum_j gate[t, j] (h W2[e])[slot(t, j)]
//   grouped products: y = x W[e]
// ("用Ascend C写一个MoE融合算子", listings "Expert计算" and "Scatter + 加权".)
//
// With a handful of rows the work is the stream of the weights: 2 or ~0.53
// bytes per weight against 2 n FLOPs for n rows.  So the kernel is built
// around that stream.
//   * Work split: the weights of a product are cut into items (entry x 128
//     columns) of K chunks of 16 KB (64 rows of bf16, 256 rows of 4-bit
//     codes); the chunks, in item order, are dealt to the CTAs in equal
//     contiguous ranges, one CTA per SM.  Every SM reads the same number of
//     bytes whatever the shape, and at most its first and last item are
//     shared with other CTAs.  A CTA's sum of a shared item goes to a partial
//     tile in the workspace; the CTA that finishes the item last (a ticket
//     counter, nobody waits) adds the tiles in CTA order, so the sum has one
//     order whoever comes last.
//   * One warp issues TMA loads into a ring of weight stages, and runs ahead
//     of everything: while the CTAs meet at the grid barrier between the two
//     products, the ring already fills with W2.
//   * Three loader warps bring the rows' K chunk (x, then h) to shared memory
//     as the tensor core's N operand.
//   * Eight warps multiply: m16n8k16 products with the weights as M (16
//     columns of W) and the rows as N (8 at a time), 4 warps across the
//     columns x 2 across K.  A weight is loaded from shared memory once and
//     used for every row.  bf16 weights come out of the 128-byte-swizzled
//     stage by ldmatrix.trans.  4-bit codes are turned into bf16 in
//     registers: (128 + c) is the bf16 0x4300 | c, minus 136 is exact; the
//     products are exact in fp32, each scale group is summed in fp32 and
//     multiplied by its scale in fp32.
//   tcgen05 is not used: it would want the 4-bit weights expanded to bf16 in
//   shared memory (94 bytes per clock written and read where the SM's shared
//   memory moves 128), and for bf16 the stream, not the multiply, is the
//   bound: one m16n8k16 per 256 weights is a tenth of the tensor rate at 8
//   rows.
//   * Combine: a CTA that has finished its part of a column block counts
//     itself in; the last one sums every token's experts in slot order.
// The grid barrier needs all CTAs resident, which the cooperative launch
// guarantees; it and every other wait is bounded.
#pragma once

#include "decode_internal.h"
#include "tc_common.cuh"

namespace moe {
namespace {

constexpr int DF_WN = 4;         // consumer warps across the columns
constexpr int DF_FIN = 32 * DF_WN;  // threads that write an item out
constexpr int DF_W_BYTES = 16384;
constexpr int DF_MAX_WSTAGES = 12;
constexpr int DF_MAX_BSTAGES = 6;
constexpr int DF_SMEM_LIMIT = 227 * 1024;

// named barriers: consumers, writers of an item
constexpr int BAR_CONS = 1;
constexpr int BAR_FIN = 2;

__device__ __forceinline__ void named_sync(int id, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
// barrier that also tells every thread whether any of them says `bad`
__device__ __forceinline__ bool named_any(int id, int n, bool bad) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((uint32_t)bad)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_load_3d_hint(void* dst, const CUtensorMap* m, uint64_t* bar,
                                                 int c0, int c1, int c2, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "l"(pol)
      : "memory");
}
__device__ __forceinline__ unsigned ld_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void red_release(unsigned* p, unsigned v) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void lds128(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void lds64(uint32_t a, uint32_t& r0, uint32_t& r1) {
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t x) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the same with a sum that begins at zero
__device__ __forceinline__ void mma_bf16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// codes i and i + 4 of a word (rows i and i + 4 of its 8) as a bf16 pair
// (c - 8) / 64, exactly (the scale is multiplied by 64).  A code at bits 0-3
// or 4-7 of a half word is, read as bf16, c or 16 c times 2^-133 (the numbers
// below 2^-125 are evenly spaced), so one masked word and one fused
// multiply-add make a pair, and a word needs one shift: 9 instructions for 8
// codes where (128 + c) - 136 takes 11, of which the shifts and masks run at
// half rate (matrix-vector product 18.8 -> 17.9 us).
template <int I>
__device__ __forceinline__ uint32_t q4_pair(uint32_t v) {
  const uint32_t p = (I & 2 ? v >> 8 : v) & (I & 1 ? 0x00F000F0u : 0x000F000Fu);
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;"
      : "=r"(d)
      : "r"(p), "r"(I & 1 ? 0x7D007D00u : 0x7F007F00u), "r"(0xBE00BE00u));  // 2^123, 2^127; -8 / 64
  return d;
}

// GELU(z) = 0.5 z (1 + erf(z / sqrt 2)) with erfc by Abramowitz & Stegun,
// formula 7.1.26 (|error| <= 1.5e-7), arranged so 1 + erf is never formed by
// cancellation (as in ffn_gemm.cu).
__device__ __forceinline__ float dec_gelu(float z) {
  const float ax = fabsf(z) * 0.70710678118654752440f;
  const float t = __fdividef(1.0f, fmaf(0.3275911f, ax, 1.0f));
  const float poly =
      t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f),
                       -0.284496736f),
               0.254829592f);
  const float c = poly * __expf(-ax * ax);
  return 0.5f * z * (z >= 0.0f ? 2.0f - c : c);
}
__device__ __forceinline__ float dec_silu(float z) { return __fdividef(z, 1.0f + __expf(-z)); }

// 8 elements of h of row r of an entry, from the partial tiles of CTAs o0..o1
// (in that order), activated and rounded to bf16.
__device__ __forceinline__ uint4 sum_h_piece(const DecFfnArgs& p, int o0, int o1, int r, int kk,
                                             bool swiglu) {
  const int cl = swiglu ? kk & 63 : kk & 127;
  const size_t tile = (size_t)p.row_cap * kDecBN;
  float z[8], u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = u[i] = 0.f;
#pragma unroll 2
  for (int o = o0; o <= o1; ++o) {
    const float4* s = reinterpret_cast<const float4*>(p.parts + (size_t)(o * 2 + (o == o0 ? 1 : 0)) * tile +
                                                      r * kDecBN + cl);
    const float4 a = __ldcg(s), b = __ldcg(s + 1);
    z[0] += a.x; z[1] += a.y; z[2] += a.z; z[3] += a.w;
    z[4] += b.x; z[5] += b.y; z[6] += b.z; z[7] += b.w;
    if (swiglu) {
      const float4 d = __ldcg(s + 16), e = __ldcg(s + 17);
      u[0] += d.x; u[1] += d.y; u[2] += d.z; u[3] += d.w;
      u[4] += e.x; u[5] += e.y; u[6] += e.z; u[7] += e.w;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = swiglu ? dec_silu(z[i]) * u[i] : dec_gelu(z[i]);
  return make_uint4(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]), pack_bf16x2(z[4], z[5]),
                    pack_bf16x2(z[6], z[7]));
}

template <int V>
struct Int {
  static constexpr int value = V;
};

template <bool Q4, int NT>
struct Cfg {
  // consumer warps: KG groups of 4 across the columns; group i takes every
  // KG-th chunk, so that a warp has a chunk's whole K to keep its pipes full
  // between two waits.  With 64 rows the sums need the registers of 2 groups.
  static constexpr int KG = Q4 && NT < 8 ? 3 : 2;
  static constexpr int LOADERS = Q4 && NT == 8 ? 2 : 3;
  static constexpr int CONSUMERS = DF_WN * KG;
  static constexpr int THREADS = 32 * (1 + LOADERS + CONSUMERS);
  static constexpr int KC = Q4 ? kDecKC4 : kDecKC16;   // K rows of a chunk
  static constexpr int S_BYTES = Q4 ? 8 * 2 * 128 : 0; // scales: up to 8 groups x 2 boxes x 128 B
  static constexpr int W_STAGE = DF_W_BYTES + S_BYTES;
  static constexpr int B_TILE = KC * 16;               // 8 rows x KC bf16
  static constexpr int B_STAGE = B_TILE * NT;
  static constexpr int B_STAGES = !Q4 || NT == 1 ? 6 : KG;
  static constexpr int RED = (KG - 1) * DF_WN * 2 * NT * 4 * 32 * 4;  // sums across the groups
  static constexpr int CTRL = 12 * 1024;
  static constexpr int FIT = (DF_SMEM_LIMIT - 1024 - CTRL - RED - B_STAGE * B_STAGES) / W_STAGE;
  static constexpr int W_STAGES = (FIT < DF_MAX_WSTAGES ? FIT : DF_MAX_WSTAGES) / KG * KG;
  static constexpr size_t SMEM =
      1024 + (size_t)W_STAGES * W_STAGE + (size_t)B_STAGES * B_STAGE + RED + CTRL;
  static_assert(W_STAGES >= 4, "weight ring");
  static_assert(SMEM <= DF_SMEM_LIMIT, "shared memory");
  // A wait tells the phases of a barrier apart by parity only, so whoever
  // waits for a stage's phase must know the one before it to be over.  A
  // group finishes its chunks in order, but the groups (and the copies in
  // flight) overtake each other: every stage therefore has one group and one
  // loader of its own.
  static_assert(W_STAGES % KG == 0 && B_STAGES % KG == 0 && B_STAGES % LOADERS == 0, "ring owners");
  static_assert(B_STAGES <= DF_MAX_BSTAGES, "row ring");
};

struct Ctrl {
  uint64_t wfull[DF_MAX_WSTAGES], wempty[DF_MAX_WSTAGES];
  uint64_t bfull[DF_MAX_BSTAGES], bempty[DF_MAX_BSTAGES];
  int abort_flag;
  int n_entries;
  int last;
  DecEntry ent[kDecMaxEntries];
  int2 owner[kDecMaxEntries];    // combine: CTAs of the column block's items
  uint16_t row_entry[MOED_MAX_ROWS];
  int slot[MOED_MAX_ROWS];       // layer: [T, k]
  float gate[MOED_MAX_ROWS];
};
static_assert(sizeof(Ctrl) <= 12 * 1024, "control area");

// One product's chunks, in item order, dealt to the first G = min(CTAs, total)
// CTAs: CTA c < G takes chunks [total c / G, total (c + 1) / G), at least one.
// The host keeps total * CTAs below 2^32.
struct Split {
  uint32_t total, G;
  __device__ __forceinline__ Split(uint32_t n, uint32_t ctas) : total(n), G(min(ctas, n)) {}
  __device__ __forceinline__ uint32_t start(uint32_t c) const {
    return c < G ? total * c / G : total;
  }
  // the CTA that holds chunk x: the largest c with total c / G < x + 1
  __device__ __forceinline__ int owner(uint32_t x) const {
    return (int)(((x + 1) * G - 1) / total);
  }
};

// A split item of the first product with at most this many rows is not put
// together by the CTA that finishes it: the second product's row loaders add
// its partial tiles when they read it.  That saves a ticket and a trip to
// memory before the grid barrier, and costs every reader the sum and the
// activation of the elements it reads, which a few rows' loaders have the time for.
constexpr int kReaderRows = 2;

// One chunk of 4-bit weights for a warp's 32 columns and the first NTA 8-row
// tiles: acc += W^T x.  wl, bl: this lane's addresses in the stages (word row
// 0 / 1 of a step by wofs); sl: its 4 columns' scales.  Everything is
// unrolled and nothing branches, so that loads, unpacking and products of
// different steps overlap.
template <int NT, int NTA, int GRP>
__device__ __forceinline__ void chunk_q4(float (&acc)[2][NT][4], uint32_t w0, const uint32_t (&wofs)[2],
                                         uint32_t bl, uint32_t sl) {
  constexpr int STEPS = GRP / 32;  // 32 rows of K each
#pragma unroll
  for (int grp = 0; grp < kDecKC4 / GRP; ++grp) {
    float part[2][NTA][4];
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
      const uint32_t blk = (uint32_t)(grp * STEPS + st) >> 1, i = (uint32_t)(grp * STEPS + st) & 1;
      uint32_t v[4];  // columns 4g .. 4g + 3 of 8 rows of K
      lds128(w0 + blk * 1024 + wofs[i], v);
      uint32_t b[NTA][4];
#pragma unroll
      for (int n = 0; n < NTA; ++n) lds128(bl + n * kDecKC4 * 16 + blk * 1024 + i * 512, b[n]);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint32_t va = v[2 * m], vb = v[2 * m + 1];
        uint32_t a[8];
        a[0] = q4_pair<0>(va);
        a[1] = q4_pair<0>(vb);
        a[2] = q4_pair<1>(va);
        a[3] = q4_pair<1>(vb);
        a[4] = q4_pair<2>(va);
        a[5] = q4_pair<2>(vb);
        a[6] = q4_pair<3>(va);
        a[7] = q4_pair<3>(vb);
#pragma unroll
        for (int n = 0; n < NTA; ++n) {
          if (st == 0)
            mma_bf16_zero(part[m][n], a[0], a[1], a[2], a[3], b[n][0], b[n][1]);
          else
            mma_bf16(part[m][n], a[0], a[1], a[2], a[3], b[n][0], b[n][1]);
          mma_bf16(part[m][n], a[4], a[5], a[6], a[7], b[n][2], b[n][3]);
        }
      }
    }
    uint32_t s01, s23;
    lds64(sl + grp * 128, s01, s23);
    const float s[4] = {64.f * bf16_lo(s01), 64.f * bf16_hi(s01), 64.f * bf16_lo(s23), 64.f * bf16_hi(s23)};
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NTA; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[m][n][r] = fmaf(s[2 * m + (r >> 1)], part[m][n][r], acc[m][n][r]);
  }
}

// The same for a chunk of bf16 weights.
template <int NT, int NTA>
__device__ __forceinline__ void chunk_bf16(float (&acc)[2][NT][4], uint32_t w0,
                                           const uint32_t (&wofs)[2], uint32_t bl) {
#pragma unroll
  for (int blk = 0; blk < kDecKC16 / 32; ++blk) {  // 32 rows of K
    uint32_t a[2][2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) ldsm_x4_t(w0 + (blk * 32 + hf * 16) * 128 + wofs[m], a[m][hf]);
#pragma unroll
    for (int n = 0; n < NTA; ++n) {
      uint32_t b[4];
      lds128(bl + n * kDecKC16 * 16 + blk * 512, b);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        mma_bf16(acc[m][n], a[m][0][0], a[m][0][1], a[m][0][2], a[m][0][3], b[0], b[1]);
        mma_bf16(acc[m][n], a[m][1][0], a[m][1][1], a[m][1][2], a[m][1][3], b[2], b[3]);
      }
    }
  }
}

// GRP: rows per scale of 4-bit weights; 0: bf16 weights.
template <int GRP, int NT>
__global__ void __launch_bounds__(Cfg<(GRP > 0), NT>::THREADS, 1)
    decode_ffn_kernel(const __grid_constant__ DecFfnMaps maps, const DecFfnArgs p) {
  constexpr bool Q4 = GRP > 0;
  using C = Cfg<Q4, NT>;
  constexpr int KG = C::KG;
  constexpr int CTHREADS = 32 * C::CONSUMERS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sW = smem;                                      // [W_STAGES][16 KB]
  uint8_t* sS = sW + C::W_STAGES * DF_W_BYTES;             // [W_STAGES][S_BYTES]
  uint8_t* sB = sS + C::W_STAGES * C::S_BYTES;             // [B_STAGES][B_STAGE]
  float* sRed = reinterpret_cast<float*>(sB + C::B_STAGES * C::B_STAGE);
  Ctrl& c = *reinterpret_cast<Ctrl*>(reinterpret_cast<uint8_t*>(sRed) + C::RED);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int cta = blockIdx.x;
  const uint32_t G = gridDim.x;
  const bool layer = p.act != kDecNone;
  const bool swiglu = p.act == kDecSwiGLU;

  if (tid == 64) {
    tma_prefetch_desc(&maps.w1);
    if (Q4) tma_prefetch_desc(&maps.s1);
    if (layer) {
      tma_prefetch_desc(&maps.w2);
      if (Q4) tma_prefetch_desc(&maps.s2);
    }
  }
  if (tid == 0) {
    for (int i = 0; i < C::W_STAGES; ++i) {
      mbar_init(&c.wfull[i], 1);
      mbar_init(&c.wempty[i], DF_WN);
    }
    for (int i = 0; i < C::B_STAGES; ++i) {
      mbar_init(&c.bfull[i], 1);
      mbar_init(&c.bempty[i], DF_WN);
    }
    c.abort_flag = 0;
    fence_mbar_init();
  }
  pdl_launch_dependents();
  pdl_wait();
  // the first kernel's list
  if (tid == 32) c.n_entries = min(__ldcg(p.ctrl + kDecCountOffset / 4), p.max_entries);
  for (int i = tid; i < p.max_entries; i += C::THREADS) {
    const int4 v = __ldcg(reinterpret_cast<const int4*>(p.entries) + i);
    c.ent[i] = DecEntry{v.x, v.y, v.z, v.w};
  }
  if (layer)
    for (int i = tid; i < p.T * p.k; i += C::THREADS) {
      c.slot[i] = __ldcg(p.slot + i);
      c.gate[i] = __ldcg(p.gate + i);
    }
  __syncthreads();
  const int n_ent = c.n_entries;
  const WaitCtl wc{&c.abort_flag, p.status, p.wait_limit_ns};

  if (n_ent == 0) {  // every assignment dropped: y = 0 (grouped products: nothing to write)
    if (layer) {
      const size_t n = (size_t)p.T * p.N2;  // N2 = H, a multiple of 8
      for (size_t i = ((size_t)cta * C::THREADS + tid) * 8; i < n; i += (size_t)G * C::THREADS * 8)
        *reinterpret_cast<uint4*>(p.y + i) = make_uint4(0, 0, 0, 0);
    }
    return;
  }

  const int phases = layer ? 2 : 1;
  if (warp == 0) {
    // ------------------------------------------------ weight producer
    if (lane == 0) {
      const uint64_t pol = l2_evict_first_policy();
      constexpr int srows = Q4 ? kDecKC4 / (Q4 ? GRP : 1) : 0;  // scale rows of a chunk
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int ph = 0; ph < phases && ok; ++ph) {
        const int NB = ph ? p.nb2 : p.nb1, KCN = ph ? p.kc2 : p.kc1;
        const Split sp((uint32_t)n_ent * NB * KCN, G);
        const CUtensorMap* mw = ph ? &maps.w2 : &maps.w1;
        const CUtensorMap* ms = ph ? &maps.s2 : &maps.s1;
        uint32_t x = sp.start(cta);
        const uint32_t end = sp.start(cta + 1);
        while (x < end && ok) {
          const int item = (int)(x / KCN);
          const int k0 = (int)(x - (uint32_t)item * KCN);
          const int k1 = (int)min((uint32_t)KCN, k0 + (end - x));
          const int ei = ph ? item % n_ent : item / NB;
          const int nb = ph ? item / n_ent : item % NB;
          const int e = c.ent[ei].expert;
          // first columns of the tile's two 64-column halves
          const bool sg = ph == 0 && swiglu;
          const int ca = sg ? nb * 64 : nb * kDecBN;
          const int cb = sg ? p.N1 + nb * 64 : ca + 64;
          for (int kc = k0; kc < k1; ++kc) {
            if (!mbar_wait(&c.wempty[stage], phase ^ 1u, wc)) {
              ok = false;
              break;
            }
            uint64_t* bar = &c.wfull[stage];
            uint8_t* dst = sW + stage * DF_W_BYTES;
            if constexpr (Q4) {
              mbar_arrive_expect_tx(bar, DF_W_BYTES + srows * 256);
              tma_load_3d_hint(dst, mw, bar, ca, kc * 32, e, pol);
              tma_load_3d_hint(dst + 4096, mw, bar, ca + 32, kc * 32, e, pol);
              tma_load_3d_hint(dst + 8192, mw, bar, cb, kc * 32, e, pol);
              tma_load_3d_hint(dst + 12288, mw, bar, cb + 32, kc * 32, e, pol);
              uint8_t* ds = sS + stage * C::S_BYTES;
              tma_load_3d_hint(ds, ms, bar, ca, kc * srows, e, pol);
              tma_load_3d_hint(ds + srows * 128, ms, bar, cb, kc * srows, e, pol);
            } else {
              mbar_arrive_expect_tx(bar, DF_W_BYTES);
              tma_load_3d_hint(dst, mw, bar, ca, kc * 64, e, pol);
              tma_load_3d_hint(dst + 8192, mw, bar, cb, kc * 64, e, pol);
            }
            ++issued;
            if (++stage == C::W_STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          x += k1 - k0;
        }
      }
      // a CTA that gave up still waits for its copies in flight (bounded)
      if (!ok || c.abort_flag) {
        for (int m = max(0, issued - C::W_STAGES); m < issued; ++m) {
          const uint32_t a = smem_u32(&c.wfull[m % C::W_STAGES]);
          const uint32_t par = (uint32_t)((m / C::W_STAGES) & 1);
          const uint64_t t0 = global_timer_ns();
          while (!mbar_try_wait(a, par) && global_timer_ns() - t0 < p.wait_limit_ns) {
          }
        }
      }
    }
    __syncwarp();
  } else if (warp <= C::LOADERS) {
    // ------------------------------------------------ row loaders
    const int lw = warp - 1;
    constexpr bool g32 = GRP == 32;
    uint32_t q = 0;  // chunks of this CTA so far (both products)
    bool ok = true;
    for (int ph = 0; ph < phases && ok; ++ph) {
      const int NB = ph ? p.nb2 : p.nb1, KCN = ph ? p.kc2 : p.kc1;
      const int K = ph ? p.K2 : p.K1;
      const Split sp((uint32_t)n_ent * NB * KCN, G);
      uint32_t x = sp.start(cta);
      const uint32_t end = sp.start(cta + 1);
      if (ph == 1 && x < end) {  // every CTA's h must be there
        int got = 1;
        if (lane == 0) {
          const uint64_t t0 = global_timer_ns();
          for (uint32_t it = 1; ld_acquire(p.barrier) < G; ++it) {
            if ((it & 63u) == 0) {
              if (c.abort_flag || global_timer_ns() - t0 > p.wait_limit_ns) {
                if (!c.abort_flag) {
                  *const_cast<volatile int*>(&c.abort_flag) = 1;
                  record_status(p.status, MOE_DEV_TIMEOUT);
                }
                got = 0;
                break;
              }
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, got, 0) != 0;
      }
      while (x < end && ok) {
        const int item = (int)(x / KCN);
        const int k0 = (int)(x - (uint32_t)item * KCN);
        const int k1 = (int)min((uint32_t)KCN, k0 + (end - x));
        const int ei = ph ? item % n_ent : item / NB;
        const DecEntry en = c.ent[ei];
        // source rows of this lane's two row numbers, lane and lane + 32
        const uint16_t* src = ph ? p.h : p.x;
        int r0 = en.row0 + lane, r1 = en.row0 + lane + 32;
        if (layer && ph == 0) {
          const int tk = p.T * p.k;
          if (lane < en.n) r0 = min(max(__ldg(p.perm + r0), 0), tk - 1) / p.k;
          if (lane + 32 < en.n) r1 = min(max(__ldg(p.perm + r1), 0), tk - 1) / p.k;
        }
        for (int kc = k0; kc < k1; ++kc, ++q) {
          if (q % C::LOADERS != (uint32_t)lw) continue;
          const uint32_t bs = q % C::B_STAGES;
          const uint32_t par = (q / C::B_STAGES) & 1;
          const uint32_t dst0 = smem_u32(sB + bs * C::B_STAGE);
          constexpr int PCS = C::KC / 8;       // 16-byte pieces of a row
          constexpr int RPP = 32 / PCS;        // rows per pass of the warp
          constexpr int UN = NT * 8 / RPP < 8 ? NT * 8 / RPP : 8;  // passes in flight together
          const int j = lane % PCS;
          const int kk = kc * C::KC + j * 8;
          // this lane's elements of h: the CTAs that share their item
          int o0 = 0, o1 = 0;
          if (ph == 1 && en.n <= kReaderRows && kk < K) {
            const int nb = swiglu ? kk >> 6 : kk >> 7;
            const Split s1((uint32_t)n_ent * p.nb1 * p.kc1, G);
            const uint32_t i0 = (uint32_t)(ei * p.nb1 + nb) * p.kc1;
            o0 = s1.owner(i0);
            o1 = s1.owner(i0 + p.kc1 - 1);
          }
          for (int rb = 0; rb < en.n; rb += RPP * UN) {
            uint4 v[UN];
#pragma unroll
            for (int u = 0; u < UN; ++u) {
              const int r = rb + u * RPP + lane / PCS;
              const int sr = __shfl_sync(0xffffffffu, (rb + u * RPP) < 32 ? r0 : r1, r & 31);
              v[u] = make_uint4(0, 0, 0, 0);
              if (r < en.n && kk < K && o0 == o1)
                v[u] = __ldcg(reinterpret_cast<const uint4*>(src + (size_t)sr * K + kk));
            }
            if (o0 != o1) {
#pragma unroll
              for (int u = 0; u < (kReaderRows + RPP - 1) / RPP; ++u) {
                const int r = u * RPP + lane / PCS;
                if (r < en.n) v[u] = sum_h_piece(p, o0, o1, r, kk, swiglu);
              }
            }
            // the rows' loads are on their way before the stage is free
            if (rb == 0 && !mbar_wait(&c.bempty[bs], par ^ 1u, wc)) {
              ok = false;
              break;
            }
#pragma unroll
            for (int u = 0; u < UN; ++u) {
              const int r = rb + u * RPP + lane / PCS;
              if (r >= en.n) continue;
              const uint32_t base = dst0 + (uint32_t)((r >> 3) * C::B_TILE);
              const uint32_t g = (uint32_t)(r & 7);
              if constexpr (Q4) {
                // 8 rows of K = one word of codes, held by the lanes t of an
                // m16n8k16 as the pairs (0, 4), (1, 5), (2, 6), (3, 7)
                const int jj = j & 7;
                const uint32_t t = g32 ? (uint32_t)(jj & 3) : (uint32_t)(jj >> 1);
                const uint32_t i = g32 ? (uint32_t)(jj >> 2) : (uint32_t)(jj & 1);
                sts128(base + (uint32_t)(j >> 3) * 1024 + i * 512 + t * 128 +
                           ((g ^ (2 * t)) * 16),
                       __byte_perm(v[u].x, v[u].z, 0x5410), __byte_perm(v[u].x, v[u].z, 0x7632),
                       __byte_perm(v[u].y, v[u].w, 0x5410), __byte_perm(v[u].y, v[u].w, 0x7632));
              } else {
                // word t of this piece is pair i = j % 4 of lane t's 16 bytes
                const uint32_t b0 = base + (uint32_t)(j >> 2) * 512 + (uint32_t)(j & 3) * 4;
                const uint32_t w4[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
                for (uint32_t t = 0; t < 4; ++t) sts32(b0 + t * 128 + ((g ^ (2 * t)) * 16), w4[t]);
              }
            }
          }
          if (!ok) break;
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.bfull[bs]);
        }
        x += k1 - k0;
      }
    }
  } else {
    // ------------------------------------------------ multiply, finish items
    const int cw = warp - 1 - C::LOADERS;
    const int wn = cw & (DF_WN - 1);
    const int kg = cw / DF_WN;
    const int g = lane >> 2, t = lane & 3;
    const int ctid = tid - 32 * (1 + C::LOADERS);  // < DF_FIN: kg = 0
    // this group's next chunk: its number q among the CTA's chunks (q mod KG =
    // kg), its place in the rings and their parities
    uint32_t q = (uint32_t)kg, qi = 0;
    int ws = kg, bs = kg;
    uint32_t wpar = 0, bpar = 0;
    static_assert(KG <= C::W_STAGES && KG <= C::B_STAGES, "a group steps over KG stages");
    bool ok = true;
    if (layer)  // the entry of each row, for the combine
      for (int i = ctid; i < n_ent; i += CTHREADS)
        for (int r = 0; r < c.ent[i].n; ++r) c.row_entry[c.ent[i].row0 + r] = (uint16_t)i;

    for (int ph = 0; ph < phases && ok; ++ph) {
      const int NB = ph ? p.nb2 : p.nb1, KCN = ph ? p.kc2 : p.kc1;
      const int N = ph ? p.N2 : p.N1;
      const Split sp((uint32_t)n_ent * NB * KCN, G);
      const bool sg = ph == 0 && swiglu;
      uint32_t x = sp.start(cta);
      const uint32_t end = sp.start(cta + 1);

      // this lane's place in a weight stage: tile columns 32 wn + ..
      uint32_t wofs[2], sofs = 0;
      if constexpr (Q4) {
        // word row 2t + i of step i (4i + t with 32-row groups, whose rows
        // must not mix): lane t holds 8 rows of K, the loaders order x alike
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t row = GRP == 32 ? (uint32_t)(4 * i + t) : (uint32_t)(2 * t + i);
          wofs[i] = (uint32_t)wn * 4096 + row * 128 + (((uint32_t)g ^ row) * 16);
        }
        sofs = (uint32_t)(wn >> 1) * (uint32_t)(kDecKC4 / (Q4 ? GRP : 1)) * 128 +
               (uint32_t)((wn & 1) * 32 + 4 * g) * 2;
      } else {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const uint32_t ch = (uint32_t)((wn & 1) * 4 + m * 2) + (uint32_t)((lane >> 3) & 1);
          const uint32_t row = (uint32_t)((lane >> 4) * 8 + (lane & 7));
          wofs[m] = (uint32_t)(wn >> 1) * 8192 + row * 128 + ((ch ^ (row & 7)) * 16);
        }
      }
      // element (m, n, r) of this lane: tile column and row of the entry
      auto col_of = [&](int m, int r) {
        return 32 * wn + (Q4 ? 4 * g + 2 * m + (r >> 1) : 16 * m + g + 8 * (r >> 1));
      };
      auto row_of = [&](int n, int r) { return n * 8 + 2 * t + (r & 1); };

      int cur_nb = -1;  // second product: column block of the items done so far
      while (ok) {
        const bool more = x < end;
        const int item = more ? (int)(x / KCN) : 0;
        const int nb = more ? (ph ? item / n_ent : item % NB) : -1;
        if (ph == 1 && cur_nb >= 0 && nb != cur_nb) {
          // ---- this CTA's part of column block cur_nb is written: count in,
          // and combine the block if it is the last part
          const uint32_t b0 = (uint32_t)cur_nb * n_ent * KCN;
          for (int i = ctid; i < n_ent; i += CTHREADS) {
            const uint32_t i0 = b0 + (uint32_t)i * KCN;
            c.owner[i] = make_int2(sp.owner(i0), sp.owner(i0 + KCN - 1));
          }
          named_sync(BAR_CONS, CTHREADS);
          if (ctid == 0) {
            const int parts = c.owner[n_ent - 1].y - c.owner[0].x + 1;
            __threadfence();
            c.last = atomicAdd(p.col_tickets + cur_nb, 1u) == (unsigned)(parts - 1);
            __threadfence();
          }
          named_sync(BAR_CONS, CTHREADS);
          if (c.last) {
            const int col0 = cur_nb * kDecBN;
            for (int i = ctid; i < p.T * (kDecBN / 2); i += CTHREADS) {
              const int tok = i / (kDecBN / 2);
              const int cl = (i % (kDecBN / 2)) * 2;
              if (col0 + cl >= N) continue;
              float y0 = 0.f, y1 = 0.f;
#pragma unroll 4
              for (int j = 0; j < p.k; ++j) {
                const int row = c.slot[tok * p.k + j];
                if (row < 0) continue;
                const float w = c.gate[tok * p.k + j];
                const int ei = c.row_entry[row];
                const int2 own = c.owner[ei];
                float2 v;
                if (own.x == own.y) {
                  v = __ldcg(reinterpret_cast<const float2*>(p.yfull + (size_t)row * N + col0 + cl));
                } else {
                  v = make_float2(0.f, 0.f);
                  const int rr = row - c.ent[ei].row0;
#pragma unroll 4
                  for (int o = own.x; o <= own.y; ++o) {
                    const float2 u = __ldcg(reinterpret_cast<const float2*>(
                        p.parts2 + ((size_t)(o * 2 + (o == own.x ? 1 : 0)) * p.row_cap + rr) * kDecBN +
                        cl));
                    v.x += u.x;
                    v.y += u.y;
                  }
                }
                y0 = fmaf(w, v.x, y0);
                y1 = fmaf(w, v.y, y1);
              }
              *reinterpret_cast<uint32_t*>(p.y + (size_t)tok * N + col0 + cl) = pack_bf16x2(y0, y1);
            }
          }
        }
        if (!more) break;
        cur_nb = nb;
        const int k0 = (int)(x - (uint32_t)item * KCN);
        const int k1 = (int)min((uint32_t)KCN, k0 + (end - x));
        const DecEntry en = c.ent[ph ? item % n_ent : item / NB];

        float acc[2][NT][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[m][n][r] = 0.f;

        for (; q < qi + (uint32_t)(k1 - k0); q += KG) {
          if (!mbar_wait(&c.wfull[ws], wpar, wc) || !mbar_wait(&c.bfull[bs], bpar, wc)) {
            ok = false;
            break;
          }
          const uint32_t w0 = smem_u32(sW + ws * DF_W_BYTES);
          const uint32_t b0 = smem_u32(sB + bs * C::B_STAGE) + (uint32_t)(t * 128 + ((g ^ (2 * t)) * 16));
          const auto chunk = [&](auto nta) {
            constexpr int NTA = decltype(nta)::value;
            if constexpr (Q4)
              chunk_q4<NT, NTA, GRP>(acc, w0, wofs, b0, smem_u32(sS + ws * C::S_BYTES) + sofs);
            else
              chunk_bf16<NT, NTA>(acc, w0, wofs, b0);
          };
          if (NT == 1 || en.n <= 8)
            chunk(Int<1>{});
          else if (NT == 2 || en.n <= 16)
            chunk(Int<NT < 2 ? NT : 2>{});
          else if (NT == 4 || en.n <= 32)
            chunk(Int<NT < 4 ? NT : 4>{});
          else
            chunk(Int<NT>{});
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&c.wempty[ws]);
            mbar_arrive(&c.bempty[bs]);
          }
          if ((ws += KG) >= C::W_STAGES) {
            ws -= C::W_STAGES;
            wpar ^= 1u;
          }
          if ((bs += KG) >= C::B_STAGES) {
            bs -= C::B_STAGES;
            bpar ^= 1u;
          }
        }
        qi += (uint32_t)(k1 - k0);
        // ---- sum over the warps that split K: the others hand over to kg = 0.
        // A wait that ran out in any warp ends the work of all of them here.
        if (kg > 0) {
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int r = 0; r < 4; ++r)
                sRed[(((kg - 1) * 2 * NT + m * NT + n) * 4 + r) * DF_FIN + wn * 32 + lane] = acc[m][n][r];
        }
        if (named_any(BAR_CONS, CTHREADS, !ok)) {
          ok = false;
          break;
        }
        if (kg == 0) {
#pragma unroll
          for (int u = 0; u < KG - 1; ++u)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  acc[m][n][r] += sRed[((u * 2 * NT + m * NT + n) * 4 + r) * DF_FIN + wn * 32 + lane];
          const bool whole = k0 == 0 && k1 == KCN;
          bool write = whole;
          if (!whole) {
            // partial tile of this CTA: slot 0 if the item began in an
            // earlier CTA, else slot 1
            float* mine = (ph ? p.parts2 : p.parts) +
                          (size_t)(cta * 2 + (k0 > 0 ? 0 : 1)) * p.row_cap * kDecBN;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  if (row_of(n, r) < en.n) mine[row_of(n, r) * kDecBN + col_of(m, r)] = acc[m][n][r];
            if (ph == 0 && (!layer || en.n > kReaderRows)) {
              const uint32_t i0 = (uint32_t)item * KCN;
              const int c0 = sp.owner(i0), c1 = sp.owner(i0 + KCN - 1);
              named_sync(BAR_FIN, DF_FIN);
              if (ctid == 0) {
                __threadfence();
                c.last = atomicAdd(p.item_tickets + c0, 1u) == (unsigned)(c1 - c0);
                __threadfence();
              }
              named_sync(BAR_FIN, DF_FIN);
              if (c.last) {
                write = true;
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                  for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                      float v = 0.f;
                      if (row_of(n, r) < en.n) {
                        const float* src = p.parts + row_of(n, r) * kDecBN + col_of(m, r);
                        for (int o = c0; o <= c1; ++o)
                          v += __ldcg(src + (size_t)(o * 2 + (o == c0 ? 1 : 0)) * p.row_cap * kDecBN);
                      }
                      acc[m][n][r] = v;
                    }
              }
            }
          }
          if (write) {
            if (ph == 1) {  // whole items of the second product stay in fp32 for the combine
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                  for (int r = 0; r < 4; ++r) {
                    const int col = nb * kDecBN + col_of(m, r);
                    if (row_of(n, r) < en.n && col < N)
                      p.yfull[(size_t)(en.row0 + row_of(n, r)) * N + col] = acc[m][n][r];
                  }
            } else {
              uint16_t* out = layer ? p.h : p.y;
              if (sg) {  // gate columns meet up columns: warps 2, 3 hand over to 0, 1
                named_sync(BAR_FIN, DF_FIN);  // sRed is read
                if (wn >= 2) {
#pragma unroll
                  for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                      for (int r = 0; r < 4; ++r)
                        sRed[((m * NT + n) * 4 + r) * 64 + (wn - 2) * 32 + lane] = acc[m][n][r];
                }
                named_sync(BAR_FIN, DF_FIN);
              }
              if (!sg || wn < 2) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                  for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                      const int col = nb * (sg ? 64 : kDecBN) + col_of(m, r);
                      if (row_of(n, r) < en.n && col < N) {
                        float v = acc[m][n][r];
                        if (sg)
                          v = dec_silu(v) * sRed[((m * NT + n) * 4 + r) * 64 + wn * 32 + lane];
                        else if (layer)
                          v = dec_gelu(v);
                        out[(size_t)(en.row0 + row_of(n, r)) * N + col] =
                            (uint16_t)(pack_bf16x2(v, 0.f) & 0xFFFFu);
                      }
                    }
              }
            }
          }
        }
        x += k1 - k0;
        // sRed is read (every consumer passes here once an item)
        if (x < end) named_sync(BAR_CONS, CTHREADS);
      }
      if (ph == 0 && layer) {
        // this CTA's h is written: arrive at the grid barrier
        named_sync(BAR_CONS, CTHREADS);
        if (ctid == 0) {
          __threadfence();
          red_release(p.barrier, 1u);
        }
      }
    }
  }
}

template <int GRP, int NT>
cudaError_t ffn_launch(const DecFfnMaps& m, const DecFfnArgs& a, int ctas, cudaStream_t st) {
  using C = Cfg<(GRP > 0), NT>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3((unsigned)C::THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_ffn_kernel<GRP, NT>, m, a);
}

template <int GRP>
cudaError_t ffn_rows(const DecFfnMaps& m, const DecFfnArgs& a, int ctas, cudaStream_t st) {
  if (a.row_cap <= 8) return ffn_launch<GRP, 1>(m, a, ctas, st);
  if (a.row_cap <= 16) return ffn_launch<GRP, 2>(m, a, ctas, st);
  if (a.row_cap <= 32) return ffn_launch<GRP, 4>(m, a, ctas, st);
  return ffn_launch<GRP, 8>(m, a, ctas, st);
}

template <int GRP, int NT>
cudaError_t ffn_attr() {
  return cudaFuncSetAttribute(decode_ffn_kernel<GRP, NT>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)Cfg<(GRP > 0), NT>::SMEM);
}

template <int GRP>
cudaError_t ffn_attrs() {
  cudaError_t e = ffn_attr<GRP, 1>();
  if (e == cudaSuccess) e = ffn_attr<GRP, 2>();
  if (e == cudaSuccess) e = ffn_attr<GRP, 4>();
  if (e == cudaSuccess) e = ffn_attr<GRP, 8>();
  return e;
}

}  // namespace
}  // namespace moe
