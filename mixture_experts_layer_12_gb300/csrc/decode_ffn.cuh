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
//     tile in the workspace, and the tiles are added in CTA order, so the sum
//     has one order whoever comes last.
//   * One warp issues TMA loads of weights into a ring of stages and runs ahead
//     of everything: while the CTAs meet at the grid barrier between the two
//     products, the ring already fills with W2.
//   * Three warps copy the rows' K chunk (x, then h) into the same stage with
//     cp.async.  With 150 KB of weights on their way to every SM any other
//     access waits in the same queues for 2-3 us, so the rows have to be asked
//     for as early as the weights are: warps that loaded a chunk each and
//     waited for it were what bound the kernel (a 4-bit chunk took 1400
//     clocks, 600 of them multiplying).
//   * The consumer warps multiply: m16n8k16 products with the weights as M (32
//     columns of W per warp) and the rows as N (8 at a time).  A weight is
//     loaded from shared memory once and used for every row.  bf16 weights
//     come out of the 128-byte-swizzled stage by ldmatrix.trans.  4-bit codes
//     are turned into bf16 in registers; the products are exact in fp32, 32
//     rows of K are summed in fp32 and multiplied by their scale in fp32.
//   tcgen05 is not used: for bf16 the stream, not the multiply, is the bound (one
//   m16n8k16 per 256 weights is a tenth of the tensor rate at 8 rows), and 4-bit
//   weights expanded to bf16 in shared memory would write and read 94 bytes per
//   clock there, of the 128 it moves.  Both hold for few rows: from 17 rows of an
//   expert on, with 4 bits, the products and their scaling take more clocks than
//   the memory (860 and 1560 a chunk for 16 and 32 rows, where it takes 700).
//   Weights unpacked into tensor memory as the A operand have not been tried.
//   * Between the products h goes through memory.  An item shared by several
//     CTAs is put together by its first CTA, whose last it is, while the later
//     ones begin with it and have counted in by then; by all CTAs, after a grid
//     barrier, where it has many rows; or, where a CTA's part of the second
//     product needs little of h, by every CTA for the elements it needs.
//   * Combine: after a grid barrier all CTAs sum the tokens' experts in slot
//     order, 128 columns of a token per warp.
// The grid barriers need all CTAs resident, which the cooperative launch
// guarantees; they and every other wait are bounded.
// Measured with the first kernel, GPU time of a call: one token, 8 experts of 4096 x
// 14336, 2 of them: 80 us in bf16 (5.9 TB/s, 0.87 of the copy bandwidth), 47 us gated
// in 4 bits; 16 tokens in 4 bits 97 us (4.9 TB/s), 64 tokens 231; 64 experts of 2048 x
// 1408, 4 of them, gated: 25 us in bf16, of which 10 are the weights; 4096 x 14336 in
// 4 bits times a row: 12.4 us, 4.5 of them the weights.  What is left beside the stream is a
// chain of trips to memory: the list (1 us) and the first chunk (2 us), partial tiles
// and h between the products (4-5 us) and the combine (2-3 us).
#pragma once

#include "decode_internal.h"
#include "tc_common.cuh"

namespace moe {
namespace {

constexpr int DF_WN = 4;            // consumer warps across the columns
constexpr int DF_FIN = 32 * DF_WN;  // threads that write an item out
constexpr int DF_W_BYTES = 16384;
// 8 chunks of 16 KB keep the memory busy; with 12 on their way everything else
// (rows, partial tiles) waits longer behind them, and one token's bf16 layer of
// 4096 x 14336 takes 82.5 us instead of 79.6.  6 are as good but for many rows.
constexpr int DF_MAX_STAGES = 8;
constexpr int DF_SMEM = 227 * 1024;
constexpr int DF_CACHE = 24 * 1024; // h kept whole by its readers: at most this much of it

// Consumer warps: KG groups of 4 across the columns; group i takes every KG-th
// chunk, so that a warp has a chunk's whole K to keep its pipes full between two
// waits, and writes out every KG-th item while the other goes on multiplying.
// 2 groups unpack and multiply a 4-bit chunk of up to 8 rows in 530 to 630
// clocks, where one SM's share of the memory brings it in 700.  With 3 groups the
// registers spill, and the layers took as long.
constexpr int KG = 2;
constexpr int DF_LOADERS = 3;  // row loaders: 12 warps in all, 3 to a scheduler

// grid barriers: the first product's tiles are written, h is, the second's are
constexpr int kGridTiles = 0, kGridH = 1, kGridY = 2;

// named barriers: set-up; all consumers; the writers of an item (one per group); an
// item's hand-over between the groups (one per writing group)
constexpr int BAR_SETUP = 0;
constexpr int BAR_CONS = 1;
constexpr int BAR_FIN = 2;
constexpr int BAR_ITEM = BAR_FIN + KG;
constexpr int BAR_ROWS = BAR_ITEM + KG;  // the row loaders

__device__ __forceinline__ void named_sync(int id, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ void named_arrive(int id, int n) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}
// 16 bytes to shared memory, zeros where `bytes` is 0; arrives on the barrier
// (as one of its expected arrivals) when this thread's copies are done
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_load_3d_hint(void* dst, const CUtensorMap* m, uint64_t* bar,
                                                 int c0, int c1, int c2, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "l"(pol)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d_hint(void* dst, const CUtensorMap* m, uint64_t* bar,
                                                 int c0, int c1, int c2, int c3, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "l"(pol)
      : "memory");
}
__device__ __forceinline__ unsigned ld_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// counts in: earlier writes of the CTA (a barrier before it) are visible to whoever
// sees the count
__device__ __forceinline__ void red_release(unsigned* p, unsigned v) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
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
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(a), "r"(x), "r"(y) : "memory");
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
// (c - 8) / 64, exactly (an item's sums are multiplied by 64 at its end).  A code at bits 0-3
// or 4-7 of a half word is, read as bf16, c or 16 c times 2^-133 (the numbers
// below 2^-125 are evenly spaced), so one masked word and one fused
// multiply-add make a pair, and a word needs one shift: 9 instructions for 8
// codes where (128 + c) - 136 takes 11, of which the shifts and masks run at
// half rate (one row times 4096 x 14336: 18.8 -> 17.9 us when it was introduced).
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

struct Ctrl {
  uint64_t full[DF_MAX_STAGES], empty[DF_MAX_STAGES];
  int abort_flag;
  int n_entries;
  int max_rows;
  DecEntry ent[kDecMaxEntries];
  uint16_t row_entry[MOED_MAX_ROWS];  // layer: entry of a row
  int16_t tok[MOED_MAX_ROWS];         // row of x of a dispatch row
  int16_t slot[MOED_MAX_ROWS];        // layer: [T, k]
  float gate[MOED_MAX_ROWS];
};
static_assert(sizeof(Ctrl) <= 12 * 1024, "control area");

// One product's chunks, in item order, dealt to the first G CTAs: CTA c < G takes
// chunks [total c / G, total (c + 1) / G), at least one.  `least`: chunks that are
// worth a CTA of their own (a small product cut finer is read faster than its
// many partial tiles are added).  The host keeps total * CTAs below 2^32.
struct Split {
  uint32_t total, G;
  __device__ __forceinline__ Split(uint32_t n, uint32_t ctas, uint32_t least)
      : total(n), G(max(1u, min(ctas, n / least))) {}
  __device__ __forceinline__ uint32_t start(uint32_t c) const {
    return c < G ? total * c / G : total;
  }
  // the CTA that holds chunk x: the largest c with total c / G < x + 1
  __device__ __forceinline__ int owner(uint32_t x) const {
    return (int)(((x + 1) * G - 1) / total);
  }
};

__device__ __forceinline__ void add4(float4& a, const float4 b) {
  a.x += b.x;
  a.y += b.y;
  a.z += b.z;
  a.w += b.w;
}

// 4 columns of the first product (and of the up projection), activated and rounded
// to bf16: h is the operand of the second product, whose weights are bf16 or exact in
// it, and moe_forward rounds it too; two halves of it would double that product.
// It is most of what a layer's y is off beyond its own rounding (2.3e-3 of y against 64
// bits, 1.7e-3 from the rounding of y).
__device__ __forceinline__ uint2 activated(int act, float4 z, const float4& u) {
  if (act == kDecSwiGLU) {
    z = make_float4(dec_silu(z.x) * u.x, dec_silu(z.y) * u.y, dec_silu(z.z) * u.z, dec_silu(z.w) * u.w);
  } else if (act == kDecGelu) {
    z = make_float4(dec_gelu(z.x), dec_gelu(z.y), dec_gelu(z.z), dec_gelu(z.w));
  }
  return make_uint2(pack_bf16x2(z.x, z.y), pack_bf16x2(z.z, z.w));
}
__device__ __forceinline__ void write_piece(const DecFfnArgs& p, size_t at, const float4& z, const float4& u) {
  *reinterpret_cast<uint2*>((p.act == kDecNone ? p.y : p.h) + at) = activated(p.act, z, u);
}

// The first product's items and partial tiles: 2^sh columns of h each, rows of 128
// floats; `up`: from a gate's column to the up projection's; `tile`: floats of a tile.
struct Items {
  int sh, up;
  size_t tile;
};

// A whole item of the first product, from its sums in shared memory (z, and u where
// gated), by one group (128 threads): 4 columns of a row per thread and step.
__device__ __forceinline__ void write_item(const DecFfnArgs& p, const Items& g, const DecEntry& en, int nb,
                                           int ftid, const float* z, const float* u) {
  const bool swiglu = p.act == kDecSwiGLU;
#pragma unroll 1
  for (int i = ftid; i < en.n << (g.sh - 2); i += DF_FIN) {
    const int r = i >> (g.sh - 2), cl = (i - (r << (g.sh - 2))) * 4;
    const int col = (nb << g.sh) + cl;
    if (col >= p.N1) continue;  // N1 is a multiple of 8
    const float4 a = *reinterpret_cast<const float4*>(z + r * kDecBN + cl);
    write_piece(p, (size_t)(en.row0 + r) * p.N1 + col, a,
                swiglu ? *reinterpret_cast<const float4*>(u + r * kDecBN + cl) : a);
  }
}

// A shared item of the first product by its first CTA, all consumer threads: its
// own sums, from shared memory, and the tiles of the `more` CTAs after it in that
// order (their slot 0).
template <int CTHREADS>
__device__ __forceinline__ void finish_item(const DecFfnArgs& p, const Items& g, const DecEntry& en, int nb,
                                            const float* own_z, const float* own_u, int cta, int more, int ctid) {
  const bool swiglu = p.act == kDecSwiGLU;
#pragma unroll 1
  for (int i = ctid; i < en.n << (g.sh - 2); i += CTHREADS) {
    const int r = i >> (g.sh - 2), cl = (i - (r << (g.sh - 2))) * 4;
    const int col = (nb << g.sh) + cl;
    if (col >= p.N1) continue;  // N1 is a multiple of 8
    const int at = r * kDecBN + cl;
    const float* s = p.parts + (size_t)(cta * 2) * g.tile + at;
    float4 z = *reinterpret_cast<const float4*>(own_z + at);
    float4 u = swiglu ? *reinterpret_cast<const float4*>(own_u + at) : z;
#pragma unroll 4
    for (int o = 1; o <= more; ++o) {
      add4(z, __ldcg(reinterpret_cast<const float4*>(s + (size_t)(2 * o) * g.tile)));
      if (swiglu) add4(u, __ldcg(reinterpret_cast<const float4*>(s + (size_t)(2 * o) * g.tile + g.up)));
    }
    write_piece(p, (size_t)(en.row0 + r) * p.N1 + col, z, u);
  }
}

// Warp-wide wait until a counter in memory has reached `value`; gives up when another
// role of the CTA did, or makes the others give up when it ran out.  One warp of a
// CTA waits and the others wait for it: 152 polls at a time delay the arrivals and
// everybody's data less than 1216 (one token's layer of narrow experts 27.5 -> 26.7 us).
__device__ __forceinline__ void count_wait(const DecFfnArgs& p, const unsigned* at, uint32_t value, int& abort_flag,
                                           int lane) {
  volatile int* abort = &abort_flag;
  if (lane == 0) {
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1; ld_acquire(at) < value; ++it) {
      if ((it & 63u) == 0) {
        if (*abort) break;
        if (global_timer_ns() - t0 > p.wait_limit_ns) {
          *abort = 1;
          record_status(p.status, MOE_DEV_TIMEOUT);
          break;
        }
      }
    }
  }
  __syncwarp();  // orders the other lanes' reads after lane 0's acquire
}

// y by the consumer warps of all CTAs, once every CTA's parts of it are there:
// 128 columns of a token per warp and step, 4 per lane, its experts summed in slot
// order, their rows whole from yfull or, where CTAs share the item, from their
// tiles in order (the first one's slot 1, the later ones' slot 0).
// The same tile of 4 experts is asked for at once: one expert after the other is 4
// trips to memory in a row (narrow experts, one token: 26.8 us instead of 25.1).
// DEEP: tiles of each of them in flight together, as many as the registers of the
// kernel leave room for.
template <int DEEP>
__device__ __forceinline__ void combine(const DecFfnArgs& p, Ctrl& c, const Split& sp, int cw,
                                        int gw, int warps, int threads, int lane) {
  const int N = p.N2;
  const size_t tile = (size_t)p.row_cap * kDecBN;
  const int tasks = p.T * p.nb2;
  bool waited = false;
  if (gw >= tasks && (int)blockIdx.x < tasks) named_sync(BAR_CONS, threads);  // another warp's wait, below
#pragma unroll 1
  for (int task = gw; task < tasks; task += warps) {
    const int tok = task / p.nb2, nb = task % p.nb2;
    const int col = nb * kDecBN + lane * 4;  // N is a multiple of 8: all 4 columns or none
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int j0 = 0; j0 < p.k; j0 += 4) {  // 4 experts' loads in flight together
      const float* src[4];
      int more[4];
      float4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int row = j0 + u < p.k ? c.slot[tok * p.k + j0 + u] : -1;
        more[u] = 0;
        src[u] = nullptr;
        if (row >= 0) {
          const int ei = c.row_entry[row];
          const uint32_t i0 = ((uint32_t)nb * c.n_entries + ei) * p.kc2;
          const int o0 = sp.owner(i0);
          more[u] = sp.owner(i0 + p.kc2 - 1) - o0;
          src[u] = more[u] == 0 ? p.yfull + (size_t)row * N + col
                                : p.parts2 + (size_t)(o0 * 2 + 1) * tile + (row - c.ent[ei].row0) * kDecBN + lane * 4;
        }
      }
      if (!waited) {
        if (cw == 0) count_wait(p, p.barrier + kGridY, p.arrivals, c.abort_flag, lane);
        named_sync(BAR_CONS, threads);
        waited = true;
      }
      if (col < N) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          v[u] = src[u] ? __ldcg(reinterpret_cast<const float4*>(src[u])) : make_float4(0.f, 0.f, 0.f, 0.f);
        const int most = max(max(more[0], more[1]), max(more[2], more[3]));
#pragma unroll 1
        for (int o0 = 1; o0 <= most; o0 += DEEP) {
          float4 t[DEEP][4];
#pragma unroll
          for (int d = 0; d < DEEP; ++d)
#pragma unroll
            for (int u = 0; u < 4; ++u)
              t[d][u] = o0 + d <= more[u]
                            ? __ldcg(reinterpret_cast<const float4*>(src[u] + (size_t)(2 * (o0 + d) - 1) * tile))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int d = 0; d < DEEP; ++d)
#pragma unroll
            for (int u = 0; u < 4; ++u) add4(v[u], t[d][u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (src[u]) {
            const float w = c.gate[tok * p.k + j0 + u];
            y.x = fmaf(w, v[u].x, y.x);
            y.y = fmaf(w, v[u].y, y.y);
            y.z = fmaf(w, v[u].z, y.z);
            y.w = fmaf(w, v[u].w, y.w);
          }
        }
      }
    }
    if (col < N)
      *reinterpret_cast<uint2*>(p.y + (size_t)tok * N + col) =
          make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
  }
}

// All shared items of the first product by the consumer warps of all CTAs, once
// every CTA's tiles are there: a row of an item per warp and step.
__device__ __forceinline__ void finish_all(const DecFfnArgs& p, const Items& g, Ctrl& c, const Split& sp, int gw, int warps,
                                           int lane) {
  const bool swiglu = p.act == kDecSwiGLU;
  const int KCN = p.kc1, rows = c.max_rows;
  const int tasks = ((int)sp.G - 1) * rows;  // an item belongs to the first border of CTAs inside it
#pragma unroll 1
  for (int task = gw; task < tasks; task += warps) {
    const uint32_t b = (uint32_t)(task / rows) + 1;
    const int r = task % rows;
    const uint32_t x = sp.start(b);
    const int item = (int)(x / KCN);
    const uint32_t i0 = (uint32_t)item * KCN;
    if (x == i0 || sp.owner(i0) != (int)b - 1) continue;
    const DecEntry en = c.ent[item / p.nb1];
    if (r >= en.n) continue;
    const int more = sp.owner(i0 + KCN - 1) - ((int)b - 1);
    const int col = (item % p.nb1 << g.sh) + lane * 4;
    if (col >= p.N1 || lane * 4 >= 1 << g.sh) continue;
    const float* s = p.parts + (size_t)((b - 1) * 2 + 1) * g.tile + r * kDecBN + lane * 4;
    float4 z = __ldcg(reinterpret_cast<const float4*>(s));
    float4 u = swiglu ? __ldcg(reinterpret_cast<const float4*>(s + g.up)) : z;
#pragma unroll 4
    for (int o = 1; o <= more; ++o) {
      const float* q = s + (size_t)(2 * o - 1) * g.tile;
      add4(z, __ldcg(reinterpret_cast<const float4*>(q)));
      if (swiglu) add4(u, __ldcg(reinterpret_cast<const float4*>(q + g.up)));
    }
    write_piece(p, (size_t)(en.row0 + r) * p.N1 + col, z, u);
  }
}

template <int V>
struct Int {
  static constexpr int value = V;
};

template <bool Q4, int NT>
struct Cfg {
  static constexpr int CONSUMERS = DF_WN * KG;
  static constexpr int THREADS = 32 * (1 + DF_LOADERS + CONSUMERS);
  static constexpr int KC = Q4 ? kDecKC4 : kDecKC16;    // K rows of a chunk
  static constexpr int PITCH = KC * 2 + 16;             // bytes of a row's chunk: no bank conflicts
  static constexpr int S_BYTES = Q4 ? 8 * 256 : 0;      // scales: up to 8 groups x 128 columns
  static constexpr int W_STAGE = DF_W_BYTES + S_BYTES;
  static constexpr int RED_GROUP = DF_FIN * 2 * NT * 4;    // floats a group hands over: 8 NT rows x 128
  static constexpr int RED = KG * RED_GROUP * 4;
  static constexpr int CTRL = 12 * 1024;
  static constexpr int SPACE = DF_SMEM - 1024 - RED - CTRL;  // for the rings
  // Reads of rows past an entry's last stay inside: RED and CTRL follow the rows.  An
  // entry is multiplied in tiles of 8, 16, 32 or 64 rows, of which it has more than
  // half, or has 1 of 8.
  static_assert(RED + CTRL >= (NT == 1 ? 7 : 4 * NT - 1) * PITCH, "room behind the rows");
  static_assert(SPACE >= 2 * KG * W_STAGE, "weight ring");
};

// One chunk of 4-bit weights for a warp's 32 columns and the first NTA 8-row
// tiles: acc += W^T x.  w0: the weight stage, wofs: this lane's place in it at
// even and odd steps of 32 rows of K; bl, bofs: the same in the rows; sl: its 4
// columns' scales.  Nothing branches and, as far as the registers go, everything
// is unrolled, so that loads, unpacking and products of different steps overlap.
// The sum over a group of rows (over 32 of them where more sums would not fit the
// registers) begins at zero and is scaled and added in fp32; sums over 32 rows of
// larger groups take a 4-bit layer of 16 tokens from 110 to 115 us.
template <int NT, int NTA, int GRP>
__device__ __forceinline__ void chunk_q4(float (&acc)[2][NT][4], uint32_t w0, const uint32_t (&wofs)[2],
                                         uint32_t bl, const uint32_t (&bofs)[2], uint32_t sl) {
  constexpr int UNROLL = NTA == 1 ? kDecKC4 / 64 : NTA == 2 ? 2 : 1;
  constexpr uint32_t SUM = NT <= 2 ? GRP : 32;  // rows of a sum
  float s[4] = {0.f, 0.f, 0.f, 0.f}, part[NTA][2][4];
#pragma unroll UNROLL
  for (uint32_t blk = 0; blk < kDecKC4 / 64; ++blk) {  // 64 rows of K
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i) {
      const uint32_t step = blk * 2 + i;
      const bool first = step % (SUM / 32) == 0, last = (step + 1) % (SUM / 32) == 0;
      if (GRP < 128 ? step % (GRP / 32) == 0 : first && i == 0) {
        uint32_t s01, s23;
        lds64(sl + (blk * 64 + i * 32) / GRP * 256, s01, s23);
        s[0] = bf16_lo(s01);
        s[1] = bf16_hi(s01);
        s[2] = bf16_lo(s23);
        s[3] = bf16_hi(s23);
      }
      uint32_t v[4];  // columns 4g .. 4g + 3 of 8 rows of K
      lds128(w0 + blk * 1024 + wofs[i], v);
      uint32_t a[2][8];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint32_t va = v[2 * m], vb = v[2 * m + 1];
        a[m][0] = q4_pair<0>(va);
        a[m][1] = q4_pair<0>(vb);
        a[m][2] = q4_pair<1>(va);
        a[m][3] = q4_pair<1>(vb);
        a[m][4] = q4_pair<2>(va);
        a[m][5] = q4_pair<2>(vb);
        a[m][6] = q4_pair<3>(va);
        a[m][7] = q4_pair<3>(vb);
      }
#pragma unroll
      for (int n = 0; n < NTA; ++n) {
        uint32_t x[4];  // the same 8 rows of K, paired as the codes are
        lds128(bl + n * 8 * (kDecKC4 * 2 + 16) + blk * 128 + bofs[i], x);
        const uint32_t b0 = __byte_perm(x[0], x[2], 0x5410), b1 = __byte_perm(x[0], x[2], 0x7632);
        const uint32_t b2 = __byte_perm(x[1], x[3], 0x5410), b3 = __byte_perm(x[1], x[3], 0x7632);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if (first)
            mma_bf16_zero(part[n][m], a[m][0], a[m][1], a[m][2], a[m][3], b0, b1);
          else
            mma_bf16(part[n][m], a[m][0], a[m][1], a[m][2], a[m][3], b0, b1);
          mma_bf16(part[n][m], a[m][4], a[m][5], a[m][6], a[m][7], b2, b3);
          if (last)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[m][n][r] = fmaf(s[2 * m + (r >> 1)], part[n][m][r], acc[m][n][r]);
        }
      }
    }
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
      ldsm_x4(bl + n * 8 * (kDecKC16 * 2 + 16) + blk * 64, b);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        mma_bf16(acc[m][n], a[m][0][0], a[m][0][1], a[m][0][2], a[m][0][3], b[0], b[1]);
        mma_bf16(acc[m][n], a[m][1][0], a[m][1][1], a[m][1][2], a[m][1][3], b[2], b[3]);
      }
    }
  }
}

// GRP: rows per scale of 4-bit weights; 0: bf16 weights; kDecPair: bf16, gated, and
// the chunks of the gate and of the up projection alternate.
template <int GRP, int NT>
__global__ void __launch_bounds__(Cfg<(GRP > 0), NT>::THREADS, 1)
    decode_ffn_kernel(const __grid_constant__ DecFfnMaps maps, const DecFfnArgs p) {
  constexpr bool Q4 = GRP > 0;
  using C = Cfg<Q4, NT>;
  constexpr int CTHREADS = 32 * C::CONSUMERS;
  constexpr int PCS = C::KC / 8;  // 16-byte pieces of a row's chunk
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  // [weights | scales | rows] fill SPACE, divided below once the rows are known
  uint8_t* sW = smem;
  float* sRed = reinterpret_cast<float*>(smem + C::SPACE);
  Ctrl& c = *reinterpret_cast<Ctrl*>(smem + C::SPACE + C::RED);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int cta = blockIdx.x;
  const uint32_t G = gridDim.x;
  const bool layer = p.act != kDecNone;
  const bool swiglu = p.act == kDecSwiGLU;
  // Gated experts: an item is 64 columns of the gate and 64 of the up projection, and
  // a chunk holds both; or (pair) 128 of either, whose chunks alternate, so that one
  // group of consumers sums the gate and the other the up projection.
  constexpr bool pair = GRP == kDecPair;
  const Items g1{swiglu && !pair ? 6 : 7, pair ? p.row_cap * kDecBN : 64,
                 (size_t)p.row_cap * kDecBN * (pair ? 2 : 1)};

  if (tid == 0) {
    for (int i = 0; i < DF_MAX_STAGES; ++i) {
      mbar_init(&c.full[i], 1 + 32 * DF_LOADERS);  // the weights' producer, the row loaders' lanes
      mbar_init(&c.empty[i], DF_WN);
    }
    c.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.w1);
    if (layer) tma_prefetch_desc(&maps.w2);
  }
  pdl_launch_dependents();
  pdl_wait();
  // the first kernel's list, by the weights' warp, which goes on as soon as it
  // has it; the routing by the others
  if (warp == 0) {
    const int2 v = __ldcg(reinterpret_cast<const int2*>(p.ctrl + kDecCountOffset / 4));
    for (int i = lane; i < p.max_entries; i += 32) {
      const int4 e = __ldcg(reinterpret_cast<const int4*>(p.entries) + i);
      c.ent[i] = DecEntry{e.x, e.y, e.z, e.w};
    }
    if (lane == 0) {
      c.n_entries = min(v.x, p.max_entries);
      c.max_rows = min(v.y, p.row_cap);
    }
    __syncwarp();
    named_arrive(BAR_SETUP, C::THREADS);
  } else {
    for (int i = tid - 32; i < p.T * p.k; i += C::THREADS - 32) {
      if (layer) {
        c.slot[i] = (int16_t)__ldcg(p.slot + i);
        c.gate[i] = __ldcg(p.gate + i);
        c.tok[i] = (int16_t)(min(max(__ldcg(p.perm + i), 0), p.T * p.k - 1) / p.k);
      } else {
        c.tok[i] = (int16_t)i;
      }
    }
    named_sync(BAR_SETUP, C::THREADS);
  }
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
  // ---- the rings: as many stages (a multiple of KG, see the consumers) as
  // fit beside the rows' chunks and, where it is small, this CTA's part of h
  const int max_rows = c.max_rows;
  const int row_bytes = max_rows * C::PITCH;
  // the second product's chunks of a CTA, at most
  const Split s2((uint32_t)n_ent * p.nb2 * p.kc2, G, p.least2);
  const uint32_t cpc = (s2.total + s2.G - 1) / s2.G;
  const bool reader = layer && cpc * (uint32_t)row_bytes <= (uint32_t)DF_CACHE;
  int S = DF_MAX_STAGES / KG * KG;
  for (; S > KG; S -= KG) {
    const int rows = reader ? max(S * row_bytes, (int)cpc * row_bytes) : S * row_bytes;
    if (S * C::W_STAGE + rows <= C::SPACE) break;
  }
  uint8_t* sS = sW + S * DF_W_BYTES;
  uint8_t* sB = sS + S * C::S_BYTES;

  const int phases = layer ? 2 : 1;
  if (warp == 0) {
    // ------------------------------------------------ weights
    if (lane == 0) {
      const uint64_t pol = l2_evict_first_policy();
      // A stage is 128 columns wide, in blocks of 128 bytes of a row.  The issue
      // of one TMA load takes its thread ~150 clocks, so a chunk should be one
      // load, or two where it has gate and up columns: blocks are a dimension
      // of the tensor map where the columns divide into them.
      constexpr int BLK = Q4 ? 32 : 64;            // columns of a block
      constexpr int BLK_BYTES = Q4 ? 4096 : 8192;  // of a stage
      constexpr int KROWS = C::KC / (Q4 ? 8 : 1);  // rows of a chunk in the weights' array
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int ph = 0; ph < phases && ok; ++ph) {
        const int NB = ph ? p.nb2 : p.nb1, KCN = ph ? p.kc2 : p.kc1;
        const Split sp((uint32_t)n_ent * NB * KCN, G, ph ? p.least2 : p.least1);
        const CUtensorMap* mw = ph ? &maps.w2 : &maps.w1;
        const bool blocked = ph ? p.blocked2 : p.blocked1;
        uint32_t x = sp.start(cta);
        const uint32_t end = sp.start(cta + 1);
        while (x < end && ok) {
          const int item = (int)(x / KCN);
          const int k0 = (int)(x - (uint32_t)item * KCN);
          const int k1 = (int)min((uint32_t)KCN, k0 + (end - x));
          const int ei = ph ? item % n_ent : item / NB;
          const int nb = ph ? item / n_ent : item % NB;
          const int e = c.ent[ei].expert;
          // first columns of the tile's two 64-column halves: gated, the
          // gate's 64 columns and the up projection's
          const bool sg = ph == 0 && swiglu && !pair;
          const int ca = sg ? nb * 64 : nb * kDecBN;
          const int cb = sg ? p.N1 + nb * 64 : ca + 64;
          const int two = pair && ph == 0 ? 1 : 0;  // the chunks of gate and up in turn
          for (int i2 = k0 << two; i2 < k1 << two; ++i2) {
            const int kc = i2 >> two, up = (i2 & two) * p.N1;
            if (!mbar_wait(&c.empty[stage], phase ^ 1u, wc)) {
              ok = false;
              break;
            }
            uint64_t* bar = &c.full[stage];
            uint8_t* dst = sW + stage * DF_W_BYTES;
            mbar_arrive_expect_tx(bar, DF_W_BYTES);
            if (blocked) {
              tma_load_4d_hint(dst, mw, bar, 0, kc * KROWS, (ca + up) / BLK, e, pol);
              if (sg) tma_load_4d_hint(dst + DF_W_BYTES / 2, mw, bar, 0, kc * KROWS, cb / BLK, e, pol);
            } else {
#pragma unroll
              for (int i = 0; i < kDecBN / BLK; ++i)
                tma_load_3d_hint(dst + i * BLK_BYTES, mw, bar,
                                 (i < kDecBN / BLK / 2 ? ca : cb - 64) + up + i * BLK, kc * KROWS, e, pol);
            }
            ++issued;
            if (++stage == S) {
              stage = 0;
              phase ^= 1u;
            }
          }
          x += k1 - k0;
        }
      }
      // The CTA must not leave with copies in flight.  The barriers also count the
      // row loaders, which do not arrive any more after a wait ran out: then a
      // bounded while for each stage that was issued and not seen full.  A stage is
      // issued again only after its copies before were seen full by all its consumers
      // (they free nothing else), so the parity names the last ones.
      for (int m = max(0, issued - S); m < issued; ++m) {
        const uint32_t par = (uint32_t)((m / S) & 1);
        if (mbar_wait(&c.full[m % S], par, wc)) continue;
        const uint32_t a = smem_u32(&c.full[m % S]);
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(a, par) && global_timer_ns() - t0 < 1000000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp <= DF_LOADERS) {
    // ------------------------------------------------ rows
    // every loader takes every chunk: rows lw, lw + 3, ..; the last one the
    // scales too (a row costs its warp ~150 clocks to ask for)
    const int lw = warp - 1;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int ph = 0; ph < phases; ++ph) {
      const int NB = ph ? p.nb2 : p.nb1, KCN = ph ? p.kc2 : p.kc1;
      const int K = ph ? p.K2 : p.K1;
      const uint16_t* src = ph ? p.h : p.x;
      const Split sp((uint32_t)n_ent * NB * KCN, G, ph ? p.least2 : p.least1);
      uint32_t x = sp.start(cta);
      const uint32_t end = sp.start(cta + 1);
      const bool copies = ph == 0 || !reader;
      const uint16_t* scales = ph ? p.s2 : p.s1;
      const int N = ph ? p.N2 : p.N1;
      const bool sg = Q4 && ph == 0 && swiglu;
      const int ncols = sg ? 2 * N : N;  // columns of W
      const int two = pair && ph == 0 ? 1 : 0;  // a chunk of rows for the gate's and the up projection's weights
      if (ph == 1 && copies && x < end) {
        // a loader that gave up before comes here too; its lanes may have done so one
        // by one, what follows is the whole warp's (a vote per chunk costs the 4-bit
        // layer of 16 tokens 1.5 us)
        ok = __all_sync(0xffffffffu, ok);
        if (lw == 0 && ok) count_wait(p, p.barrier + kGridH, p.arrivals, c.abort_flag, lane);
        named_sync(BAR_ROWS, 32 * DF_LOADERS);
        ok = __all_sync(0xffffffffu, ok && *const_cast<volatile int*>(&c.abort_flag) == 0);
      }
      while (x < end && ok) {
        const int item = (int)(x / KCN);
        const int k0 = (int)(x - (uint32_t)item * KCN);
        const int k1 = (int)min((uint32_t)KCN, k0 + (end - x));
        const DecEntry en = c.ent[ph ? item % n_ent : item / NB];
        const int nb = ph ? item / n_ent : item % NB;
        // What a chunk costs its loader paces the stream (with the addresses
        // computed for every chunk of 4 bits 1000 clocks for 4 rows, where memory
        // takes 700), so all that does not change between chunks is worked out here.
        constexpr int RPP = 32 / PCS;                          // rows per pass of the warp
        constexpr int RSTEP = RPP * DF_LOADERS;                // of all loaders
        constexpr int PASSES = (8 * NT + RSTEP - 1) / RSTEP;
        constexpr int HELD = PASSES <= 3 ? PASSES : 0;         // rows whose addresses are kept
        const int r0 = lw * RPP + lane / PCS;
        int kk = k0 * C::KC + lane % PCS * 8;
        const uint16_t* rows[HELD > 0 ? HELD : 1];
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
          const int r = r0 + i * RSTEP;
          rows[i] = src + kk;
          if (r < en.n) rows[i] += (size_t)(ph ? en.row0 + r : c.tok[en.row0 + r]) * K;
        }
        // 4 bits: a chunk's scales, [256 / GRP rows][128 columns], by the last
        // loader: 8 columns of every second row per lane
        constexpr int GRP1 = Q4 ? GRP : 256;
        constexpr int SROWS = 256 / GRP1;
        const bool scaling = Q4 && lw == DF_LOADERS - 1;
        const int c8 = (lane & 15) * 8;
        const int scol = sg ? nb * 64 + (c8 & 63) : nb * kDecBN + c8;
        int sr = k0 * SROWS + (lane >> 4);
        const int send = scaling && scol < N ? K / GRP1 : 0;   // zeros past the end of K or of the columns
        const uint16_t* sp = scales;
        if (scaling) sp += ((size_t)en.expert * (K / GRP1) + sr) * ncols + scol + (sg && c8 >= 64 ? N : 0);
        const bool any = scaling || (copies && lw * RPP < en.n);
        for (int i2 = k0 << two; i2 < k1 << two; ++i2) {
          if (!mbar_wait(&c.empty[stage], phase ^ 1u, wc)) {
            ok = false;
            break;
          }
          const int step = (i2 & two) == two ? C::KC : 0;
          uint64_t* bar = &c.full[stage];
          if (scaling) {
            const uint32_t dst = smem_u32(sS) + (uint32_t)(stage * C::S_BYTES + (lane >> 4) * 256 + c8 * 2);
#pragma unroll
            for (int m = 0; m < SROWS / 2; ++m) {
              const bool in = sr + 2 * m < send;
              cp_async16(dst + m * 512, in ? sp + (size_t)(2 * m) * ncols : scales, in ? 16u : 0u);
            }
            sr += SROWS;
            sp += (size_t)SROWS * ncols;
          }
          if (copies) {
            const uint32_t dst = smem_u32(sB) + (uint32_t)(stage * row_bytes + r0 * C::PITCH + lane % PCS * 16);
            const uint32_t n = kk < K ? 16u : 0u;              // zeros past the end of K
            if constexpr (HELD > 0) {
#pragma unroll
              for (int i = 0; i < HELD; ++i) {
                if (r0 + i * RSTEP < en.n)
                  cp_async16(dst + i * (RSTEP * C::PITCH), kk < K ? rows[i] : src, n);
                rows[i] += step;
              }
            } else {
              const uint16_t* s = src + (kk < K ? kk : 0);
#pragma unroll 4
              for (int r = r0; r < en.n; r += RSTEP) {
                const int row = ph ? en.row0 + r : c.tok[en.row0 + r];
                cp_async16(dst + (uint32_t)((r - r0) * C::PITCH), s + (size_t)row * K, n);
              }
            }
            kk += step;
          }
          if (any)
            cp_async_arrive(bar);
          else if (lane == 0)
            mbar_arrive_n(bar, 32);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        x += k1 - k0;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ------------------------------------------------ multiply, finish items
    const int cw = warp - 1 - DF_LOADERS;
    const int wn = cw & (DF_WN - 1);
    const int kg = cw / DF_WN;
    const int g = lane >> 2, t = lane & 3;
    const int ctid = tid - 32 * (1 + DF_LOADERS);
    const int ftid = ctid & (DF_FIN - 1);  // among the group's threads
    // This group's next chunk: its number q among the CTA's chunks (q mod KG =
    // kg), its stage and that stage's parity.  A wait tells the phases of a
    // barrier apart by parity only, so whoever waits for a stage's phase must
    // know the one before it to be over; groups and copies in flight overtake
    // each other, so every stage belongs to one group (S mod KG = 0).
    // After a wait that ran out the consumers go through all their barriers and
    // counters as before, multiplying whatever the stages hold (a branch around the
    // products would need the warp's lanes to agree: a vote per chunk, 1.5 us of the
    // 4-bit layer of 16 tokens): nobody else hangs, and the status word says that the
    // result is void.  They free no stage any more: copies into it may still be on
    // their way, and new ones would leave its barrier a phase behind what everybody
    // takes it for.
    bool ok = true;
    uint32_t q = (uint32_t)kg, qi = 0, q2 = 0;
    int stage = kg;
    uint32_t par = 0;
    uint32_t n_items = 0;  // items of this CTA so far: number i is written by group i mod KG
    if (layer)
      for (int i = ctid; i < n_ent; i += CTHREADS)
        for (int r = 0; r < c.ent[i].n; ++r) c.row_entry[c.ent[i].row0 + r] = (uint16_t)i;

    // this lane's place in a weight stage (tile columns 32 wn + ..) and in
    // the rows
    uint32_t wofs[2], bofs[2], bl, sofs = 0;
    if constexpr (Q4) {
      // word row 2t + i of step i (4i + t with 32-row groups, whose rows must
      // not mix): lane t holds 8 rows of K
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t row = GRP == 32 ? (uint32_t)(4 * i + t) : (uint32_t)(2 * t + i);
        wofs[i] = (uint32_t)wn * 4096 + row * 128 + (((uint32_t)g ^ row) * 16);
        bofs[i] = row * 16;
      }
      bl = (uint32_t)(g * C::PITCH);
      sofs = (uint32_t)(wn * 32 + 4 * g) * 2;
    } else {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint32_t ch = (uint32_t)((wn & 1) * 4 + m * 2) + (uint32_t)((lane >> 3) & 1);
        const uint32_t row = (uint32_t)((lane >> 4) * 8 + (lane & 7));
        wofs[m] = (uint32_t)(wn >> 1) * 8192 + row * 128 + ((ch ^ (row & 7)) * 16);
        bofs[m] = 0;
      }
      bl = (uint32_t)((lane & 7) * C::PITCH + (lane >> 3) * 16);
    }
    // element (m, n, r) of this lane: tile column and row of the entry
    auto col_of = [&](int m, int r) {
      return 32 * wn + (Q4 ? 4 * g + 2 * m + (r >> 1) : 16 * m + g + 8 * (r >> 1));
    };
    auto row_of = [&](int n, int r) { return n * 8 + 2 * t + (r & 1); };

    for (int ph = 0; ph < phases; ++ph) {
      const int NB = ph ? p.nb2 : p.nb1, KCN = ph ? p.kc2 : p.kc1;
      const int N = ph ? p.N2 : p.N1;
      const Split sp((uint32_t)n_ent * NB * KCN, G, ph ? p.least2 : p.least1);
      uint32_t x = sp.start(cta);
      const uint32_t end = sp.start(cta + 1);
      const bool cached = ph == 1 && reader;

      if (cached && x < end) {
        // ---- this CTA's part of h, chunk after chunk, once every CTA's is
        // there: whole items as they are, shared ones summed from their tiles.
        // A thread's pieces are worked out before the wait, and their loads
        // are in flight together.
        constexpr int UN = 2;
        q2 = qi;
        const Split s1((uint32_t)n_ent * p.nb1 * p.kc1, G, p.least1);
        const int total = (int)(end - x) * max_rows * PCS;
        for (int i0 = ctid; i0 < total || i0 == ctid; i0 += UN * CTHREADS) {
          const float* part[UN];     // first tile of a shared item's piece
          const uint16_t* whole[UN]; // or the piece of h
          int more[UN];
#pragma unroll
          for (int u = 0; u < UN; ++u) {
            const int i = i0 + u * CTHREADS;
            part[u] = nullptr;
            whole[u] = nullptr;
            more[u] = -1;            // nothing to store
            if (i < total) {
              const int j = i % PCS, rc = i / PCS;
              const int r = rc % max_rows;
              const uint32_t xc = x + (uint32_t)(rc / max_rows);
              const int item = (int)(xc / KCN);
              const int ei = item % n_ent;
              const DecEntry en = c.ent[ei];
              const int kk = (int)(xc - (uint32_t)item * KCN) * C::KC + j * 8;
              if (r < en.n) {
                more[u] = 0;         // zeros past the end of K
                if (kk < p.K2) {
                  const uint32_t f = (uint32_t)(ei * p.nb1 + (kk >> g1.sh)) * p.kc1;
                  const int o0 = s1.owner(f);
                  more[u] = s1.owner(f + p.kc1 - 1) - o0;
                  if (more[u] == 0)
                    whole[u] = p.h + (size_t)(en.row0 + r) * p.K2 + kk;
                  else
                    part[u] = p.parts + (size_t)(o0 * 2 + 1) * g1.tile + r * kDecBN + (kk & ((1 << g1.sh) - 1));
                }
              }
            }
          }
          if (i0 == ctid) {
            if (cw == 0) count_wait(p, p.barrier + kGridH, p.arrivals, c.abort_flag, lane);
            named_sync(BAR_CONS, CTHREADS);
          }
          // the same tile of all pieces (their halves) at once
          float4 z[2 * UN], g2[2 * UN];
          uint2 v[2 * UN];
          const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
          int most = 0;
#pragma unroll
          for (int i = 0; i < 2 * UN; ++i) {
            const int u = i / 2, h = i % 2;
            most = max(most, more[u]);
            v[i] = make_uint2(0, 0);
            z[i] = g2[i] = none;
            if (whole[u]) v[i] = __ldcg(reinterpret_cast<const uint2*>(whole[u]) + h);
            if (part[u]) {
              z[i] = __ldcg(reinterpret_cast<const float4*>(part[u]) + h);
              if (swiglu) g2[i] = __ldcg(reinterpret_cast<const float4*>(part[u] + g1.up) + h);
            }
          }
#pragma unroll 1
          for (int o = 1; o <= most; ++o) {
            float4 z1[2 * UN], u1[2 * UN];
#pragma unroll
            for (int i = 0; i < 2 * UN; ++i) {
              const int u = i / 2, h = i % 2;
              z1[i] = u1[i] = none;
              if (o <= more[u]) {
                const float* t = part[u] + (size_t)(2 * o - 1) * g1.tile;
                z1[i] = __ldcg(reinterpret_cast<const float4*>(t) + h);
                if (swiglu) u1[i] = __ldcg(reinterpret_cast<const float4*>(t + g1.up) + h);
              }
            }
#pragma unroll
            for (int i = 0; i < 2 * UN; ++i) {
              add4(z[i], z1[i]);
              add4(g2[i], u1[i]);
            }
          }
#pragma unroll
          for (int i = 0; i < 2 * UN; ++i) {
            const int u = i / 2, h = i % 2, piece = i0 + u * CTHREADS;
            if (more[u] > 0) v[i] = activated(p.act, z[i], g2[i]);
            if (more[u] >= 0)
              sts64(smem_u32(sB) + (uint32_t)(piece / PCS) * C::PITCH + (uint32_t)(piece % PCS) * 16 + h * 8, v[i].x,
                    v[i].y);
          }
        }
        named_sync(BAR_CONS, CTHREADS);
      }

      while (x < end) {
        const int item = (int)(x / KCN);
        const int nb = ph ? item / n_ent : item % NB;
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

        const uint32_t chunks = (uint32_t)(k1 - k0) << (pair && ph == 0 ? 1 : 0);
        for (; q < qi + chunks; q += KG) {
          ok = ok && mbar_wait(&c.full[stage], par, wc);
          __syncwarp();
          const uint32_t w0 = smem_u32(sW + stage * DF_W_BYTES);
          const uint32_t b0 = smem_u32(sB) + bl + (cached ? q - q2 : (uint32_t)stage) * (uint32_t)row_bytes;
          const auto chunk = [&](auto nta) {
            constexpr int NTA = decltype(nta)::value;
            if constexpr (Q4)
              chunk_q4<NT, NTA, GRP>(acc, w0, wofs, b0, bofs, smem_u32(sS + stage * C::S_BYTES) + sofs);
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
          if (ok && lane == 0) mbar_arrive(&c.empty[stage]);
          if ((stage += KG) >= S) {
            stage -= S;
            par ^= 1u;
          }
        }
        qi += chunks;
        x += (uint32_t)(k1 - k0);
        if constexpr (Q4) {  // the codes were taken as (c - 8) / 64
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[m][n][r] *= 64.f;
        }

        // ---- the groups in turn sum both parts and write the item out; the
        // other hands over and goes on.  It hands over again only after an item
        // of its own, for which the first has come to a barrier after this
        // reading.
        const int writer = (int)(n_items % KG);
        float* mine_red = sRed + kg * C::RED_GROUP;
        ++n_items;
        if (kg != writer) {
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int r = 0; r < 4; ++r) mine_red[((m * NT + n) * 4 + r) * DF_FIN + ftid] = acc[m][n][r];
          named_arrive(BAR_ITEM + writer, CTHREADS);
          continue;
        }
        named_sync(BAR_ITEM + writer, CTHREADS);
        const int bar_fin = BAR_FIN + kg;
        float* tile_s = sRed + kg * C::RED_GROUP;
        float* red = sRed + (1 - kg) * C::RED_GROUP;
        // The item's sums as rows of 128 columns in this group's own space (it
        // is free while the group writes), so that only real rows cost
        // anything and every access to memory is 4 columns wide.
        const auto lay_down = [&](float* to, const float (&v)[2][NT][4]) {
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (row_of(n, r) < en.n) to[row_of(n, r) * kDecBN + col_of(m, r)] = v[m][n][r];
        };
        if (pair && ph == 0) {
          // the other's sums are of other columns: as rows too, in its space, once
          // everybody has taken his own
          float other[2][NT][4];
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int r = 0; r < 4; ++r) other[m][n][r] = red[((m * NT + n) * 4 + r) * DF_FIN + ftid];
          named_sync(bar_fin, DF_FIN);
          lay_down(red, other);
        } else {
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[m][n][r] += red[((m * NT + n) * 4 + r) * DF_FIN + ftid];
        }
        lay_down(tile_s, acc);
        named_sync(bar_fin, DF_FIN);
        // group 0 has summed the gate, group 1 the up projection
        const float* tile_z = pair && ph == 0 ? sRed : tile_s;
        const float* tile_u = pair ? sRed + C::RED_GROUP : tile_s + 64;
        // the first product's shared items by their first CTA, where it has no
        // readers and few rows: its own sums stay here until the loop ends
        const bool by_first = NT < 4 && ph == 0 && !reader;
        if (by_first && k0 == 0 && k1 != KCN) continue;
        if (k0 != 0 || k1 != KCN) {
          // a shared item: this CTA's partial tile, slot 0 if the item began in
          // an earlier CTA, else slot 1
          float* mine = (ph ? p.parts2 : p.parts) + (size_t)(cta * 2 + (k0 > 0 ? 0 : 1)) *
                                                        (ph ? (size_t)p.row_cap * kDecBN : g1.tile);
          for (int i = ftid * 4; i < en.n * kDecBN; i += DF_FIN * 4) {
            *reinterpret_cast<float4*>(mine + i) = *reinterpret_cast<const float4*>(tile_z + i);
            if (pair && ph == 0)
              *reinterpret_cast<float4*>(mine + g1.up + i) = *reinterpret_cast<const float4*>(tile_u + i);
          }
        } else if (ph == 1) {  // whole items of the second product stay in fp32 for the combine
          for (int i = ftid * 4; i < en.n * kDecBN; i += DF_FIN * 4) {
            const int col = nb * kDecBN + (i & (kDecBN - 1));
            if (col < N)
              *reinterpret_cast<float4*>(p.yfull + (size_t)(en.row0 + i / kDecBN) * N + col) =
                  *reinterpret_cast<const float4*>(tile_s + i);
          }
        } else {
          write_item(p, g1, en, nb, ftid, tile_z, tile_u);
        }
        named_sync(bar_fin, DF_FIN);  // before this space is handed over again
        if (by_first && k0 != 0 && ftid == 0)
          red_release(p.item_counts + sp.owner((uint32_t)item * KCN), 1u);
      }

      // ---- every group has written its items: now what they share with other
      // CTAs, by all consumer threads (more loads in flight, and the multiplying
      // loop's registers are free: a spill costs this kernel a trip to memory
      // behind the weights, as shared memory leaves no L1 to speak of)
      named_sync(BAR_CONS, CTHREADS);
      const int gw = cw * (int)G + cta, warps = C::CONSUMERS * (int)G;
      if (ph == 0) {
        if (!reader && NT >= 4) {
          // many rows: by all CTAs, after a grid barrier
          if (ctid == 0) red_release(p.barrier + kGridTiles, 1u);
          if (cw == 0) count_wait(p, p.barrier + kGridTiles, p.arrivals, c.abort_flag, lane);
          named_sync(BAR_CONS, CTHREADS);
          finish_all(p, g1, c, sp, gw, warps, lane);
        } else if (!reader) {
          // few rows: the item that goes on in later CTAs, once they have counted
          // in.  They begin with it, so they have done so long ago.
          const uint32_t i0 = end / KCN * KCN;
          if (i0 != end && i0 >= sp.start(cta) && end > sp.start(cta)) {
            const int more = sp.owner(i0 + KCN - 1) - cta;
            if (cw == 0) count_wait(p, p.item_counts + cta, (uint32_t)more, c.abort_flag, lane);
            named_sync(BAR_CONS, CTHREADS);
            const int it = (int)(end / KCN);
            const float* own = sRed + (n_items - 1) % KG * C::RED_GROUP;
            finish_item<CTHREADS>(p, g1, c.ent[it / NB], it % NB, pair ? sRed : own,
                                  pair ? sRed + C::RED_GROUP : own + 64, cta, more, ctid);
          }
        }
        if (layer) {  // this CTA's h is there
          if (!reader) named_sync(BAR_CONS, CTHREADS);
          if (ctid == 0) red_release(p.barrier + kGridH, 1u);
        }
      } else {
        if (ctid == 0) red_release(p.barrier + kGridY, 1u);
        combine<(Q4 || NT > 2 ? 1 : 3)>(p, c, sp, cw, gw, warps, CTHREADS, lane);
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
  cfg.dynamicSmemBytes = DF_SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  set_pdl_attr(attr[1]);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
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
                              cudaFuncAttributeMaxDynamicSharedMemorySize, DF_SMEM);
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
