// decode_ffn.cu -- second kernel of the decode operators: the expert products
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
#include "decode_internal.h"
#include "tc_common.cuh"

namespace moe {
namespace {

constexpr int DF_LOADERS = 3;     // 12 warps in all, 3 to a scheduler: 168 registers each
constexpr int DF_CONSUMERS = 8;  // 4 across columns x 2 across K
constexpr int DF_THREADS = 32 * (1 + DF_LOADERS + DF_CONSUMERS);
constexpr int DF_WN = 4;         // consumer warps across the columns
constexpr int DF_FIN = 32 * DF_WN;  // threads that write an item out
constexpr int DF_W_BYTES = 16384;
constexpr int DF_MAX_WSTAGES = 12;
constexpr int DF_MAX_BSTAGES = 8;
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
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// codes i and i + 4 of a word (rows i and i + 4 of its 8) as a bf16 pair
// c - 8, exactly: 0x4300 | c is 128 + c.
template <int I>
__device__ __forceinline__ uint32_t q4_pair(uint32_t v) {
  uint32_t p;
  asm("lop3.b32 %0, %1, 0x000F000F, 0x43004300, 0xEA;" : "=r"(p) : "r"(v >> (4 * I)));
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&p),
                                   __floats2bfloat162_rn(136.f, 136.f));
  return *reinterpret_cast<const uint32_t*>(&d);
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

template <bool Q4, int NT>
struct Cfg {
  static constexpr int KC = Q4 ? kDecKC4 : kDecKC16;   // K rows of a chunk
  static constexpr int S_BYTES = Q4 ? 8 * 2 * 128 : 0; // scales: up to 8 groups x 2 boxes x 128 B
  static constexpr int W_STAGE = DF_W_BYTES + S_BYTES;
  static constexpr int B_TILE = KC * 16;               // 8 rows x KC bf16
  static constexpr int B_STAGE = B_TILE * NT;
  static constexpr int B_STAGES = NT <= 2 ? 8 : Q4 && NT == 8 ? 3 : 4;
  static constexpr int RED = DF_WN * 2 * NT * 4 * 32 * 4;  // cross-K sums
  static constexpr int CTRL = 8 * 1024;
  static constexpr int FIT = (DF_SMEM_LIMIT - 1024 - CTRL - RED - B_STAGE * B_STAGES) / W_STAGE;
  static constexpr int W_STAGES = FIT < DF_MAX_WSTAGES ? FIT : DF_MAX_WSTAGES;
  static constexpr size_t SMEM =
      1024 + (size_t)W_STAGES * W_STAGE + (size_t)B_STAGES * B_STAGE + RED + CTRL;
  static_assert(W_STAGES >= 4, "weight ring");
  // a loader that has filled chunk q - DF_LOADERS knows chunk
  // q - DF_LOADERS - B_STAGES to be consumed; its wait for q's stage tells
  // phases apart by parity only if q - 2 B_STAGES is consumed too
  static_assert(B_STAGES >= DF_LOADERS && B_STAGES <= DF_MAX_BSTAGES, "row ring");
  static_assert(SMEM <= DF_SMEM_LIMIT, "shared memory");
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
};
static_assert(sizeof(Ctrl) <= 8 * 1024, "control area");

// One product's chunks, in item order, dealt to the first G = min(CTAs, total)
// CTAs: CTA c < G takes chunks [total c / G, total (c + 1) / G), at least one.
struct Split {
  long long total;
  int G;
  __device__ __forceinline__ Split(long long n, int ctas)
      : total(n), G((int)min((long long)ctas, n)) {}
  __device__ __forceinline__ long long start(int c) const { return c < G ? total * c / G : total; }
  // the CTA that holds chunk x: the largest c with total c / G < x + 1
  __device__ __forceinline__ int owner(long long x) const {
    return (int)(((x + 1) * G - 1) / total);
  }
};

template <bool Q4, int NT>
__global__ void __launch_bounds__(DF_THREADS, 1)
    decode_ffn_kernel(const __grid_constant__ DecFfnMaps maps, const DecFfnArgs p) {
  using C = Cfg<Q4, NT>;
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
  const int G = gridDim.x;
  const bool layer = p.act != kDecNone;
  const bool swiglu = p.act == kDecSwiGLU;

  if (tid == 0) {
    for (int i = 0; i < C::W_STAGES; ++i) {
      mbar_init(&c.wfull[i], 1);
      mbar_init(&c.wempty[i], DF_CONSUMERS);
    }
    for (int i = 0; i < C::B_STAGES; ++i) {
      mbar_init(&c.bfull[i], 1);
      mbar_init(&c.bempty[i], DF_CONSUMERS);
    }
    c.abort_flag = 0;
    fence_mbar_init();
  }
  pdl_launch_dependents();
  pdl_wait();
  // the first kernel's list
  if (tid == 32) c.n_entries = min(__ldcg(p.ctrl + kDecCountOffset / 4), p.max_entries);
  for (int i = tid; i < p.max_entries; i += DF_THREADS) {
    const int4 v = __ldcg(reinterpret_cast<const int4*>(p.entries) + i);
    c.ent[i] = DecEntry{v.x, v.y, v.z, v.w};
  }
  __syncthreads();
  const int n_ent = c.n_entries;
  const WaitCtl wc{&c.abort_flag, p.status, p.wait_limit_ns};

  if (n_ent == 0) {  // every assignment dropped: y = 0 (grouped products: nothing to write)
    if (layer) {
      const size_t n = (size_t)p.T * p.N2;  // N2 = H, a multiple of 8
      for (size_t i = ((size_t)cta * DF_THREADS + tid) * 8; i < n; i += (size_t)G * DF_THREADS * 8)
        *reinterpret_cast<uint4*>(p.y + i) = make_uint4(0, 0, 0, 0);
    }
    return;
  }

  const int phases = layer ? 2 : 1;
  if (warp == 0) {
    // ------------------------------------------------ weight producer
    if (lane == 0) {
      tma_prefetch_desc(&maps.w1);
      if (Q4) tma_prefetch_desc(&maps.s1);
      if (layer) {
        tma_prefetch_desc(&maps.w2);
        if (Q4) tma_prefetch_desc(&maps.s2);
      }
      const uint64_t pol = l2_evict_first_policy();
      const int srows = Q4 ? kDecKC4 / p.group : 0;  // scale rows of a chunk
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int ph = 0; ph < phases && ok; ++ph) {
        const int NB = ph ? p.nb2 : p.nb1, KCN = ph ? p.kc2 : p.kc1;
        const Split sp((long long)n_ent * NB * KCN, G);
        const CUtensorMap* mw = ph ? &maps.w2 : &maps.w1;
        const CUtensorMap* ms = ph ? &maps.s2 : &maps.s1;
        long long x = sp.start(cta);
        const long long end = sp.start(cta + 1);
        while (x < end && ok) {
          const int item = (int)(x / KCN);
          const int k0 = (int)(x - (long long)item * KCN);
          const int k1 = (int)min((long long)KCN, k0 + (end - x));
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
  } else if (warp <= DF_LOADERS) {
    // ------------------------------------------------ row loaders
    const int lw = warp - 1;
    const bool g32 = Q4 && p.group == 32;
    uint32_t q = 0;  // chunks of this CTA so far (both products)
    bool ok = true;
    for (int ph = 0; ph < phases && ok; ++ph) {
      const int NB = ph ? p.nb2 : p.nb1, KCN = ph ? p.kc2 : p.kc1;
      const int K = ph ? p.K2 : p.K1;
      const Split sp((long long)n_ent * NB * KCN, G);
      long long x = sp.start(cta);
      const long long end = sp.start(cta + 1);
      if (ph == 1 && x < end) {  // every CTA's h must be there
        int got = 1;
        if (lane == 0) {
          const uint64_t t0 = global_timer_ns();
          for (uint32_t it = 1; ld_acquire(p.barrier) < (unsigned)G; ++it) {
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
        const int k0 = (int)(x - (long long)item * KCN);
        const int k1 = (int)min((long long)KCN, k0 + (end - x));
        const DecEntry en = c.ent[ph ? item % n_ent : item / NB];
        // source rows of this lane's two row numbers, lane and lane + 32
        const uint16_t* src = ph ? p.h : p.x;
        int r0 = en.row0 + lane, r1 = en.row0 + lane + 32;
        if (layer && ph == 0) {
          const int tk = p.T * p.k;
          if (lane < en.n) r0 = min(max(__ldg(p.perm + r0), 0), tk - 1) / p.k;
          if (lane + 32 < en.n) r1 = min(max(__ldg(p.perm + r1), 0), tk - 1) / p.k;
        }
        for (int kc = k0; kc < k1; ++kc, ++q) {
          if (q % DF_LOADERS != (uint32_t)lw) continue;
          const uint32_t bs = q % C::B_STAGES;
          const uint32_t par = (q / C::B_STAGES) & 1;
          if (!mbar_wait(&c.bempty[bs], par ^ 1u, wc)) {
            ok = false;
            break;
          }
          const uint32_t dst0 = smem_u32(sB + bs * C::B_STAGE);
          constexpr int PCS = C::KC / 8;       // 16-byte pieces of a row
          constexpr int RPP = 32 / PCS;        // rows per pass of the warp
          constexpr int UN = NT * 8 / RPP < 8 ? NT * 8 / RPP : 8;  // passes in flight together
          const int j = lane % PCS;
          const int kk = kc * C::KC + j * 8;
          for (int rb = 0; rb < en.n; rb += RPP * UN) {
            uint4 v[UN];
#pragma unroll
            for (int u = 0; u < UN; ++u) {
              const int r = rb + u * RPP + lane / PCS;
              const int sr = __shfl_sync(0xffffffffu, (rb + u * RPP) < 32 ? r0 : r1, r & 31);
              v[u] = make_uint4(0, 0, 0, 0);
              if (r < en.n && kk < K)
                v[u] = __ldcg(reinterpret_cast<const uint4*>(src + (size_t)sr * K + kk));
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
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.bfull[bs]);
        }
        x += k1 - k0;
      }
    }
  } else {
    // ------------------------------------------------ multiply, finish items
    const int cw = warp - 1 - DF_LOADERS;
    const int wn = cw & (DF_WN - 1);
    const int kg = cw / DF_WN;
    const int g = lane >> 2, t = lane & 3;
    const int ctid = tid - 32 * (1 + DF_LOADERS);  // 0..255; < DF_FIN: kg = 0
    int ws = 0, bs = 0;
    uint32_t wpar = 0, bpar = 0;
    bool ok = true;

    for (int ph = 0; ph < phases && ok; ++ph) {
      const int NB = ph ? p.nb2 : p.nb1, KCN = ph ? p.kc2 : p.kc1;
      const int N = ph ? p.N2 : p.N1;
      const Split sp((long long)n_ent * NB * KCN, G);
      const bool sg = ph == 0 && swiglu;
      long long x = sp.start(cta);
      const long long end = sp.start(cta + 1);

      // tile column of m16 tile m, row g / row g + 8, and its place in a stage
      //   plain:  columns 32 wn + 16 m + ..;  gated: tile 0 gate, tile 1 up,
      //   both columns 16 wn + .. of their 64-column half
      int tcol[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) tcol[m] = sg ? m * 64 + 16 * wn : 32 * wn + 16 * m;
      // bf16: ldmatrix rows of this lane; 4-bit: word offsets of this lane
      uint32_t wofs[2][2];
      uint32_t sofs[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        sofs[m] = 0;
        if constexpr (Q4) {
          const uint32_t box = (uint32_t)(tcol[m] >> 5);
          const uint32_t ch = (uint32_t)((tcol[m] & 31) >> 2) + (uint32_t)(g >> 1);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t row = p.group == 32 ? (uint32_t)(4 * i + t) : (uint32_t)(2 * t + i);
            wofs[m][i] = box * 4096 + row * 128 + ((ch ^ row) * 16) + (uint32_t)(g & 1) * 8;
          }
          sofs[m] = (uint32_t)(tcol[m] >> 6) * (uint32_t)(kDecKC4 / p.group) * 128 +
                    (uint32_t)((tcol[m] & 63) + 2 * g) * 2;
        } else {
          const uint32_t box = (uint32_t)(tcol[m] >> 6);
          const uint32_t ch = (uint32_t)((tcol[m] & 63) >> 3) + (uint32_t)((lane >> 3) & 1);
          const uint32_t row = (uint32_t)((lane >> 4) * 8 + (lane & 7));
          wofs[m][0] = box * 8192 + row * 128 + ((ch ^ (row & 7)) * 16);
          wofs[m][1] = 0;
        }
      }

      int cur_nb = -1;  // second product: column block of the items done so far
      while (ok) {
        const bool more = x < end;
        const int item = more ? (int)(x / KCN) : 0;
        const int nb = more ? (ph ? item / n_ent : item % NB) : -1;
        if (ph == 1 && cur_nb >= 0 && nb != cur_nb) {
          // ---- this CTA's part of column block cur_nb is written: count in,
          // and combine the block if it is the last part
          __threadfence();
          named_sync(BAR_CONS, 32 * DF_CONSUMERS);
          const long long b0 = (long long)cur_nb * n_ent * KCN;
          if (ctid == 0) {
            const int parts =
                sp.owner(b0 + (long long)n_ent * KCN - 1) - sp.owner(b0) + 1;
            c.last = atomicAdd(p.col_tickets + cur_nb, 1u) == (unsigned)(parts - 1);
          }
          named_sync(BAR_CONS, 32 * DF_CONSUMERS);
          if (c.last) {
            __threadfence();
            for (int i = ctid; i < n_ent; i += 32 * DF_CONSUMERS) {
              const long long i0 = b0 + (long long)i * KCN;
              c.owner[i] = make_int2(sp.owner(i0), sp.owner(i0 + KCN - 1));
              const DecEntry en = c.ent[i];
              for (int r = 0; r < en.n; ++r) c.row_entry[en.row0 + r] = (uint16_t)i;
            }
            named_sync(BAR_CONS, 32 * DF_CONSUMERS);
            const int col0 = cur_nb * kDecBN;
            for (int i = ctid; i < p.T * (kDecBN / 2); i += 32 * DF_CONSUMERS) {
              const int tok = i / (kDecBN / 2);
              const int cl = (i % (kDecBN / 2)) * 2;
              if (col0 + cl >= N) continue;
              float y0 = 0.f, y1 = 0.f;
              for (int j = 0; j < p.k; ++j) {
                const int row = __ldcg(p.slot + tok * p.k + j);
                if (row < 0) continue;
                const float w = __ldcg(p.gate + tok * p.k + j);
                const int ei = c.row_entry[row];
                const int2 own = c.owner[ei];
                float2 v;
                if (own.x == own.y) {
                  v = __ldcg(reinterpret_cast<const float2*>(p.yfull + (size_t)row * N + col0 + cl));
                } else {
                  v = make_float2(0.f, 0.f);
                  const int rr = row - c.ent[ei].row0;
                  for (int o = own.x; o <= own.y; ++o) {
                    const float2 u = __ldcg(reinterpret_cast<const float2*>(
                        p.parts + ((size_t)(o * 2 + (o == own.x ? 1 : 0)) * p.row_cap + rr) * kDecBN +
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
        const int k0 = (int)(x - (long long)item * KCN);
        const int k1 = (int)min((long long)KCN, k0 + (end - x));
        const DecEntry en = c.ent[ph ? item % n_ent : item / NB];

        float acc[2][NT][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[m][n][r] = 0.f;

        for (int kc = k0; kc < k1; ++kc) {
          if (!mbar_wait(&c.wfull[ws], wpar, wc) || !mbar_wait(&c.bfull[bs], bpar, wc)) {
            ok = false;
            break;
          }
          const uint32_t w0 = smem_u32(sW + ws * DF_W_BYTES);
          const uint32_t b0 = smem_u32(sB + bs * C::B_STAGE) + (uint32_t)(t * 128 + ((g ^ (2 * t)) * 16));
          if constexpr (Q4) {
            const uint32_t s0 = smem_u32(sS + ws * C::S_BYTES);
            float part[2][NT][4];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) part[m][n][r] = 0.f;
#pragma unroll
            for (int bb = 0; bb < 2; ++bb) {  // 64 rows of K
              const uint32_t blk = (uint32_t)(kg * 2 + bb);
#pragma unroll
              for (int i = 0; i < 2; ++i) {   // 32 of them
                uint32_t a[2][8];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                  uint32_t va, vb;
                  lds64(w0 + blk * 1024 + wofs[m][i], va, vb);
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
                for (int n = 0; n < NT; ++n) {
                  if (n * 8 >= en.n) break;
                  uint32_t b[4];
                  lds128(b0 + n * C::B_TILE + blk * 1024 + i * 512, b);
#pragma unroll
                  for (int m = 0; m < 2; ++m) {
                    mma_bf16(part[m][n], a[m][0], a[m][1], a[m][2], a[m][3], b[0], b[1]);
                    mma_bf16(part[m][n], a[m][4], a[m][5], a[m][6], a[m][7], b[2], b[3]);
                  }
                }
                // end of a scale group: every 32, 64 or 128 rows
                const bool flush = i == 1 ? (bb == 1 || p.group <= 64) : p.group == 32;
                if (flush) {
                  const uint32_t grp = (blk * 64 + (uint32_t)i * 32) / (uint32_t)p.group;
#pragma unroll
                  for (int m = 0; m < 2; ++m) {
                    const uint32_t sv = lds32(s0 + grp * 128 + sofs[m]);
                    const float sa = bf16_lo(sv), sb = bf16_hi(sv);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                      if (n * 8 >= en.n) break;
                      acc[m][n][0] = fmaf(sa, part[m][n][0], acc[m][n][0]);
                      acc[m][n][1] = fmaf(sa, part[m][n][1], acc[m][n][1]);
                      acc[m][n][2] = fmaf(sb, part[m][n][2], acc[m][n][2]);
                      acc[m][n][3] = fmaf(sb, part[m][n][3], acc[m][n][3]);
#pragma unroll
                      for (int r = 0; r < 4; ++r) part[m][n][r] = 0.f;
                    }
                  }
                }
              }
            }
          } else {
            const uint32_t blk = (uint32_t)kg;  // 32 rows of K
            uint32_t a[2][2][4];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int hf = 0; hf < 2; ++hf)
                ldsm_x4_t(w0 + (blk * 32 + hf * 16) * 128 + wofs[m][0], a[m][hf]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (n * 8 >= en.n) break;
              uint32_t b[4];
              lds128(b0 + n * C::B_TILE + blk * 512, b);
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                mma_bf16(acc[m][n], a[m][0][0], a[m][0][1], a[m][0][2], a[m][0][3], b[0], b[1]);
                mma_bf16(acc[m][n], a[m][1][0], a[m][1][1], a[m][1][2], a[m][1][3], b[2], b[3]);
              }
            }
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&c.wempty[ws]);
            mbar_arrive(&c.bempty[bs]);
          }
          if (++ws == C::W_STAGES) {
            ws = 0;
            wpar ^= 1u;
          }
          if (++bs == C::B_STAGES) {
            bs = 0;
            bpar ^= 1u;
          }
        }
        // ---- sum of the two K halves: the second half's warps hand over.  A
        // wait that ran out in any warp ends the work of all of them here.
        if (named_any(BAR_CONS, 32 * DF_CONSUMERS, !ok)) {
          ok = false;
          break;
        }
        if (kg == 1) {
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int r = 0; r < 4; ++r)
                sRed[((m * NT + n) * 4 + r) * DF_FIN + wn * 32 + lane] = acc[m][n][r];
        }
        named_sync(BAR_CONS, 32 * DF_CONSUMERS);
        if (kg == 0) {
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int r = 0; r < 4; ++r)
                acc[m][n][r] += sRed[((m * NT + n) * 4 + r) * DF_FIN + wn * 32 + lane];

          // element (m, n, r) of this lane: tile column and row of the entry
          auto col_of = [&](int m, int r) {
            return tcol[m] + (Q4 ? 2 * g + (r >> 1) : g + 8 * (r >> 1));
          };
          auto row_of = [&](int n, int r) { return n * 8 + 2 * t + (r & 1); };

          const bool whole = k0 == 0 && k1 == KCN;
          bool write = whole;
          if (!whole) {
            // partial tile of this CTA: slot 0 if the item began in an
            // earlier CTA, else slot 1
            float* mine = p.parts + (size_t)(cta * 2 + (k0 > 0 ? 0 : 1)) * p.row_cap * kDecBN;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  if (row_of(n, r) < en.n) mine[row_of(n, r) * kDecBN + col_of(m, r)] = acc[m][n][r];
            if (ph == 0) {
              const long long i0 = (long long)item * KCN;
              __threadfence();
              named_sync(BAR_FIN, DF_FIN);
              int c0 = 0, c1 = 0;
              if (ctid == 0) {
                c0 = sp.owner(i0);
                c1 = sp.owner(i0 + KCN - 1);
                c.last = atomicAdd(p.item_tickets + c0, 1u) == (unsigned)(c1 - c0)
                             ? (c0 << 16 | c1) + 1
                             : 0;
              }
              named_sync(BAR_FIN, DF_FIN);
              if (c.last) {
                c0 = (c.last - 1) >> 16;
                c1 = (c.last - 1) & 0xFFFF;
                __threadfence();
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
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                if (sg && m == 1) break;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                  for (int r = 0; r < 4; ++r) {
                    const int col = nb * (sg ? 64 : kDecBN) + col_of(m, r);
                    if (row_of(n, r) < en.n && col < N) {
                      float v = acc[m][n][r];
                      if (sg)
                        v = dec_silu(v) * acc[1][n][r];
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
      }
      if (ph == 0 && layer) {
        // this CTA's h is written: arrive at the grid barrier
        __threadfence();
        named_sync(BAR_CONS, 32 * DF_CONSUMERS);
        if (ctid == 0) red_release(p.barrier, 1u);
      }
    }
  }
}

template <bool Q4, int NT>
cudaError_t ffn_launch(const DecFfnMaps& m, const DecFfnArgs& a, int ctas, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3(DF_THREADS, 1, 1);
  cfg.dynamicSmemBytes = Cfg<Q4, NT>::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_ffn_kernel<Q4, NT>, m, a);
}

template <bool Q4, int NT>
cudaError_t ffn_attr() {
  return cudaFuncSetAttribute(decode_ffn_kernel<Q4, NT>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<Q4, NT>::SMEM);
}

template <bool Q4>
cudaError_t ffn_rows(const DecFfnMaps& m, const DecFfnArgs& a, int ctas, cudaStream_t st) {
  if (a.row_cap <= 8) return ffn_launch<Q4, 1>(m, a, ctas, st);
  if (a.row_cap <= 16) return ffn_launch<Q4, 2>(m, a, ctas, st);
  if (a.row_cap <= 32) return ffn_launch<Q4, 4>(m, a, ctas, st);
  return ffn_launch<Q4, 8>(m, a, ctas, st);
}

}  // namespace

cudaError_t launch_decode_ffn(bool q4, const DecFfnMaps& m, const DecFfnArgs& a, int ctas,
                              cudaStream_t st) {
  return q4 ? ffn_rows<true>(m, a, ctas, st) : ffn_rows<false>(m, a, ctas, st);
}

cudaError_t decode_route_set_attributes();

cudaError_t decode_set_attributes() {
  cudaError_t e = decode_route_set_attributes();
  if (e == cudaSuccess) e = ffn_attr<false, 1>();
  if (e == cudaSuccess) e = ffn_attr<false, 2>();
  if (e == cudaSuccess) e = ffn_attr<false, 4>();
  if (e == cudaSuccess) e = ffn_attr<false, 8>();
  if (e == cudaSuccess) e = ffn_attr<true, 1>();
  if (e == cudaSuccess) e = ffn_attr<true, 2>();
  if (e == cudaSuccess) e = ffn_attr<true, 4>();
  if (e == cudaSuccess) e = ffn_attr<true, 8>();
  return e;
}

}  // namespace moe
