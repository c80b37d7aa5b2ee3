// decode_route.cu -- first kernel of the decode operators: the whole route
// (logits, TopK, gate, dispatch) of at most 64 tokens by one cluster of 8
// CTAs, and the entry list of the grouped products.
//
// "用Ascend C写一个MoE融合算子", section "1. Routing + Gating 合并" and listing
// "Gather操作", as in route_fused.cu; what differs is the size.  A few tokens'
// logits are a [T, H] x [H, E] product of at most a megabyte or two, far too
// little to fill the GPU and bound by latency: one trip to memory, one
// reduction, two cluster barriers.  The H axis is split over the 8 CTAs, so
// one trip to memory brings all of W_router; within a CTA the warps split the
// remaining K steps and the experts.  The products are m16n8k16 tensor-core
// ones with W_router as the M operand (ldmatrix.trans: E is contiguous) and
// the tokens as N: bf16 products are exact in fp32, sums are fp32 in a fixed
// order (warps of a CTA, then ranks 0..7).  Every rank stores its partial
// logits into the shared memory of the rank that owns the token (rank 0 owns
// all of up to 8 tokens, else t mod 8), so that the owner reads its own
// memory after the barrier; a cluster barrier that ends before the first of these
// stores says that all ranks run.  Logits are fp32, as moe_forward's: two that are
// closer than the rounding of such a sum may be chosen in either order.  A warp per token then takes the k largest, one
// per round (two warp-wide integer reductions: the largest, then the lowest
// index that has it).  This code runs once per launch and comes cold from
// memory, so its size is its cost: the loops stay loops.  Rank 0 then holds
// every id and dispatches: at most 512 assignments, ranked within their
// expert by warp match and a scan over the warps' chunks.
//
// Measured, from the end of the kernel before to the start of the next: 4.2 us for one
// token, H = 4096, E = 8 (0.7 loading, 1.3 products and exchange, 1.2 TopK, 1.0
// dispatch and launch), 5.6 us for H = 2048, E = 64, k = 4.
#include <math.h>

#include "decode_internal.h"
#include "tc_common.cuh"

namespace moe {
namespace {

constexpr int DR_THREADS = 256;
constexpr int DR_WARPS = DR_THREADS / 32;
constexpr int DR_RANKS = 8;
constexpr int DR_MAX_ASSIGN = MOED_MAX_TOKENS * kMaxTopK;  // 512
constexpr int DR_STAGE_BYTES = 140 * 1024;  // W_router and x rows staged at a time

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm_x2(uint32_t a, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];"
               : "=r"(r0), "=r"(r1)
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void dsmem_st_u32(uint32_t cluster_saddr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_saddr), "r"(v) : "memory");
}

struct RouteLayout {
  int ep;      // experts rounded up to 16
  int tp;      // tokens rounded up to 8, 16, 32 or 64 (the kernel's token tiles)
  int kb;      // K rows staged at a time (a multiple of 16)
  int pw, px;  // row pitches of the staged W_router and x, bytes (odd multiples of 16)
  int hs;      // H rows of a CTA
  int wm;      // warps along the experts (the others split K)
  size_t stage, part, total;
};

// Row pitches of the staged W_router and x: odd multiples of 16 bytes, so that
// the 8 rows of an ldmatrix fall into different banks.
__host__ __device__ inline int w_pitch(int E) { return 16 * ((E * 2 + 15) / 16 | 1); }
__host__ __device__ inline int token_tile(int T) { return T <= 8 ? 8 : T <= 16 ? 16 : T <= 32 ? 32 : 64; }

__host__ __device__ inline RouteLayout route_layout(int T, int H, int E) {
  RouteLayout L;
  L.ep = (E + 15) / 16 * 16;
  L.tp = token_tile(T);
  L.hs = (H + DR_RANKS * 16 - 1) / (DR_RANKS * 16) * 16;
  L.pw = w_pitch(E);  // (the columns up to ep belong to the next row: of no expert)
  // kb rows of W_router (pw bytes) and of every token (2 kb + 16 bytes)
  int kb = (DR_STAGE_BYTES - 16 * L.tp) / (L.pw + 2 * L.tp) / 16 * 16;
  if (kb > L.hs) kb = L.hs;
  if (kb < 16) kb = 16;
  L.kb = kb;
  L.px = kb * 2 + 16;
  L.wm = 1;
  while (L.wm < DR_WARPS && L.wm * 16 < L.ep) L.wm *= 2;
  const size_t tiles = (size_t)kb * L.pw + (size_t)L.tp * L.px;
  const size_t red = (size_t)(DR_WARPS / L.wm) * L.tp * L.ep * 4;  // reuses the tiles' space
  // partial logits of the tokens a rank owns, from all ranks
  const size_t own = T <= DR_RANKS ? (size_t)L.tp : (size_t)(T + DR_RANKS - 1) / DR_RANKS;
  L.stage = tiles > red ? tiles : red;
  const size_t wc = T * 8 > 32 ? (size_t)(T * 8 + 31) / 32 * kMaxExperts * 4 : 0;  // the dispatch's counts
  if (L.stage < wc) L.stage = wc;
  L.stage = (L.stage + 127) / 128 * 128;
  L.part = DR_RANKS * own * L.ep * 4;
  L.total = L.stage + L.part;
  return L;
}

// fp32 -> unsigned integers of the same order, none of them 0
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);  // -0 as +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// NT: 8-token tiles.
template <int NT>
__global__ void __cluster_dims__(DR_RANKS, 1, 1) __launch_bounds__(DR_THREADS, 1)
    decode_route_kernel(const DecRouteArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_ids[DR_MAX_ASSIGN];
  __shared__ int s_off[kMaxExperts + 1];
  __shared__ int s_scan[2][DR_WARPS];
  __shared__ float s_log[DR_WARPS][kMaxExperts];
  __shared__ float s_bias[kMaxExperts];
  __shared__ uint32_t s_key[DR_WARPS][kMaxExperts];

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int rank = (int)cluster_ctarank();
  const RouteLayout L = route_layout(a.T, a.H, a.E);
  const int E = a.E, T = a.T, H = a.H, k = a.k;
  uint8_t* sW = smem;
  uint8_t* sX = smem + (size_t)L.kb * L.pw;
  float* sRed = reinterpret_cast<float*>(smem);
  float* sPart = reinterpret_cast<float*>(smem + L.stage);
  int* s_wc = reinterpret_cast<int*>(smem);  // dispatch: [chunk][expert], over the stage
  // counted here, waited for before the first store to another rank's shared memory:
  // only the cluster barrier says that all ranks have started, and ranks past the
  // end of H come to that store almost at once
  cluster_arrive();
  pdl_launch_dependents();
  pdl_wait();

  // the counters of the second kernel
  if (rank == 0 && tid < kDecCtrlInts) a.ctrl[tid] = 0;
  if (tid < E) s_bias[tid] = a.bias ? __ldg(a.bias + tid) : 0.f;  // read behind the barriers below

  // ---- partial logits of rows [h0, h1) of H
  const int h0 = min(rank * L.hs, H), h1 = min(h0 + L.hs, H);
  const int wm = warp & (L.wm - 1);        // expert tiles wm, wm + L.wm
  const int wk = warp / L.wm;              // K steps wk, wk + nk, ...
  const int nk = DR_WARPS / L.wm;
  const int mt = L.ep / 16;
  float acc[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[m][n][r] = 0.f;

  for (int hb = h0; hb < h1; hb += L.kb) {
    const int rows = min(L.kb, h1 - hb);      // a multiple of 8
    const int rows16 = (rows + 15) / 16 * 16;
    if (hb != h0) __syncthreads();
    if ((E & 7) == 0) {
      const int ch = E / 8;
      for (int i = tid; i < rows * ch; i += DR_THREADS) {
        const int r = i / ch, c = i - r * ch;
        cp_async16(smem_u32(sW + (size_t)r * L.pw + c * 16), a.w + (size_t)(hb + r) * E + c * 8);
      }
    } else {  // rows not 16-byte aligned
      const uint16_t* src = a.w + (size_t)hb * E;
      for (int i = tid; i < rows * E; i += DR_THREADS) {
        const int r = i / E, c = i - r * E;
        *reinterpret_cast<uint16_t*>(sW + (size_t)r * L.pw + c * 2) = __ldg(src + i);
      }
    }
    const int xc = rows / 8;
    for (int i = tid; i < T * xc; i += DR_THREADS) {
      const int t = i / xc, c = i - t * xc;
      cp_async16(smem_u32(sX + (size_t)t * L.px + c * 16), a.x + (size_t)t * H + hb + c * 8);
    }
    if (rows16 != rows) {  // zero the half step past the end in both operands
      for (int i = tid; i < 8 * (L.pw / 16); i += DR_THREADS) {
        const int r = rows + i / (L.pw / 16), c = i % (L.pw / 16);
        *reinterpret_cast<uint4*>(sW + (size_t)r * L.pw + c * 16) = make_uint4(0, 0, 0, 0);
      }
      for (int t = tid; t < T; t += DR_THREADS)
        *reinterpret_cast<uint4*>(sX + (size_t)t * L.px + rows * 2) = make_uint4(0, 0, 0, 0);
    }
    cp_async_wait_all();
    __syncthreads();
    for (int ks = wk; ks < rows16 / 16; ks += nk) {
      uint32_t b[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
        ldsm_x2(smem_u32(sX + (size_t)(n * 8 + (lane & 7)) * L.px + ks * 32 + ((lane >> 3) & 1) * 16),
                b[n][0], b[n][1]);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int tile = wm + m * L.wm;
        if (tile >= mt) break;
        uint32_t w[4];
        ldsm_x4_t(smem_u32(sW + (size_t)(ks * 16 + (lane >> 4) * 8 + (lane & 7)) * L.pw + tile * 32 +
                           ((lane >> 3) & 1) * 16),
                  w);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_bf16(acc[m][n], w, b[n][0], b[n][1]);
      }
    }
  }
  __syncthreads();
  // sum over the warps that split K: [wk][token][expert]
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int tile = wm + m * L.wm;
    if (tile >= mt) break;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int e = tile * 16 + (lane >> 2) + (r >> 1) * 8;
        const int t = n * 8 + (lane & 3) * 2 + (r & 1);
        sRed[((size_t)wk * L.tp + t) * L.ep + e] = acc[m][n][r];
      }
  }
  __syncthreads();
  const bool one_owner = T <= DR_RANKS;
  const int own = one_owner ? L.tp : (T + DR_RANKS - 1) / DR_RANKS;  // tokens of an owner
  const uint32_t part0 = smem_u32(sPart);
  cluster_wait();
  for (int i = tid; i < T * (L.ep / 4); i += DR_THREADS) {
    const int t = i / (L.ep / 4), c4 = i - t * (L.ep / 4);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < nk; ++w) {
      const float4 o = *reinterpret_cast<const float4*>(sRed + ((size_t)w * L.tp + t) * L.ep + c4 * 4);
      v.x += o.x;
      v.y += o.y;
      v.z += o.z;
      v.w += o.w;
    }
    const int owner = one_owner ? 0 : t % DR_RANKS, tl = one_owner ? t : t / DR_RANKS;
    dsmem_st_v4(dsmem_map(part0 + (uint32_t)(((rank * own + tl) * L.ep + c4 * 4) * 4), (uint32_t)owner),
                v.x, v.y, v.z, v.w);
  }
  cluster_sync_all();

  // ---- TopK and gate weights of the tokens this rank owns, a warp each
  for (int tl = warp; tl < own; tl += DR_WARPS) {
    const int t = one_owner ? tl : tl * DR_RANKS + rank;
    if (t >= T || (one_owner && rank != 0)) break;
    float* lg = s_log[warp];
    uint32_t* key = s_key[warp];
    for (int e = lane; e < E; e += 32) {
      float v = 0.f;
#pragma unroll
      for (int r = 0; r < DR_RANKS; ++r) v += sPart[((size_t)r * own + tl) * L.ep + e];
      if (a.bias) v += s_bias[e];
      if (isnan(v)) v = -INFINITY;
      lg[e] = v;
      key[e] = order_key(v);
    }
    int id = 0;
    float top = 0.f;
#pragma unroll 1
    for (int j = 0; j < k; ++j) {
      // each lane's largest untaken (its lowest index: strictly larger
      // replaces), then the warp's, then the lowest index that has it
      uint32_t bk = 0;
      int be = kMaxExperts;
#pragma unroll 1
      for (int e = lane; e < E; e += 32) {
        const uint32_t u = key[e];
        if (u > bk) {
          bk = u;
          be = e;
        }
      }
      const uint32_t m = __reduce_max_sync(0xffffffffu, bk);
      const int e = __reduce_min_sync(0xffffffffu, bk == m ? be : kMaxExperts);
      if (lane == (e & 31)) key[e] = 0;  // taken
      if (lane == j) {
        id = e;
        top = lg[e];
      }
      __syncwarp();
    }
    const float mx = __shfl_sync(0xffffffffu, top, 0);
    float ex = lane < k ? expf(top - mx) : 0.f;
    if (a.gating != MOE_GATE_TOPK_SOFTMAX) {  // softmax over all E first
      float zall = 0.f;
      for (int e = lane; e < E; e += 32) zall += expf(lg[e] - mx);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) zall += __shfl_xor_sync(0xffffffffu, zall, off);
      ex /= zall;
    }
    float z = ex;
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
    if (a.gating != MOE_GATE_SOFTMAX_TOPK) ex /= z;
    if (lane < k) {
      a.ids[(size_t)t * k + lane] = id;
      a.weights[(size_t)t * k + lane] = ex;
      if (one_owner)
        s_ids[t * k + lane] = id;
      else
        dsmem_st_u32(dsmem_map(smem_u32(s_ids + t * k + lane), 0), (uint32_t)id);
    }
    __syncwarp();
  }
  if (one_owner) {
    if (rank != 0) return;  // nothing of these ranks is read any more
    __syncthreads();
  } else {
    cluster_sync_all();
    if (rank != 0) return;
  }

  // ---- dispatch of all T*k assignments, in (token, slot) order
  const int n = T * k;
  if (n <= 32) {
    // one assignment per lane, the same in every warp: ranks by match, sums
    // over the assignments by shuffles, no barrier.  Lane i's `word`: expert,
    // kept or not, and for the first kept one of an expert its row blocks.
    const int id = lane < n ? s_ids[lane] : -1;
    const unsigned same = __match_any_sync(0xffffffffu, id);
    const int rank_e = __popc(same & ((1u << lane) - 1u));
    const bool kept = lane < n && (a.capacity < 0 || rank_e < a.capacity);
    const unsigned kept_mask = __ballot_sync(0xffffffffu, kept);
    const int cnt = __popc(same & kept_mask);
    const int blocks = kept && rank_e == 0 ? (cnt + a.row_block - 1) / a.row_block : 0;
    const int word = lane < n ? id | (kept ? 256 : 0) | blocks << 16 : 1 << 12;
    int my_off = 0, e_cnt = 0, e_off = 0, e_blk = 0, e_own = 0, all = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int w = __shfl_sync(0xffffffffu, word, i);
      const int e = w & 255, on = (w >> 8) & 1, b = w >> 16;
      my_off += on & (e < id);
      e_cnt += on & (e == tid);
      e_off += on & (e < tid);
      e_blk += e < tid ? b : 0;
      e_own += e == tid ? b : 0;
      all += b;
    }
    const int total = __popc(kept_mask);
    if (tid < E) {
      a.counts[tid] = e_cnt;
      a.offsets[tid] = e_off;
      for (int b = 0; b < e_own; ++b)
        a.entries[e_blk + b] =
            DecEntry{tid, e_off + b * a.row_block, min(a.row_block, e_cnt - b * a.row_block), 0};
    }
    const int longest = __reduce_max_sync(0xffffffffu, min(cnt, a.row_block));
    if (warp == 0) {
      if (lane < n) {
        a.slot[lane] = kept ? my_off + rank_e : -1;
        if (kept) a.perm[my_off + rank_e] = lane;
      }
      if (lane >= total && lane < n) a.perm[lane] = -1;
      if (lane == 0) {
        a.offsets[E] = total;
        a.ctrl[kDecCountOffset / 4] = all;
        a.ctrl[kDecCountOffset / 4 + 1] = longest;
      }
    }
    return;
  }
  const int chunks = (n + 31) / 32;
  for (int i = tid; i < chunks * kMaxExperts; i += DR_THREADS) s_wc[i] = 0;
  __syncthreads();
  int my_e[2], below[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int c = warp + u * DR_WARPS;
    my_e[u] = -1;
    below[u] = 0;
    if (c < chunks) {
      const int i = c * 32 + lane;
      int e = i < n ? s_ids[i] : -1;
      if (e < 0 || e >= E) e = -1;
      const unsigned m = __match_any_sync(0xffffffffu, e);
      below[u] = __popc(m & ((1u << lane) - 1u));
      if (e >= 0 && below[u] == 0) s_wc[c * kMaxExperts + e] = __popc(m);
      my_e[u] = e;
    }
  }
  __syncthreads();
  int kept = 0;
  if (tid < E) {
    int run = 0;
    for (int c = 0; c < chunks; ++c) {
      const int v = s_wc[c * kMaxExperts + tid];
      s_wc[c * kMaxExperts + tid] = run;
      run += v;
    }
    kept = a.capacity >= 0 ? min(run, a.capacity) : run;
  }
  // exclusive scans over the experts of the kept rows and of their row blocks
  // (16 bits each: at most 512 of either)
  const int blocks = (kept + a.row_block - 1) / a.row_block;
  int incl = kept | blocks << 16;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += v;
  }
  if (lane == 31) s_scan[0][warp] = incl;
  const int longest = __reduce_max_sync(0xffffffffu, min(kept, a.row_block));
  if (lane == 0) s_scan[1][warp] = longest;
  __syncthreads();
  int before = 0, all = 0, max_rows = 0;
#pragma unroll
  for (int w = 0; w < DR_WARPS; ++w) {
    max_rows = max(max_rows, s_scan[1][w]);
    if (w < warp) before += s_scan[0][w];
    all += s_scan[0][w];
  }
  const int total = all & 0xFFFF;
  if (tid < E) {
    const int excl = before + incl;
    const int off = (excl & 0xFFFF) - kept;
    s_off[tid] = off;
    a.counts[tid] = kept;
    a.offsets[tid] = off;
    for (int b = 0; b < blocks; ++b)
      a.entries[(excl >> 16) - blocks + b] =
          DecEntry{tid, off + b * a.row_block, min(a.row_block, kept - b * a.row_block), 0};
  }
  if (tid == 0) {
    a.offsets[E] = total;
    a.ctrl[kDecCountOffset / 4] = all >> 16;
    a.ctrl[kDecCountOffset / 4 + 1] = max_rows;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int c = warp + u * DR_WARPS;
    const int i = c * 32 + lane;
    if (c >= chunks || i >= n) continue;
    const int e = my_e[u];
    const int pos = e >= 0 ? s_wc[c * kMaxExperts + e] + below[u] : -1;
    if (pos >= 0 && (a.capacity < 0 || pos < a.capacity)) {
      a.slot[i] = s_off[e] + pos;
      a.perm[s_off[e] + pos] = i;
    } else {
      a.slot[i] = -1;
    }
  }
  for (int i = total + tid; i < n; i += DR_THREADS) a.perm[i] = -1;
}

// Entries of the grouped products: segment i's rows in blocks of row_block.
__global__ void __launch_bounds__(256) decode_prep_kernel(const DecPrepArgs a) {
  __shared__ int s_scan[8], s_rows[8], s_max[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  pdl_wait();
  for (int i = tid; i < kDecCtrlInts; i += 256) a.ctrl[i] = 0;
  // each row belongs to one entry at most, and the entries have room: offsets are
  // clamped to [0, rows] and to the largest before them (a scan), so that a
  // decreasing one gives an empty segment
  int o0 = 0, o1 = 0;
  if (tid < a.n_segments) {
    o0 = a.seg_offsets ? min(max(__ldg(a.seg_offsets + tid), 0), a.rows) : 0;
    o1 = a.seg_offsets ? min(max(__ldg(a.seg_offsets + tid + 1), 0), a.rows) : a.rows;
  }
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, o0, off);
    if (lane >= off) o0 = max(o0, v);
  }
  if (lane == 31) s_max[warp] = o0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w)
    if (w < warp) o0 = max(o0, s_max[w]);
  const int n = max(o1 - o0, 0);
  const int blocks = (n + a.row_block - 1) / a.row_block;
  int incl = blocks;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += v;
  }
  const int longest = __reduce_max_sync(0xffffffffu, min(n, a.row_block));
  if (lane == 31) {
    s_scan[warp] = incl;
    s_rows[warp] = longest;
  }
  __syncthreads();
  int base = 0, total = 0, max_rows = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w < warp) base += s_scan[w];
    total += s_scan[w];
    max_rows = max(max_rows, s_rows[w]);
  }
  int at = base + incl - blocks;
  for (int b = 0; b < blocks && at < a.max_entries; ++b, ++at)
    a.entries[at] = DecEntry{tid % a.E, o0 + b * a.row_block, min(a.row_block, n - b * a.row_block), 0};
  if (tid == 0) {
    a.ctrl[kDecCountOffset / 4] = min(total, a.max_entries);
    a.ctrl[kDecCountOffset / 4 + 1] = max_rows;
  }
}

template <int NT>
cudaError_t route_launch(const DecRouteArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(DR_RANKS, 1, 1);
  cfg.blockDim = dim3(DR_THREADS, 1, 1);
  cfg.dynamicSmemBytes = route_layout(a.T, a.H, a.E).total;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  set_pdl_attr(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_route_kernel<NT>, a);
}

template <int NT>
cudaError_t route_attr() {
  // stage plus partial logits at the largest shapes: 140 KB + 64 KB
  return cudaFuncSetAttribute(decode_route_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              DR_STAGE_BYTES + MOED_MAX_TOKENS * kMaxExperts * 4);
}

}  // namespace

cudaError_t launch_decode_route(const DecRouteArgs& a, cudaStream_t st) {
  const int nt = (a.T + 7) / 8;
  if (nt <= 1) return route_launch<1>(a, st);
  if (nt <= 2) return route_launch<2>(a, st);
  if (nt <= 4) return route_launch<4>(a, st);
  return route_launch<8>(a, st);
}

cudaError_t launch_decode_prep(const DecPrepArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  set_pdl_attr(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_prep_kernel, a);
}

cudaError_t decode_route_set_attributes() {
  cudaError_t e = route_attr<1>();
  if (e == cudaSuccess) e = route_attr<2>();
  if (e == cudaSuccess) e = route_attr<4>();
  if (e == cudaSuccess) e = route_attr<8>();
  return e;
}

}  // namespace moe
