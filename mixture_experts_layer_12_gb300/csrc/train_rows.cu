// train_rows.cu -- the training step's kernels that move rows and elements:
// rows into padded expert order, the gradients of dispatch and combine,
// activations in 8 bits, the gate's gradient and the router's sums.  All are
// bound by memory; each output element is written by one thread, so sums have
// one order.
#include "train_seg.cuh"

namespace moe {
namespace {

template <typename Kernel, typename... Args>
cudaError_t launch(Kernel k, dim3 grid, int threads, cudaStream_t st, const Args&... a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  set_pdl_attr(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, a...);
}

unsigned blocks_for(int64_t items, int64_t per_block, int64_t cap) {
  const int64_t n = (items + per_block - 1) / per_block;
  return (unsigned)(n < 1 ? 1 : n < cap ? n : cap);
}

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  f[0] = bf16_lo(u.x);
  f[1] = bf16_hi(u.x);
  f[2] = bf16_lo(u.y);
  f[3] = bf16_hi(u.y);
  f[4] = bf16_lo(u.z);
  f[5] = bf16_hi(u.z);
  f[6] = bf16_lo(u.w);
  f[7] = bf16_hi(u.w);
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  uint4 o;
  o.x = pack_bf16x2(f[0], f[1]);
  o.y = pack_bf16x2(f[2], f[3]);
  o.z = pack_bf16x2(f[4], f[5]);
  o.w = pack_bf16x2(f[6], f[7]);
  return o;
}

// ------------------------------------------------- rows in padded order --
// LPR lanes per padded row (a warp where a row has 256 columns or more): its
// segment by bisection of the padded offsets, then a copy with eight 16-byte
// loads in flight per lane.  25271 rows of 2048 columns: 25 us one matrix, 50
// both (206 MB written, the sources mostly out of L2); 16384 rows of 64 columns
// by whole warps 20 us, by 8 lanes 10.
constexpr int GTHREADS = 256;
template <int LPR>
__global__ void __launch_bounds__(GTHREADS) train_gather_kernel(const GatherArgs a) {
  __shared__ SegTable t;
  pdl_launch_dependents();
  pdl_wait();
  const int E = a.seg.E;
  if (!a.compact) {
    if (threadIdx.x < 32) seg_scan(a.seg, t, nullptr, threadIdx.x, nullptr, [](int) { return 0; });
    __syncthreads();
  }
  const int total = a.compact ? min(max(__ldg(a.seg.offsets + E), 0), a.seg.rows) : t.pad_off[E];
  const int vec = a.H / 8;
  const int lane = threadIdx.x % LPR;
  const uint16_t* src0 = a.src[blockIdx.y];
  uint16_t* dst0 = a.dst[blockIdx.y];
  constexpr int ROWS = GTHREADS / LPR;
  for (int pr = blockIdx.x * ROWS + threadIdx.x / LPR; pr < total; pr += gridDim.x * ROWS) {
    uint4* dst = reinterpret_cast<uint4*>(dst0 + (size_t)pr * a.ld);
    int r = pr;
    if (!a.compact) {
      int lo = 0, hi = E;  // the last segment that starts at or before pr
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.pad_off[mid] <= pr) lo = mid; else hi = mid;
      }
      const int i = pr - t.pad_off[lo];
      if (i >= t.rows[lo]) {
        for (int c = lane; c < vec; c += LPR) dst[c] = make_uint4(0u, 0u, 0u, 0u);
        continue;
      }
      r = t.row_off[lo] + i;
    }
    if (a.perm) r = min(max(__ldg(a.perm + r) / a.k, 0), a.T - 1);
    const uint4* src = reinterpret_cast<const uint4*>(src0 + (size_t)r * a.H);
    int c = lane;
    for (; c + 7 * LPR < vec; c += 8 * LPR) {
      uint4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = __ldg(src + c + LPR * u);
#pragma unroll
      for (int u = 0; u < 8; ++u) dst[c + LPR * u] = v[u];
    }
    for (; c < vec; c += LPR) dst[c] = __ldg(src + c);
  }
}

// ------------------------------------------------------- sums of a token's rows --
// out[t] = add[t] + sum_j w[t, j] rows[slot[t, j]] (add and w with rows in fp32
// only): a thread takes two 8-column chunks of one token (one where rows are in
// fp32: the same bytes) and asks for all k rows' before the sums.  8192 tokens of
// 2048 columns, k = 4 with drops: 22 us in bf16 (6.2 TB/s), 34 in fp32 (7.1 TB/s,
// part of it out of L2), 40 with the router's rows.
constexpr int RTHREADS = 128;
// The router's part of a token's gradient, k rows of W_router^T out of L2: as a
// product of its own into an fp32 [T, H] it took 21 us more for 8192 tokens of
// 2048 columns (and where every expert has a part it still is one: `add`).
template <int KMAX>
__device__ __forceinline__ void add_router_rows(const RowsSumArgs& a, int t, int col, float* s) {
  if (!a.dl) return;
  uint4 v[KMAX];
  float d[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    d[j] = 0.0f;
    v[j] = make_uint4(0u, 0u, 0u, 0u);
    if (j < a.k) {
      const int e = __ldg(a.ids + (size_t)t * a.k + j);
      if (e >= 0 && e < a.E) {
        d[j] = __ldg(a.dl + (size_t)t * a.k + j);
        v[j] = __ldg(reinterpret_cast<const uint4*>(a.wt + (size_t)e * a.H + col));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    float f[8];
    unpack8(v[j], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = fmaf(d[j], f[i], s[i]);
  }
}

template <int KMAX, bool F32, bool PARTS>
__global__ void __launch_bounds__(RTHREADS) rows_sum_kernel(const RowsSumArgs a) {
  constexpr int RCPT = F32 ? 1 : 2;
  pdl_launch_dependents();
  pdl_wait();
  const int t = blockIdx.x;
  const int col0 = (blockIdx.y * RTHREADS * RCPT + threadIdx.x) * 8;
  if (col0 >= a.H) return;
  if (PARTS && a.range && (t < __ldg(a.range) || t >= __ldg(a.range + a.E))) return;
  int r[KMAX];
  [[maybe_unused]] float w[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    r[j] = a.slot && j < a.k ? __ldg(a.slot + (size_t)t * a.k + j) : -1;
    if (r[j] >= a.T * a.k) r[j] = -1;  // slot is not re-validated: nothing outside rows
    if (PARTS && a.range && j == 0) r[j] = t;
    if constexpr (F32) w[j] = a.w && r[j] >= 0 ? __ldg(a.w + (size_t)t * a.k + j) : 1.0f;
  }
  if constexpr (F32) {
    float4 v[KMAX][2], s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      s[h] = a.add ? __ldg(reinterpret_cast<const float4*>(a.add + (size_t)t * a.H + col0) + h)
                   : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const size_t part = (size_t)a.T * a.k * a.H;
    for (int p = 0; p < (PARTS ? a.splits : 1); ++p) {
      const float* rows = a.rows32 + p * part + col0;
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (r[j] >= 0)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            v[j][h] = __ldg(reinterpret_cast<const float4*>(rows + (size_t)r[j] * a.H) + h);
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (r[j] >= 0)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            s[h].x = fmaf(w[j], v[j][h].x, s[h].x);
            s[h].y = fmaf(w[j], v[j][h].y, s[h].y);
            s[h].z = fmaf(w[j], v[j][h].z, s[h].z);
            s[h].w = fmaf(w[j], v[j][h].w, s[h].w);
          }
    }
    float f[8] = {s[0].x, s[0].y, s[0].z, s[0].w, s[1].x, s[1].y, s[1].z, s[1].w};
    add_router_rows<KMAX>(a, t, col0, f);
    *reinterpret_cast<uint4*>(a.out + (size_t)t * a.H + col0) = pack8(f);
  } else {
    uint4 v[KMAX][RCPT];
#pragma unroll
    for (int c = 0; c < RCPT; ++c) {
      const int col = col0 + c * RTHREADS * 8;
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (r[j] >= 0 && col < a.H)
          v[j][c] = __ldg(reinterpret_cast<const uint4*>(a.rows + (size_t)r[j] * a.H + col));
    }
#pragma unroll
    for (int c = 0; c < RCPT; ++c) {
      const int col = col0 + c * RTHREADS * 8;
      if (col >= a.H) break;
      float s[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (r[j] >= 0) {
          float f[8];
          unpack8(v[j][c], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) s[i] += f[i];
        }
      add_router_rows<KMAX>(a, t, col, s);
      *reinterpret_cast<uint4*>(a.out + (size_t)t * a.H + col) = pack8(s);
    }
  }
}

// -------------------------------------------------------- combine's gradient --
// W warps per token: dy[t] is read once, the k rows of Y beside it; row
// slot[t, j] of dY is written by its only token, dw[t, j] is summed over the
// warps in their order.  8192 tokens of 2048 columns, k = 4 with drops: 40 us (240
// MB, 6.0 TB/s).  Up to 512 columns a warp takes a token alone.
template <int KMAX, int W>
__global__ void __launch_bounds__(128) combine_backward_kernel(const CombineBackwardArgs a) {
  constexpr int TOK = 4 / W;  // tokens per block
  __shared__ float red[4][KMAX];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * TOK + warp / W;
  const bool ok = t < a.T;
  int r[KMAX];
  float w[KMAX], dot[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    r[j] = ok && j < a.k ? __ldg(a.slot + (size_t)t * a.k + j) : -1;
    if (r[j] >= a.T * a.k) r[j] = -1;  // slot is not re-validated: nothing outside Y and dY
    w[j] = r[j] >= 0 ? __ldg(a.w + (size_t)t * a.k + j) : 0.0f;
    dot[j] = 0.0f;
  }
  const int vec = a.H / 8;
  if (ok) {
    const uint4* dy = reinterpret_cast<const uint4*>(a.dy + (size_t)t * a.H);
    for (int c = (warp % W) * 32 + lane; c < vec; c += 32 * W) {
      const uint4 g4 = __ldg(dy + c);
      uint4 v[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (r[j] >= 0) v[j] = __ldg(reinterpret_cast<const uint4*>(a.Y + (size_t)r[j] * a.H) + c);
      float g[8];
      unpack8(g4, g);
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (r[j] >= 0) {
          float f[8], o[8];
          unpack8(v[j], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[j] = fmaf(g[i], f[i], dot[j]);
            o[i] = w[j] * g[i];
          }
          *(reinterpret_cast<uint4*>(a.dY + (size_t)r[j] * a.H) + c) = pack8(o);
        }
    }
  }
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], off);
    if (lane == 0) red[warp][j] = dot[j];
  }
  __syncthreads();
  if (ok && warp % W == 0 && lane < a.k) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) s += red[warp + i][lane];
    a.dw[(size_t)t * a.k + lane] = s;  // a dropped slot has read nothing: 0
  }
}

// ------------------------------------------------------ activations in 8 bits --
// A lane takes 8 columns; the 4 lanes of a group share its largest magnitude
// by two shuffles.  Groups never cross a row: `per_row` counts the chunks of a
// row rounded up to whole groups (cols % 32 == 0: none are missing and rows
// need no division).  8192 x 14336: 59 us to 8 bits (6.0 TB/s), 52 back (6.8).
constexpr int QTHREADS = 256;
constexpr int QILP = 4;
template <bool FLAT>
__global__ void __launch_bounds__(QTHREADS) quantize_a8_kernel(int64_t chunks, int per_row, int cols,
                                                               const uint16_t* x, int8_t* codes,
                                                               uint8_t* scales) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t step = (int64_t)gridDim.x * QTHREADS;
  for (int64_t i0 = (int64_t)blockIdx.x * QTHREADS + threadIdx.x; i0 - (threadIdx.x & 31) < chunks;
       i0 += step * QILP) {
    uint4 v[QILP];
    int64_t at[QILP];
#pragma unroll
    for (int u = 0; u < QILP; ++u) {
      const int64_t i = i0 + u * step;
      at[u] = -1;
      v[u] = make_uint4(0u, 0u, 0u, 0u);
      if (i < chunks) {
        if (FLAT) {
          at[u] = i * 8;
        } else {
          const int64_t row = chunks <= 0x7fffffff ? (int64_t)((uint32_t)i / (uint32_t)per_row) : i / per_row;
          const int c = (int)(i - row * per_row) * 8;
          if (c < cols) at[u] = row * cols + c;
        }
        if (at[u] >= 0) v[u] = __ldcs(reinterpret_cast<const uint4*>(x + at[u]));
      }
    }
#pragma unroll
    for (int u = 0; u < QILP; ++u) {
      const uint32_t wv[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = max(m, max(wv[i] & 0x7fffu, (wv[i] >> 16) & 0x7fffu));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const uint32_t b = a8_scale_byte(m << 16);
      const float inv = a8_inverse(b);
      if (at[u] >= 0) {
        float f[8];
        unpack8(v[u], f);
        *reinterpret_cast<uint2*>(codes + at[u]) = a8_codes8(f, inv, b);
      }
      const int64_t i = i0 + u * step;
      if (i < chunks && (threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)b;
    }
  }
}

template <bool FLAT>
__global__ void __launch_bounds__(QTHREADS) dequantize_a8_kernel(int64_t chunks, int per_row, int cols,
                                                                 const int8_t* codes,
                                                                 const uint8_t* scales, uint16_t* out) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t step = (int64_t)gridDim.x * QTHREADS;
  for (int64_t i0 = (int64_t)blockIdx.x * QTHREADS + threadIdx.x; i0 < chunks; i0 += step * QILP) {
    uint2 v[QILP];
    uint32_t b[QILP];
    int64_t at[QILP];
#pragma unroll
    for (int u = 0; u < QILP; ++u) {
      const int64_t i = i0 + u * step;
      at[u] = -1;
      if (i < chunks) {
        if (FLAT) {
          at[u] = i * 8;
        } else {
          const int64_t row = chunks <= 0x7fffffff ? (int64_t)((uint32_t)i / (uint32_t)per_row) : i / per_row;
          const int c = (int)(i - row * per_row) * 8;
          if (c < cols) at[u] = row * cols + c;
        }
        if (at[u] >= 0) {
          v[u] = __ldcs(reinterpret_cast<const uint2*>(codes + at[u]));
          b[u] = __ldg(scales + (i >> 2));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < QILP; ++u)
      if (at[u] >= 0) {
        float f[8];
        const float s = a8_scale(b[u]);
        a8_values(v[u].x, s, f);
        a8_values(v[u].y, s, f + 4);
        *reinterpret_cast<uint4*>(out + at[u]) = pack8(f);
      }
  }
}

// ------------------------------------------------------------ the gate's gradient --
// A block takes 16 tokens, a warp two (with 64 a block and one row of partial
// sums at a time 26 us for 8192 tokens of 64 experts, k = 4, and 20 for 4096 of
// 14336 columns; so 8 and 11); lane l holds experts
// l, l + 32, ...  With the weights of a softmax over the chosen experts,
// dlogit_j = w_j (dw_j - sum_i w_i dw_i) for the chosen and 0 for the others;
// with those of a softmax over all experts, dlogit_e = p_e ([e chosen] dw_e -
// sum_i w_i dw_i) for every expert.  A dropped assignment has dw = 0, not
// dlogit = 0.  dlogits go out as two bf16 numbers (16 bits and what their
// rounding left): the router's products then add the two in fp32.
constexpr int GATE_WARPS = 8;
__global__ void __launch_bounds__(GATE_WARPS * 32) gate_backward_kernel(const GateBackwardArgs a) {
  __shared__ float s_db[GATE_WARPS][kMaxExperts];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int token_blocks = (a.T + kGateTokens - 1) / kGateTokens;
  if ((int)blockIdx.x >= token_blocks) {  // W_router for the products to come
    const int64_t nt = (int64_t)(gridDim.x - token_blocks) * blockDim.x;
    const int64_t i0 = (int64_t)(blockIdx.x - token_blocks) * blockDim.x + threadIdx.x;
    if (a.wt) {
      for (int64_t i = i0; i < (int64_t)a.H / 8 * a.E; i += nt) {
        const int64_t h = i / a.E * 8;
        const int e = (int)(i % a.E);
        uint16_t v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = __ldg(a.w_router + (h + u) * a.E + e);
        *reinterpret_cast<uint4*>(a.wt + (size_t)e * a.H + h) =
            make_uint4(v[0] | (uint32_t)v[1] << 16, v[2] | (uint32_t)v[3] << 16, v[4] | (uint32_t)v[5] << 16,
                       v[6] | (uint32_t)v[7] << 16);
      }
    } else {
      const int per = a.ep / 4;  // 16-byte pieces of a row of w2
      for (int64_t i = i0; i < (int64_t)a.H * per; i += nt) {
        const int64_t h = i / per;
        int e = (int)(i - h * per) * 8;
        if (e >= a.ep) e -= a.ep;
        const uint16_t* src = a.w_router + h * a.E + e;
        uint4 v;
        if (a.E % 8 == 0) {
          v = __ldg(reinterpret_cast<const uint4*>(src));
        } else {
          uint32_t u[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) u[c] = e + c < a.E ? __ldg(src + c) : 0u;
          v = make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
        }
        *reinterpret_cast<uint4*>(a.w2 + i * 8) = v;
      }
    }
    return;
  }
  float acc[kMaxExperts / 32];
#pragma unroll
  for (int i = 0; i < kMaxExperts / 32; ++i) acc[i] = 0.0f;
  for (int i = warp; i < kGateTokens; i += GATE_WARPS) {
    const int t = blockIdx.x * kGateTokens + i;
    if (t >= a.T) break;
    const size_t tk = (size_t)t * a.k;
    int id = -1;
    float w = 0.0f, dw = 0.0f;  // of slot `lane`
    if (lane < a.k) {
      id = __ldg(a.ids + tk + lane);
      w = __ldg(a.weights + tk + lane);
      if (a.dw) dw = __ldg(a.dw + tk + lane);
    }
    if (!a.dw) {
      // all k rows' partial sums at once: their latency is this kernel's time
      const int sl = lane < a.k ? __ldg(a.slot + tk + lane) : -1;
      float s[kMaxTopK];
      int r[kMaxTopK];
#pragma unroll
      for (int j = 0; j < kMaxTopK; ++j) {
        r[j] = __shfl_sync(0xffffffffu, sl, j);
        if (j >= a.k || r[j] >= a.rows) r[j] = -1;
        s[j] = 0.0f;
      }
#pragma unroll 4
      for (int u = lane; u < a.units; u += 32) {
#pragma unroll
        for (int j = 0; j < kMaxTopK; ++j)
          if (r[j] >= 0) s[j] += __ldg(a.part + (size_t)r[j] * a.units + u);
      }
#pragma unroll
      for (int j = 0; j < kMaxTopK; ++j) {
        if (j >= a.k) break;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s[j] += __shfl_xor_sync(0xffffffffu, s[j], off);
        if (lane == j) dw = s[j];
      }
    }
    float S = lane < a.k ? w * dw : 0.0f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) S += __shfl_xor_sync(0xffffffffu, S, off);
    const float mine = w * (dw - S);
    if (a.dlk && lane < a.k) a.dlk[tk + lane] = mine;
    uint16_t* out = a.dl + (size_t)t * 2 * a.ep;
#pragma unroll
    for (int u = 0; u < kMaxExperts / 32; ++u) {
      const int e = lane + 32 * u;
      if (32 * u >= a.ep) break;
      float d = 0.0f;
      if (a.gating == MOE_GATE_SOFTMAX_TOPK) {
        const float pe = e < a.E ? __ldg(a.probs + (size_t)t * a.E + e) : 0.0f;
        float up = -S;
        for (int j = 0; j < a.k; ++j) {
          const int ej = __shfl_sync(0xffffffffu, id, j);
          const float dj = __shfl_sync(0xffffffffu, dw, j);
          if (ej == e) up += dj;
        }
        d = e < a.E ? pe * up : 0.0f;
      } else {
        for (int j = 0; j < a.k; ++j) {
          const int ej = __shfl_sync(0xffffffffu, id, j);
          const float dj = __shfl_sync(0xffffffffu, mine, j);
          if (ej == e && e < a.E) d += dj;
        }
      }
      acc[u] += d;
      if (e < a.ep) {
        const __nv_bfloat16 hi = __float2bfloat16_rn(d);
        const float rest = d - __bfloat162float(hi);
        const __nv_bfloat16 lo = __float2bfloat16_rn(isfinite(d) ? rest : 0.0f);
        out[e] = __bfloat16_as_ushort(hi);
        out[a.ep + e] = __bfloat16_as_ushort(lo);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kMaxExperts / 32; ++u) s_db[warp][lane + 32 * u] = acc[u];
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += GATE_WARPS * 32) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < GATE_WARPS; ++i) s += s_db[i][e];
    a.db_part[(size_t)blockIdx.x * a.E + e] = s;
  }
}

// ----------------------------------------------------------- the router's sums --
// The first blocks sum the token blocks' dlogits, a warp per expert (one thread
// per expert took 11 us for 128 blocks), the others the K splits of dW_router.
constexpr int SUM_THREADS = 256;
__global__ void __launch_bounds__(SUM_THREADS) router_reduce_kernel(const RouterReduceArgs a, int db_blocks) {
  pdl_launch_dependents();
  pdl_wait();
  if ((int)blockIdx.x < db_blocks) {
    const int lane = threadIdx.x & 31;
    const int e = blockIdx.x * (SUM_THREADS / 32) + (threadIdx.x >> 5);
    if (e >= a.E) return;
    float s = 0.0f;
#pragma unroll 4
    for (int b = lane; b < a.n_db; b += 32) s += __ldg(a.db_part + (size_t)b * a.E + e);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (lane == 0) a.db[e] = s;
    return;
  }
  // eight columns of a row of the partial sums: their first and second halves
  const size_t plane = (size_t)a.H * 2 * a.ep;
  const int per = a.ep / 8;
  const int64_t n = (int64_t)a.H * per;
  for (int64_t i = (int64_t)(blockIdx.x - db_blocks) * SUM_THREADS + threadIdx.x; i < n;
       i += (int64_t)(gridDim.x - db_blocks) * SUM_THREADS) {
    const int64_t h = i / per;
    const int e0 = (int)(i - h * per) * 8;
    const float* src = a.part + h * 2 * a.ep + e0;
    float hi[8], lo[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) hi[u] = lo[u] = 0.0f;
#pragma unroll 8
    for (int s = 0; s < a.S; ++s) {
      const float4* p = reinterpret_cast<const float4*>(src + s * plane);
      const float4* q = reinterpret_cast<const float4*>(src + s * plane + a.ep);
      const float4 p0 = __ldg(p), p1 = __ldg(p + 1), q0 = __ldg(q), q1 = __ldg(q + 1);
      hi[0] += p0.x, hi[1] += p0.y, hi[2] += p0.z, hi[3] += p0.w;
      hi[4] += p1.x, hi[5] += p1.y, hi[6] += p1.z, hi[7] += p1.w;
      lo[0] += q0.x, lo[1] += q0.y, lo[2] += q0.z, lo[3] += q0.w;
      lo[4] += q1.x, lo[5] += q1.y, lo[6] += q1.z, lo[7] += q1.w;
    }
    uint16_t* dst = a.dw_router + h * a.E + e0;
#pragma unroll
    for (int u = 0; u < 8; ++u) hi[u] += lo[u];
    if (a.E % 8 == 0) {
      *reinterpret_cast<uint4*>(dst) = pack8(hi);
    } else {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (e0 + u < a.E) dst[u] = __bfloat16_as_ushort(__float2bfloat16_rn(hi[u]));
    }
  }
}

// One warp per token; lane l holds experts l, l + 32, ...
__global__ void __launch_bounds__(256) router_softmax_kernel(const float* logits, int S,
                                                             int ldl, const float* bias, int T,
                                                             int E, float* probs) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= T) return;
  float v[kMaxExperts / 32];
  float m = -INFINITY;
#pragma unroll
  for (int u = 0; u < kMaxExperts / 32; ++u) {
    const int e = lane + 32 * u;
    v[u] = -INFINITY;
    if (e < E) {
      v[u] = __ldg(logits + (size_t)t * ldl + e);
      for (int i = 1; i < S; ++i) v[u] += __ldg(logits + ((size_t)i * T + t) * ldl + e);
      if (bias) v[u] += __ldg(bias + e);
      if (isnan(v[u])) v[u] = -INFINITY;  // masked, as the route has it
    }
    m = fmaxf(m, v[u]);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  float s = 0.0f;
#pragma unroll
  for (int u = 0; u < kMaxExperts / 32; ++u) {
    v[u] = lane + 32 * u < E ? expf(v[u] - m) : 0.0f;
    s += v[u];
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
#pragma unroll
  for (int u = 0; u < kMaxExperts / 32; ++u) {
    const int e = lane + 32 * u;
    if (e < E) probs[(size_t)t * E + e] = v[u] / s;
  }
}

}  // namespace

template <int LPR>
static cudaError_t gather(const GatherArgs& a, int sms, cudaStream_t st) {
  const int planes = a.src[1] ? 2 : 1;
  const unsigned gx = blocks_for(a.seg.rows_pad, GTHREADS / LPR,
                                 (int64_t)(sms > 0 ? sms : 1) * (2048 / GTHREADS) / planes);
  return launch(train_gather_kernel<LPR>, dim3(gx, planes), GTHREADS, st, a);
}
cudaError_t launch_train_gather(const GatherArgs& a, int sms, cudaStream_t st) {
  return a.H >= 256 ? gather<32>(a, sms, st) : gather<8>(a, sms, st);
}

template <bool F32, bool PARTS>
static cudaError_t rows_sum(const RowsSumArgs& a, cudaStream_t st) {
  const int per = RTHREADS * 8 * (F32 ? 1 : 2);
  const dim3 grid((unsigned)a.T, (unsigned)((a.H + per - 1) / per), 1);
  if (a.k <= 1) return launch(rows_sum_kernel<1, F32, PARTS>, grid, RTHREADS, st, a);
  if (a.k <= 2) return launch(rows_sum_kernel<2, F32, PARTS>, grid, RTHREADS, st, a);
  if (a.k <= 4) return launch(rows_sum_kernel<4, F32, PARTS>, grid, RTHREADS, st, a);
  return launch(rows_sum_kernel<8, F32, PARTS>, grid, RTHREADS, st, a);
}
cudaError_t launch_rows_sum(const RowsSumArgs& a, cudaStream_t st) {
  if (!a.rows32) return rows_sum<false, false>(a, st);
  // (a loop over one part takes 15% longer than none)
  return a.splits > 1 || a.range ? rows_sum<true, true>(a, st) : rows_sum<true, false>(a, st);
}

template <int W>
static cudaError_t combine_backward_w(const CombineBackwardArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)((a.T + 4 / W - 1) / (4 / W)));
  if (a.k <= 1) return launch(combine_backward_kernel<1, W>, grid, 128, st, a);
  if (a.k <= 2) return launch(combine_backward_kernel<2, W>, grid, 128, st, a);
  if (a.k <= 4) return launch(combine_backward_kernel<4, W>, grid, 128, st, a);
  return launch(combine_backward_kernel<8, W>, grid, 128, st, a);
}
cudaError_t launch_combine_backward(const CombineBackwardArgs& a, cudaStream_t st) {
  return a.H <= 512 ? combine_backward_w<1>(a, st) : combine_backward_w<4>(a, st);
}

cudaError_t launch_quantize_a8(int64_t rows, int cols, const uint16_t* x, int8_t* codes, uint8_t* scales,
                               int sms, cudaStream_t st) {
  const int per_row = (int)(((int64_t)cols + 31) / 32 * 4);
  const int64_t chunks = rows * per_row;
  const unsigned g = blocks_for(chunks, QTHREADS * QILP, (int64_t)(sms > 0 ? sms : 1) * (2048 / QTHREADS) * 4);
  if (cols % 32 == 0) return launch(quantize_a8_kernel<true>, dim3(g), QTHREADS, st, chunks, per_row, cols, x, codes, scales);
  return launch(quantize_a8_kernel<false>, dim3(g), QTHREADS, st, chunks, per_row, cols, x, codes, scales);
}

cudaError_t launch_dequantize_a8(int64_t rows, int cols, const int8_t* codes, const uint8_t* scales,
                                 uint16_t* out, int sms, cudaStream_t st) {
  const int per_row = (int)(((int64_t)cols + 31) / 32 * 4);
  const int64_t chunks = rows * per_row;
  const unsigned g = blocks_for(chunks, QTHREADS * QILP, (int64_t)(sms > 0 ? sms : 1) * (2048 / QTHREADS) * 4);
  if (cols % 32 == 0)
    return launch(dequantize_a8_kernel<true>, dim3(g), QTHREADS, st, chunks, per_row, cols, codes, scales, out);
  return launch(dequantize_a8_kernel<false>, dim3(g), QTHREADS, st, chunks, per_row, cols, codes, scales, out);
}

cudaError_t launch_gate_backward(const GateBackwardArgs& a, cudaStream_t st) {
  const int64_t items = a.wt ? (int64_t)a.H / 8 * a.E : (int64_t)a.H * a.ep / 4;
  const unsigned grid = (unsigned)((a.T + kGateTokens - 1) / kGateTokens) + blocks_for(items, GATE_WARPS * 32, 512);
  return launch(gate_backward_kernel, dim3(grid), GATE_WARPS * 32, st, a);
}

cudaError_t launch_router_reduce(const RouterReduceArgs& a, cudaStream_t st) {
  const int db_blocks = a.db ? (a.E + SUM_THREADS / 32 - 1) / (SUM_THREADS / 32) : 0;
  const unsigned g = db_blocks + blocks_for((int64_t)a.H * a.ep / 8, SUM_THREADS, 1024);
  return launch(router_reduce_kernel, dim3(g), SUM_THREADS, st, a, db_blocks);
}

cudaError_t launch_router_softmax(const float* logits, int S, int ldl, const float* bias, int T, int E,
                                  float* probs, cudaStream_t st) {
  return launch(router_softmax_kernel, dim3((unsigned)((T + 7) / 8)), 256, st, logits, S, ldl, bias, T, E,
                probs);
}

}  // namespace moe
