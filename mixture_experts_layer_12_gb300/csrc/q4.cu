// q4.cu -- bf16 weights to 4-bit codes with group scales, and back (the
// layout is described in moe_decode.h).
//
// quantize: per group of `group` rows and per column, scale = bf16(max|w| / 7)
// and c - 8 = round(w / scale), ties to even.  Bound by memory: 2 bytes in and
// about 0.53 out per weight, read once.  A warp takes one group of 32 columns
// (64 for groups of 32): 8 (4) lanes share the rows of 8 columns, so every load
// is 16 bytes, the lanes of a warp take 64 (128) bytes of a row, a lane holds
// its group/8 rows in registers and the maximum is 3 (2) shuffles away.  With
// 64 columns for groups of 128 a lane held twice as much and too few warps were
// left on an SM to load while others convert.
//
// The division has to round as the exact quotient does, without costing a
// division per weight.  w and scale have 8-bit mantissas, so a quotient that is
// not a tie (n + 1/2) is at least 1/510 away from one: (2 w - (2n + 1) scale) /
// (2 scale) with integers above and at most 510 below.  w * (1 / scale) is
// within 2^-20 of the quotient, |quotient| <= 7.03, and its rounding to fp16
// moves by at most 2^-9 = 1/512 to a multiple of 2^-8 (or of a finer step), of
// which ties are some: ties come back to the tie and nothing else reaches one,
// since 1/510 - 1/512 > 2^-20.  One fp16 addition for two weights then rounds to
// integers: 6 instructions per weight, where fp32 took 8.  Scales below 2^-100 (where
// 1 / scale may overflow) take the division.
//
// Measured for 4 x 4096 x 14336 in groups of 128: 95 us, 6.2 TB/s (115 us with 64
// columns to a warp and fp32 rounding).
//
// dequantize: w = bf16((c - 8) * scale): the product of 4 and 8 bits is exact
// in fp32, so one bf16 multiply rounds it once.  Bound by the 2 bytes written
// per weight: the same matrices take 86 us, 6.9 TB/s.
#include <cuda_fp16.h>
#include <math.h>

#include "decode_internal.h"
#include "tc_common.cuh"

namespace moe {
namespace {

constexpr int Q_THREADS = 128;

__device__ __forceinline__ uint32_t abs_max_u16x2(uint32_t a, uint32_t b) {
  return __vmaxu2(a, b & 0x7FFF7FFFu);
}

// The code of x by the division itself: scales where 1 / scale may overflow,
// infinities and NaN (whose code is 0).  Out of line: it is hardly ever taken.
__device__ __noinline__ uint32_t code_by_division(float x, float s) {
  const float q = s > 0.f ? x / s : 0.f;
  return (uint32_t)(int)(rintf(fminf(fmaxf(q, -8.f), 7.f)) + 8.f);
}

// SUBS: lanes that share the group's rows; NB: 8-row blocks per lane
template <int NB, int SUBS>
__global__ void __launch_bounds__(Q_THREADS)
    quantize_kernel(const uint16_t* __restrict__ w, uint32_t* __restrict__ codes,
                    uint16_t* __restrict__ scales, int N, int col_tiles, long long warps) {
  const int lane = threadIdx.x & 31;
  const long long wid = (long long)blockIdx.x * (Q_THREADS / 32) + (threadIdx.x >> 5);
  pdl_launch_dependents();
  pdl_wait();
  if (wid >= warps) return;
  const long long grp = wid / col_tiles;  // group of rows, over all experts
  constexpr int CHUNKS = 32 / SUBS;
  const int col = ((int)(wid - grp * col_tiles) * CHUNKS + lane % CHUNKS) * 8;
  const int sub = lane / CHUNKS;
  const bool in = col < N;                // N % 8 == 0: all 8 columns or none
  const long long row0 = grp * (NB * SUBS * 8);

  uint4 v[NB][8];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      v[b][r] = make_uint4(0, 0, 0, 0);
      if (in)
        v[b][r] = __ldcs(reinterpret_cast<const uint4*>(
            w + (size_t)(row0 + (b * SUBS + sub) * 8 + r) * N + col));
    }
  // largest |w| per column as bf16 bits: unsigned order puts infinities above
  // all finite values and NaN above those
  uint32_t mx[4] = {0, 0, 0, 0};
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      mx[0] = abs_max_u16x2(mx[0], v[b][r].x);
      mx[1] = abs_max_u16x2(mx[1], v[b][r].y);
      mx[2] = abs_max_u16x2(mx[2], v[b][r].z);
      mx[3] = abs_max_u16x2(mx[3], v[b][r].w);
    }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int o = CHUNKS; o < 32; o *= 2) mx[i] = __vmaxu2(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
  if (!in) return;
  float s[8], inv[8];
  uint32_t sp[4];
  bool slow = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sp[i] = pack_bf16x2(bf16_lo(mx[i]) / 7.0f, bf16_hi(mx[i]) / 7.0f);
    s[2 * i] = bf16_lo(sp[i]);
    s[2 * i + 1] = bf16_hi(sp[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    inv[i] = s[i] > 0.f ? 1.0f / s[i] : 0.f;  // a zero scale gives codes of zero
    slow |= !(s[i] == 0.f || (s[i] > 7.888609e-31f && s[i] < INFINITY));  // 2^-100
  }
  if (sub == 0)
    *reinterpret_cast<uint4*>(scales + (size_t)grp * N + col) = make_uint4(sp[0], sp[1], sp[2], sp[3]);

#pragma unroll
  for (int b = 0; b < NB; ++b) {
    uint32_t word[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (!slow) {
      // Rows r and r + 4 as a pair of fp16, whose step below 8 is at most 2^-8;
      // adding 1.5 * 2^10 then rounds both to integers, ties to even, and leaves
      // them in the low bits.  |w / scale| is at most 7.03 here (scale is within
      // 2^-8 of max|w| / 7): no clamp.  (word << 4) + bits sums
      // sum_r (0x6600 + c_r - 8) 16^r over both halves; the constant part is
      // taken off at the end.
      constexpr uint32_t kOff = 0x1111u * 0x66006600u - 0x88888888u;
#pragma unroll
      for (int r = 3; r >= 0; --r) {
        const uint32_t lo[4] = {v[b][r].x, v[b][r].y, v[b][r].z, v[b][r].w};
        const uint32_t hi[4] = {v[b][r + 4].x, v[b][r + 4].y, v[b][r + 4].z, v[b][r + 4].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = (i & 1) ? bf16_hi(lo[i >> 1]) : bf16_lo(lo[i >> 1]);
          const float z = (i & 1) ? bf16_hi(hi[i >> 1]) : bf16_lo(hi[i >> 1]);
          const __half2 q = __hadd2(__floats2half2_rn(x * inv[i], z * inv[i]), __float2half2_rn(1536.f));
          word[i] = (word[i] << 4) + *reinterpret_cast<const uint32_t*>(&q);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) word[i] -= kOff;
    } else {
#pragma unroll
      for (int r = 7; r >= 0; --r) {
        const uint32_t w4[4] = {v[b][r].x, v[b][r].y, v[b][r].z, v[b][r].w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          word[i] = (word[i] << 4) +
                    code_by_division((i & 1) ? bf16_hi(w4[i >> 1]) : bf16_lo(w4[i >> 1]), s[i]);
      }
    }
    uint32_t* dst = codes + ((size_t)(row0 / 8) + b * SUBS + sub) * N + col;
    *reinterpret_cast<uint4*>(dst) = make_uint4(word[0], word[1], word[2], word[3]);
    *reinterpret_cast<uint4*>(dst + 4) = make_uint4(word[4], word[5], word[6], word[7]);
  }
}

constexpr int DQ_THREADS = 256;

// codes i and i + 4 of a word times the column's scale, as a bf16 pair
template <int I>
__device__ __forceinline__ uint32_t deq_pair(uint32_t v, __nv_bfloat162 s) {
  const uint32_t p = ((v >> (4 * I)) & 0x000F000Fu) | 0x43004300u;  // 128 + c
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&p),
                                   __floats2bfloat162_rn(136.f, 136.f));
  const __nv_bfloat162 r = __hmul2(d, s);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// One thread: 8 columns of one row of code words (8 rows of w).
__global__ void __launch_bounds__(DQ_THREADS)
    dequantize_kernel(const uint32_t* __restrict__ codes, const uint16_t* __restrict__ scales,
                      uint16_t* __restrict__ w, int N, int words_per_group, long long n) {
  pdl_launch_dependents();
  pdl_wait();
  const long long i = (long long)blockIdx.x * DQ_THREADS + threadIdx.x;
  if (i >= n) return;
  const int cols = N / 8;
  const long long kr = i / cols;  // row of code words, over all experts
  const int col = (int)(i - kr * cols) * 8;
  const uint4 ca = __ldcs(reinterpret_cast<const uint4*>(codes + (size_t)kr * N + col));
  const uint4 cb = __ldcs(reinterpret_cast<const uint4*>(codes + (size_t)kr * N + col + 4));
  const uint4 sc = __ldg(reinterpret_cast<const uint4*>(scales + (size_t)(kr / words_per_group) * N + col));
  const uint32_t cw[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
  const uint32_t sw[4] = {sc.x, sc.y, sc.z, sc.w};
  uint32_t out[8][4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {  // columns 2c and 2c + 1
    const uint32_t s0 = __byte_perm(sw[c], 0, 0x1010), s1 = __byte_perm(sw[c], 0, 0x3232);
    const __nv_bfloat162 sa = *reinterpret_cast<const __nv_bfloat162*>(&s0);
    const __nv_bfloat162 sb = *reinterpret_cast<const __nv_bfloat162*>(&s1);
    const uint32_t a = cw[2 * c], b = cw[2 * c + 1];
    const uint32_t pa[4] = {deq_pair<0>(a, sa), deq_pair<1>(a, sa), deq_pair<2>(a, sa), deq_pair<3>(a, sa)};
    const uint32_t pb[4] = {deq_pair<0>(b, sb), deq_pair<1>(b, sb), deq_pair<2>(b, sb), deq_pair<3>(b, sb)};
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      out[r][c] = __byte_perm(pa[r], pb[r], 0x5410);
      out[r + 4][c] = __byte_perm(pa[r], pb[r], 0x7632);
    }
  }
#pragma unroll
  for (int r = 0; r < 8; ++r)
    *reinterpret_cast<uint4*>(w + (size_t)(kr * 8 + r) * N + col) =
        make_uint4(out[r][0], out[r][1], out[r][2], out[r][3]);
}

template <typename... KArgs, typename... Args>
cudaError_t q4_launch(void (*kern)(KArgs...), long long blocks, int threads, cudaStream_t st,
                      Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  set_pdl_attr(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

cudaError_t launch_quantize_q4(int E, int K, int N, int group, const uint16_t* w, uint32_t* codes,
                               uint16_t* scales, cudaStream_t st) {
  const int cols = group == 32 ? 64 : 32;  // columns of a warp
  const int tiles = (N + cols - 1) / cols;
  const long long warps = (long long)E * (K / group) * tiles;
  const long long blocks = (warps + Q_THREADS / 32 - 1) / (Q_THREADS / 32);
  switch (group) {
    case 32: return q4_launch(quantize_kernel<1, 4>, blocks, Q_THREADS, st, w, codes, scales, N, tiles, warps);
    case 64: return q4_launch(quantize_kernel<1, 8>, blocks, Q_THREADS, st, w, codes, scales, N, tiles, warps);
    default: return q4_launch(quantize_kernel<2, 8>, blocks, Q_THREADS, st, w, codes, scales, N, tiles, warps);
  }
}

cudaError_t launch_dequantize_q4(int E, int K, int N, int group, const uint32_t* codes,
                                 const uint16_t* scales, uint16_t* w, cudaStream_t st) {
  const long long n = (long long)E * (K / 8) * (N / 8);
  const long long blocks = (n + DQ_THREADS - 1) / DQ_THREADS;
  return q4_launch(dequantize_kernel, blocks, DQ_THREADS, st, codes, scales, w, N, group / 8, n);
}

}  // namespace moe
