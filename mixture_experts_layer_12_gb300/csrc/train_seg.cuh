// train_seg.cuh -- the segment table every training kernel builds from the
// dispatch offsets, and the 8-bit format's arithmetic.
#pragma once

#include "tc_common.cuh"
#include "train_internal.h"

namespace moe {

// Row segments in shared memory: compact and padded first rows, lengths.
struct SegTable {
  int row_off[kMaxExperts];
  int rows[kMaxExperts];
  int pad_off[kMaxExperts + 1];
};

// One warp: the table, and tile_start[0 .. E] = exclusive sums of
// tiles_of(rows).  E <= 256: lane l holds segments 8 l .. 8 l + 7.  Offsets that
// had to be cut set MOE_DEV_BAD_ID in *status.
template <typename F>
__device__ __forceinline__ void seg_scan(const SegArgs& s, SegTable& t, int* tile_start, int lane,
                                         int* status, F tiles_of) {
  int n[8], o[8];
  int pad_sum = 0;
  bool bad = false;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int e = lane * 8 + u;
    n[u] = 0;
    o[u] = 0;
    if (e < s.E) {
      int hi;
      if (s.offsets) {
        const int o0 = __ldg(s.offsets + e), o1 = __ldg(s.offsets + e + 1);
        o[u] = min(max(o0, 0), s.rows);
        hi = min(o1, s.rows);
        bad |= o0 < 0 || o1 < o0 || o1 > s.rows;
      } else {
        o[u] = (int)min((long long)e * s.chunk, (long long)s.rows);
        hi = (int)min((long long)o[u] + s.chunk, (long long)s.rows);
      }
      n[u] = max(hi - o[u], 0);
    }
    pad_sum += (n[u] + kSegPad - 1) / kSegPad * kSegPad;
  }
  // rows of all segments together may pass int's range for offsets that run
  // back and forth: saturating sums
  int incl = pad_sum < 0 ? 0x7fffffff : pad_sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl = (int)min((long long)incl + y, 0x7fffffffll);
  }
  int run = __shfl_up_sync(0xffffffffu, incl, 1);
  if (lane == 0) run = 0;
  int tsum = 0;
  int tn[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int e = lane * 8 + u;
    tn[u] = 0;
    if (e < s.E) {
      const long long end = (long long)run + (n[u] + kSegPad - 1) / kSegPad * kSegPad;
      if (end > s.rows_pad) {  // overlapping segments: nothing past the buffers
        n[u] = 0;
        bad = true;
      }
      t.row_off[e] = o[u];
      t.rows[e] = n[u];
      t.pad_off[e] = min(run, s.rows_pad);
      run = (int)min(end, 0x7fffffffll);
      tn[u] = tiles_of(n[u]);
      if (e == s.E - 1) t.pad_off[s.E] = min(run, s.rows_pad);
    }
    tsum += tn[u];
  }
  if (bad) record_status(status, MOE_DEV_BAD_ID);
  if (!tile_start) return;
  int ti = tsum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, ti, off);
    if (lane >= off) ti += y;
  }
  int tr = ti - tsum;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int e = lane * 8 + u;
    if (e < s.E) tile_start[e] = tr;
    tr += tn[u];
  }
  if (lane == 31) tile_start[s.E] = ti;
}

// ---- activations in 8 bits (include/moe_train.h): groups of 32 share the
// power of two 2^(b - 127), the smallest with max |v| <= 127 * 2^(b - 127).
// 127 = 1.984375 * 2^6, so with max |v| = m * 2^x (1 <= m < 2) the exponent is
// x - 6, or x - 5 for m > 1.984375 (mantissa field above 0x7e0000): adding
// 0x1ffff to the bits carries into the exponent in just that case.
__device__ __forceinline__ uint32_t a8_scale_byte(uint32_t abs_max_bits) {
  if (abs_max_bits >= 0x7f800000u) return 255u;  // an infinity or a NaN
  const int b = (int)((abs_max_bits + 0x1ffffu) >> 23) - 6;
  return (uint32_t)max(b, 1);
}
// 1 / scale, exact (b = 255: 0, so that the group's codes are 0 or dropped)
__device__ __forceinline__ float a8_inverse(uint32_t b) {
  return b == 255u ? 0.0f : __uint_as_float((254u - b) << 23);
}
// half to even; a group of the largest exponent keeps |code| <= 63, as
// 64 * 2^122 is not finite
__device__ __forceinline__ int a8_code(float v, float inv, uint32_t b) {
  const int lim = b == 249u ? 63 : 127;
  if (b == 255u) return 0;
  return min(max(__float2int_rn(v * inv), -lim), lim);
}
__device__ __forceinline__ float a8_scale(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7fc00000u : b == 0u ? 0x00400000u : b << 23);
}
// Four codes of a word as floats times s: a byte under the exponent of 2^23 is
// 2^23 + 128 + code once its sign bit is turned, and needs no conversion.
__device__ __forceinline__ void a8_values(uint32_t w, float s, float* f) {
  const uint32_t u = w ^ 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = (__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 | i)) - 8388736.0f) * s;
}
// 8 values as codes.  v / scale is exact and at most 127, so adding 1.5 * 2^23
// rounds it half to even into the low byte; only a scale byte of 249 or more
// (the largest magnitudes, infinities, NaN) needs limits.
__device__ __forceinline__ uint2 a8_codes8(const float* v, float inv, uint32_t b) {
  uint32_t t[8];
  if (b < 249u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = __float_as_uint(fmaf(v[i], inv, 12582912.0f));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = (uint32_t)a8_code(v[i], inv, b);
  }
  uint2 q;
  q.x = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
  q.y = __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410);
  return q;
}

}  // namespace moe
