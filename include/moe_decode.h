/*
 * moe_decode.h -- C ABI of the MoE layer's decode operators on GB300
 * (sm_103a), in the same library as moe.h and with its conventions: device
 * pointers owned by the caller (row-major, contiguous, 16-byte aligned), a
 * caller-owned workspace, calls that only enqueue work on `stream`, argument
 * checks on the host before anything is enqueued, MOE_OK or an MOE_ERR_*
 * code, moe_last_error_string() for the message and moe_get_device_status()
 * for the status word in the first bytes of a workspace.
 *
 *   moed_forward       the whole layer for a few tokens, bf16 experts
 *   moed_forward_q4    the same with 4-bit experts and group scales
 *   moed_matvec_q4     y[r] = x[r] W[e(r)] for a few rows grouped by expert,
 *                      W in 4 bits with group scales
 *   moed_quantize_q4   bf16 weights to 4 bits with group scales
 *   moed_dequantize_q4 and back (for the large products of a prompt)
 *
 * 4-bit weights.  A matrix W [E, K, N] is held as
 *   codes  [E, K/8, N] uint32: bits 4i .. 4i+3 of word (e, r, n) are the code
 *          c of row 8r + i, column n
 *   scales [E, K/group, N] bf16, one per column and `group` rows
 * and stands for W[e, kk, n] = (c - 8) * scales[e, kk / group, n], c in
 * 0..15.  group is 32, 64 or 128 and divides K; N is a multiple of 8.  Any
 * code and any scale (negative and zero ones too) may be passed; a product
 * uses (c - 8) and the scale as they are, without rounding their product.
 *
 * Limits (MOE_ERR_UNSUPPORTED beyond them): those of moe.h, and
 * T <= MOED_MAX_TOKENS for the layers, rows <= MOED_MAX_ROWS for the
 * products, H and F multiples of group for moed_forward_q4.
 */
#ifndef MOE_GB300_MOE_DECODE_H
#define MOE_GB300_MOE_DECODE_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOED_MAX_TOKENS 64
#define MOED_MAX_ROWS 512

/* Workspace bytes of moed_forward and moed_forward_q4 for the shape.
 * Returns 0 for a shape they do not take. */
MOE_API size_t moed_workspace_size(const moe_shape* s);

/*
 * The five steps of the layer (moe_forward) for T <= MOED_MAX_TOKENS tokens in
 * two kernels: one cluster of 8 CTAs routes and dispatches every token, then
 * a cooperative launch over all SMs streams the weights of the experts that
 * have rows, once, and combines.  Arguments and routing outputs as for
 * moe_forward (the same experts, weights, drops and order); the arithmetic
 * is moe_forward's except that the expert outputs are kept in fp32 until the
 * weighted sum (moe_forward rounds them to bf16 when k > 1).  h is rounded to
 * bf16.  The result does not depend on how the work is split over the SMs'
 * timing: the same inputs give the same bits.
 * Experts may be masked by a bias of -inf (a NaN logit counts as one): they
 * are chosen after all others, lower index first, with weight 0.  Where that
 * leaves a token no expert the softmax has no value: it goes to experts
 * 0 .. k-1, and its weights and its row of y are NaN.  All of this is
 * moe_forward's too.  Non-finite values of x stay in their token's row.
 * Calls on different streams may overlap if they share no workspace and no
 * output; host threads that call on one stream with one workspace have to
 * take turns (a call enqueues two kernels).  y may be x.  T = 0 clears counts / offsets, as moe_forward does.
 */
MOE_API int moed_forward(const moe_shape* s, const uint16_t* x, const uint16_t* w_router,
                         const float* b_router, const uint16_t* w1, const uint16_t* w2,
                         uint16_t* y, int32_t* ids, float* weights, int32_t* counts,
                         int32_t* offsets, int32_t* perm, int32_t* slot, void* ws,
                         size_t ws_bytes, void* stream);

/*
 * moed_forward with both expert matrices in 4 bits: w1 codes [E, H/8, F]
 * (or [E, H/8, 2F] = gate | up for MOE_EXPERT_SWIGLU) and scales
 * [E, H/group, F or 2F]; w2 codes [E, F/8, H] and scales [E, F/group, H].
 */
MOE_API int moed_forward_q4(const moe_shape* s, int32_t group, const uint16_t* x,
                            const uint16_t* w_router, const float* b_router,
                            const uint32_t* w1_codes, const uint16_t* w1_scales,
                            const uint32_t* w2_codes, const uint16_t* w2_scales, uint16_t* y,
                            int32_t* ids, float* weights, int32_t* counts, int32_t* offsets,
                            int32_t* perm, int32_t* slot, void* ws, size_t ws_bytes,
                            void* stream);

/*
 * Self-test of the streaming kernel's bounded waits, beside
 * moe_selftest_wait_timeout: the layer (group = 0: bf16 weights, no scales;
 * else as moed_forward_q4) with waits of at most limit_ns nanoseconds
 * (1e3 .. 1e9), between its products for one CTA more than there are.  Those
 * waits run out, every CTA gives up and leaves, and MOE_DEV_TIMEOUT is set in
 * the workspace's status word (not in a call without rows, which does not
 * wait: T = 0, or every assignment dropped).  The routing outputs are the
 * layer's, y is void; the next call with the workspace is an ordinary one.
 * Nothing traps or hangs.
 */
MOE_API int moed_selftest_wait_timeout(const moe_shape* s, int32_t group, const uint16_t* x,
                                       const uint16_t* w_router, const float* b_router,
                                       const void* w1, const uint16_t* w1_scales, const void* w2,
                                       const uint16_t* w2_scales, uint16_t* y, int32_t* ids,
                                       float* weights, int32_t* counts, int32_t* offsets,
                                       int32_t* perm, int32_t* slot, void* ws, size_t ws_bytes,
                                       uint64_t limit_ns, void* stream);

/* Workspace bytes of moed_matvec_q4; 0 for sizes it does not take. */
MOE_API size_t moed_matvec_q4_workspace_size(int32_t rows, int32_t n_segments, int32_t K,
                                             int32_t N);

/*
 * y[r] = x[r] W[i % E] for the rows r of segment i, seg_offsets[i] <= r <
 * seg_offsets[i+1] (as in moe_expert_ffn); fp32 sums, y rounded to bf16 once.
 *   x [rows, K] bf16, codes [E, K/8, N], scales [E, K/group, N],
 *   seg_offsets [n_segments+1] int32 (device, non-decreasing, at most rows;
 *   clamped to [0, rows] and to the largest before them, never followed out of
 *   range: a row belongs to the first segment that reaches it) or NULL with
 *   n_segments = 1: all rows, 1 <= n_segments <= 256, y [rows, N] bf16, which
 *   must not overlap x; rows of y outside every segment are not written.
 * rows = 0 enqueues nothing but the status clear.
 */
MOE_API int moed_matvec_q4(int32_t rows, int32_t K, int32_t N, int32_t E, int32_t group,
                           int32_t n_segments, const uint16_t* x, const uint32_t* codes,
                           const uint16_t* scales, const int32_t* seg_offsets, uint16_t* y,
                           void* ws, size_t ws_bytes, void* stream);

/*
 * w [E, K, N] bf16 -> codes, scales.  Per group and column: scale =
 * bf16(max|w| / 7), c - 8 = round(w / scale) to nearest, ties to even,
 * clamped to [-8, 7]; a scale of zero gives codes of zero (c = 8).  A group
 * that holds a NaN gets a NaN scale and one that holds an infinity an
 * infinite scale, so that its products are not finite.  No workspace.
 */
MOE_API int moed_quantize_q4(int32_t E, int32_t K, int32_t N, int32_t group, const uint16_t* w,
                             uint32_t* codes, uint16_t* scales, void* stream);

/* w[e, kk, n] = bf16((c - 8) * scale), rounded once.  No workspace. */
MOE_API int moed_dequantize_q4(int32_t E, int32_t K, int32_t N, int32_t group,
                               const uint32_t* codes, const uint16_t* scales, uint16_t* w,
                               void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_MOE_DECODE_H */
