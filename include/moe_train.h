/*
 * moe_train.h -- C ABI of the training operators of the GB300 MoE layer: the
 * gradients of every step of moe.h's forward, the layer's forward that keeps
 * what they need, and activations kept in 8 bits.
 *
 * The forward is moe.h's (same routing, dispatch order, capacity, activation
 * and combine; see there).  With dy the gradient of y, row r = slot[t, j] the
 * kept assignment of token t's j-th expert, w its gate weight and e its
 * expert:
 *   g[r]   = dy[t] W2[e]^T
 *   dw[t,j] = <g[r], h[r]>           (0 for a dropped assignment)
 *   dz[r]  = w g[r] act'(z[r])
 *   dW2[e] = sum_r (w h[r])^T dy[t]  dW1[e] = sum_r x[t]^T dz[r]
 *   dx[t]  = sum_j dz[slot[t,j]] W1[e]^T + dlogits[t] W_router^T
 *   dW_router = x^T dlogits          db = sum_t dlogits[t]
 * with S = sum_j w[t,j] dw[t,j] and
 *   MOE_GATE_TOPK_SOFTMAX, ..._RENORM: dlogits of the j-th chosen expert =
 *     w[t,j] (dw[t,j] - S), 0 for the others;
 *   MOE_GATE_SOFTMAX_TOPK: dlogits[e] = p[t,e] ([e chosen] dw - S).
 * The choice of the experts and of what a capacity drops is not differentiated.
 * h and act' come from the KEPT z: with act GELU (erf form) z = x W1, with
 * SwiGLU z = (x W_gate, x W_up).
 *
 * Precision: bf16 operands, fp32 accumulation and epilogues; w h and dz are
 * rounded to bf16 once, as the tensor cores' operands, and so is the forward's
 * h; dlogits travel as two bf16 numbers (16 bits and the rest); expert outputs
 * and their rows' gradients stay in fp32 inside a layer's call; every output is
 * rounded once.  No
 * atomics: results do not depend on timing.
 *
 * Conventions are moe.h's (device pointers, 16-byte aligned, row-major and
 * contiguous, caller's stream, nothing allocated, checked on the host before
 * anything is enqueued, T = 0 accepted), with these differences:
 *   - `status` is a caller's device block of at least MOE_WS_MIN_BYTES, zero
 *     before its first use: calls set bits in its first word and never clear
 *     them; moe_get_device_status(status, ...) reads and clears it.
 *   - `ws` holds nothing before or after a call.
 *   - H <= 2^25 and F <= 2^29 (MOE_ERR_UNSUPPORTED).
 *   - What a call writes (outputs, status, ws) must not overlap what it reads,
 *     nor one output another: refused with MOE_ERR_INVALID_ARG.
 *   - offsets, perm, slot and ids are a dispatch's (moe_route, moe_dispatch);
 *     entries outside their range are not followed outside a buffer, and
 *     offsets that are not ascending within [0, T*k] set MOE_DEV_BAD_ID.
 */
#ifndef MOE_GB300_MOE_TRAIN_H
#define MOE_GB300_MOE_TRAIN_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Activations in 8 bits.  x [rows, cols] bf16 <-> codes [rows, cols] int8 and
 * scales [rows, ceil(cols / 32)] bytes: 32 columns (the last group of a row may
 * hold fewer) share the scale 2^(b - 127), the smallest power of two with
 * max |x| <= 127 * 2^(b - 127) and b >= 1; a code is x / scale rounded half to
 * even.  In a group of the largest scale that bf16 needs (b = 249) codes stay
 * within 63, as 64 of them would be infinite.  A group that holds an infinity
 * or a NaN has b = 255, codes 0, and stands for 32 NaN.  code * scale is exact
 * in bf16, so products take kept values as they are; the error is at most half
 * a scale: 1/127 of the group's largest magnitude (more only below 2^-119,
 * where b = 1, and up to a whole scale with b = 249).
 * cols % 8 == 0; rows * cols < 2^46.
 */
MOE_API int moet_quantize_a8(int64_t rows, int32_t cols, const uint16_t* x, int8_t* codes,
                             uint8_t* scales, void* stream);
MOE_API int moet_dequantize_a8(int64_t rows, int32_t cols, const int8_t* codes,
                               const uint8_t* scales, uint16_t* out, void* stream);

/*
 * The gradient of moe_dispatch_rows: dx[t] = sum over kept slots j of
 * dxp[slot[t, j]] (fp32 in slot order, rounded to bf16).  s: T, H, E, k.
 */
MOE_API int moet_dispatch_rows_backward(const moe_shape* s, const uint16_t* dxp, const int32_t* slot,
                                        uint16_t* dx, void* stream);

/*
 * The gradients of moe_combine: dY[slot[t, j]] = weights[t, j] * dy[t] and
 * dweights[t, j] = <dy[t], Y[slot[t, j]]> (fp32; 0 for a dropped slot).
 * Y, dY [T*k, H]; rows of dY that no slot names are not written.
 */
MOE_API int moet_combine_backward(const moe_shape* s, const uint16_t* dy, const uint16_t* Y,
                                  const float* weights, const int32_t* slot, uint16_t* dY,
                                  float* dweights, void* stream);

/*
 * moe_expert_ffn (one segment per expert: rows [offsets[e], offsets[e+1]) of
 * xp) that also keeps z for the backward pass.
 *   keep_bits 16: z bf16 [T*k, F] (SwiGLU [T*k, 2, F]), z_scales ignored
 *   keep_bits  8: z int8 codes of that shape, z_scales [T*k, (2,) ceil(F/32)],
 *                 rounded from the fp32 accumulators
 * Rows outside every segment are not written.
 */
MOE_API size_t moet_expert_ffn_workspace_size(const moe_shape* s);
MOE_API int moet_expert_ffn(const moe_shape* s, int32_t keep_bits, const uint16_t* xp,
                            const uint16_t* w1, const uint16_t* w2, const int32_t* offsets,
                            uint16_t* Y, void* z, uint8_t* z_scales, void* status, void* ws,
                            size_t ws_bytes, void* stream);

/*
 * The gradients of that call: from dY [T*k, H], dxp [T*k, H] (rows outside
 * every segment are not written), dw1 and dw2 as w1 and w2 (zeros for an expert
 * without rows).
 */
MOE_API size_t moet_expert_ffn_backward_workspace_size(const moe_shape* s);
MOE_API int moet_expert_ffn_backward(const moe_shape* s, int32_t keep_bits, const uint16_t* xp,
                                     const void* z, const uint8_t* z_scales, const uint16_t* w1,
                                     const uint16_t* w2, const int32_t* offsets, const uint16_t* dY,
                                     uint16_t* dxp, uint16_t* dw1, uint16_t* dw2, void* status,
                                     void* ws, size_t ws_bytes, void* stream);

/*
 * probs [T, E] fp32 = softmax(x W_router + b_router) over all experts, what
 * MOE_GATE_SOFTMAX_TOPK's gradient needs of the forward.  As in the route a
 * logit of -inf or NaN masks its expert (probability 0); a token whose logits
 * all do has NaN.
 */
MOE_API size_t moet_router_probs_workspace_size(const moe_shape* s);
MOE_API int moet_router_probs(const moe_shape* s, const uint16_t* x, const uint16_t* w_router,
                              const float* b_router, float* probs, void* status, void* ws,
                              size_t ws_bytes, void* stream);

/*
 * The gradients of the router and the gate from dweights [T, k]: dx [T, H]
 * (the router's part alone), dw_router [H, E] bf16, db [E] fp32 or null.
 * probs is read for MOE_GATE_SOFTMAX_TOPK only (else it may be null).
 */
MOE_API size_t moet_route_backward_workspace_size(const moe_shape* s);
MOE_API int moet_route_backward(const moe_shape* s, const uint16_t* x, const uint16_t* w_router,
                                const int32_t* ids, const float* weights, const float* probs,
                                const float* dweights, uint16_t* dx, uint16_t* dw_router, float* db,
                                void* status, void* ws, size_t ws_bytes, void* stream);

/*
 * The layer's forward for training: moe_forward's outputs, z (as
 * moet_expert_ffn), with keep_bits 8 also x in 8 bits (xk [T, H] codes,
 * xk_scales; else ignored) and with MOE_GATE_SOFTMAX_TOPK probs (else ignored).
 * y may differ from moe_forward's by roundings: expert outputs are not rounded to
 * bf16 before they are combined.
 */
MOE_API size_t moet_forward_workspace_size(const moe_shape* s);
MOE_API int moet_forward(const moe_shape* s, int32_t keep_bits, const uint16_t* x,
                         const uint16_t* w_router, const float* b_router, const uint16_t* w1,
                         const uint16_t* w2, uint16_t* y, int32_t* ids, float* weights,
                         int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* slot, void* z,
                         uint8_t* z_scales, int8_t* xk, uint8_t* xk_scales, float* probs,
                         void* status, void* ws, size_t ws_bytes, void* stream);

/*
 * Every gradient of that call: x is bf16 (keep_bits 16) or its codes with
 * x_scales; db may be null.  y and the experts' outputs are not needed.
 */
MOE_API size_t moet_backward_workspace_size(const moe_shape* s, int32_t keep_bits);
MOE_API int moet_backward(const moe_shape* s, int32_t keep_bits, const uint16_t* dy, const void* x,
                          const uint8_t* x_scales, const uint16_t* w_router, const uint16_t* w1,
                          const uint16_t* w2, const int32_t* ids, const float* weights,
                          const int32_t* offsets, const int32_t* perm, const int32_t* slot,
                          const void* z, const uint8_t* z_scales, const float* probs, uint16_t* dx,
                          uint16_t* dw_router, float* db, uint16_t* dw1, uint16_t* dw2, void* status,
                          void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_MOE_TRAIN_H */
