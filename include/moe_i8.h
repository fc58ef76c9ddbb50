/* moe_i8.h — operators of libmoe on 8-bit whole numbers: matrix products, the
 * expert stage and the few-token layer on weights with one scale per output
 * channel, beside those of moe_serve.h.
 *
 * The conventions of moe.h and moe_serve.h hold here too: device pointers to
 * dense row-major arrays, int32 indices, caller-owned buffers, nothing
 * allocated, nothing synchronised, every argument checked on the host before any
 * HIP call, results deterministic. Arrays of no rows (rows or M of 0) may be
 * NULL; nothing is done then. Every other array starts at a multiple of 16 bytes
 * (MOE_EINVAL otherwise where the kernels depend on it).
 *
 *   prefill: moe_forward_fused_i8 = moe_route -> moe_experts_i8
 *            moe_experts_i8 = moe_permute_fused -> moe_quantize_i8_rows (x) ->
 *              moe_gemm_gate_up_i8 -> the down product -> the per-token sum
 *   decode:  moe_forward_few_i8
 */
#ifndef MOE_I8_H_
#define MOE_I8_H_

#include "moe_serve.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- 8-bit integer operands. Codes are whole numbers; a row of the reduction
 * axis (a token; an output channel of a weight) shares one float32 scale. With
 * amax the row's largest magnitude,
 *   scale = amax / 127,   code = the whole number nearest to 127 v / amax, halves to even
 * (0 and 0 for a row of zeros); the codes are those of exact arithmetic. A row
 * with a NaN or an infinity has scale NaN and codes 0: what is computed from it
 * is NaN. */

/* Rows [rows, K] of bf16 -> codes q [rows, K] and scale [rows]. Weights are
 * quantised once with the same call: w_gate, w_up [E,I,H] as E*I rows, w_down
 * [E,H,I] as E*H rows. rows >= 0 and K > 0, K % 8 == 0 (MOE_EINVAL otherwise);
 * rows below 2^28 - 16, for K > 512 2^26 - 4, for K > 2048 2^24 - 1
 * (MOE_EUNSUPPORTED otherwise). */
moe_status moe_quantize_i8_rows(int32_t rows, int32_t K, const void* in, int8_t* q, float* scale, hipStream_t stream);

/* Grouped product: for each expert e and row p in [offsets[e], offsets[e+1]),
 *   out[p,n] = bf16(row_weight[p] a_scale[p] w_scale[e,n] sum_k aq[p,k] wq[e,n,k])
 * with exact sums, rounded to fp32 once. aq [M,K], a_scale [M], wq [E,N,K],
 * w_scale [E,N], out [M,N] bf16. Codes may be any in [-128, 127]. offsets,
 * row_weight and rows outside the experts' as moe_gemm_fp8_block.
 * 0 <= M < 2^30; N % 8 == 0, K % 16 == 0, K < 2^17 (the sums' range), E <= 1024,
 * N K and 512 N below 2^31 (MOE_EUNSUPPORTED otherwise). */
moe_status moe_gemm_i8(int32_t M, int32_t E, int32_t N, int32_t K, const int8_t* aq, const float* a_scale,
                       const int32_t* offsets, const int8_t* wq, const float* w_scale, const float* row_weight, void* out,
                       hipStream_t stream);

/* Bytes of workspace of the three calls below (0 for a shape they reject): the
 * sort's counts, and silu(g) u in 24 bits between product and codes. */
size_t moe_i8_workspace_bytes(moe_shape s);

/* Gathered gate/up GEMM with the SwiGLU epilogue, its result quantised per row:
 *   v = silu(g) * u,  g = deq(xq[row_token[p]]) deq(Wg[e])^T, u likewise,
 *   aq [T*k,I], a_scale [T*k]: v's codes. In between v is held in 24 bits of its
 *   largest magnitude in 128 columns.
 * offsets and rows outside the experts' as moe_gemm_fp8_block.
 * xq [T,H], x_scale [T]; wq_gate, wq_up [E,I,H] with scales [E,I]. The shape
 * limits of moe_gemm_gate_up_fp8_block, and H and I below 2^17, T k I below 2^35
 * - 2048 (MOE_EUNSUPPORTED otherwise). ws of ws_bytes >= moe_i8_workspace_bytes(s),
 * at a multiple of 16 bytes. */
moe_status moe_gemm_gate_up_i8(moe_shape s, const int8_t* xq, const float* x_scale, const int32_t* row_token,
                               const int32_t* offsets, const int8_t* wq_gate, const float* w_gate_scale,
                               const int8_t* wq_up, const float* w_up_scale, int8_t* aq, float* a_scale, void* ws,
                               size_t ws_bytes, hipStream_t stream);

/* moe_experts_fp8_block on 8-bit integer weights: moe_permute_fused,
 * moe_quantize_i8_rows (x), moe_gemm_gate_up_i8, the down product (wq_down
 * [E,H,I], scales [E,H]) and the per-token sum; o_perm as there. */
moe_status moe_experts_i8(moe_shape s, const void* x, const int32_t* topk_idx, const float* topk_w,
                          const int8_t* wq_gate, const float* w_gate_scale, const int8_t* wq_up, const float* w_up_scale,
                          const int8_t* wq_down, const float* w_down_scale, int32_t* counts, int32_t* offsets,
                          int32_t* sorted_to_flat, int32_t* flat_to_sorted, int32_t* row_token, float* row_weight,
                          int8_t* xq, float* x_scale, int8_t* aq, float* a_scale, void* o_perm, void* y, void* ws,
                          size_t ws_bytes, hipStream_t stream);

/* moe_route (logits, topk_idx, topk_w), then moe_experts_i8. */
moe_status moe_forward_fused_i8(moe_shape s, const void* x, const void* w_router, const float* logit_bias,
                                const int8_t* wq_gate, const float* w_gate_scale, const int8_t* wq_up,
                                const float* w_up_scale, const int8_t* wq_down, const float* w_down_scale, float* logits,
                                int32_t* topk_idx, float* topk_w, int32_t* counts, int32_t* offsets,
                                int32_t* sorted_to_flat, int32_t* flat_to_sorted, int32_t* row_token, float* row_weight,
                                int8_t* xq, float* x_scale, int8_t* aq, float* a_scale, void* o_perm, void* y, void* ws,
                                size_t ws_bytes, hipStream_t stream);

/* moe_forward_few on 8-bit integer weights (moe_quantize_i8_rows): codes convert
 * to bf16 exactly, the activations stay in bf16 (not quantised, unlike
 * moe_forward_fused_i8, to which it is close within their rounding), and a
 * channel's scale multiplies its finished fp32 sum. a between gate/up and down is
 * rounded to bf16, as there: y is off by 0.0024 in the norm, where moe_experts_i8,
 * whose a is in 24 bits before its codes, is off by 0.0017 (bf16 y alone: 0.0016),
 * each against its own definition. Limits, outputs and
 * workspace (moe_few_workspace_bytes) as there; scales [E,I], [E,I] and [E,H], at
 * multiples of 16 bytes. */
moe_status moe_forward_few_i8(moe_shape s, const void* x, const void* w_router, const float* logit_bias,
                              const int8_t* wq_gate, const float* w_gate_scale, const int8_t* wq_up,
                              const float* w_up_scale, const int8_t* wq_down, const float* w_down_scale, float* logits,
                              int32_t* topk_idx, float* topk_w, void* y, void* ws, size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_I8_H_ */
