/* moe_ckpt8.h — activations kept for the backward pass in 8 bits, beside the
 * training step of moe.h.
 *
 * A row of activations is held as whole numbers in [-127, 127] with one float32
 * scale per 64 columns: with amax a block's largest magnitude,
 *   scale = amax / 127,   code = the whole number nearest to 127 v / amax, halves to even
 * (0 and 0 for a block of zeros). A block with a NaN or an infinity has scale NaN:
 * what is computed from it is NaN. A value is off by at most half a step, 2^-7.99
 * of its block's largest.
 *
 * The step keeps, per layer, the gate and up projections G and U of every sorted
 * row (2 I (1 + 1/16) bytes a row) and, if wanted, x (1 1/16 bytes a value), in the
 * place of G, U, a_w and o_perm in bf16 (6 I + 2 H bytes a row; a is not kept by
 * either). Nothing of the forward's results changes: a = silu(g) u is formed from
 * the exact g and u.
 *   forward:  moe_route -> moe_permute_fused -> moe_gemm_gate_up_ckpt8 ->
 *             moe_gemm_down -> moe_combine   [moe_quantize_ckpt8 (x)]
 *   backward: moe_gemm_down_dgrad_ckpt8 -> moe_gemm_down_wgrad_dy ->
 *             [moe_dequantize_ckpt8 (x)] moe_gemm_gate_up_bwd ->
 *             moe_unpermute_sum -> moe_route_bwd
 * The routing weights' gradient comes from the data gradient, <dy, a W_down^T> =
 * <dy W_down, a>, so that neither o_perm nor moe_combine_bwd is needed.
 *
 * The conventions of moe.h hold here too: device pointers to dense row-major
 * arrays, caller-owned buffers, nothing allocated, nothing synchronised, every
 * argument checked on the host before any HIP call, results deterministic. Arrays
 * start at multiples of 16 bytes (MOE_EINVAL otherwise where the kernels depend on
 * it).
 */
#ifndef MOE_CKPT8_H_
#define MOE_CKPT8_H_

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows [rows, K] of bf16 -> codes q [rows, K], scale [rows, ceil(K/64)], and back
 * (out [rows, K] bf16: code * scale, rounded once). The codes are those of exact
 * arithmetic. The last block of a row may be short. rows >= 0 (of 0: NULL arrays,
 * nothing is done) and K > 0, K % 8 == 0 (MOE_EINVAL otherwise); rows *
 * ceil(K/64) below 2^29 - 32 (MOE_EUNSUPPORTED otherwise). */
moe_status moe_quantize_ckpt8(int32_t rows, int32_t K, const void* in, int8_t* q, float* scale, hipStream_t stream);
moe_status moe_dequantize_ckpt8(int32_t rows, int32_t K, const int8_t* q, const float* scale, void* out,
                                hipStream_t stream);

/* moe_gemm_gate_up (x_rows = x_perm, row_token NULL) or moe_gemm_gate_up_gathered
 * (x_rows = x [T,H], sorted row p read as row row_token[p]) that keeps g and u in 8
 * bits: gq, uq [T*k,I] and g_scale, u_scale [T*k,I/64], from the fp32 sums; a
 * [T*k,I] as there. bf16 only, I*H*2 < 2^31, H and I below 2^22
 * (MOE_EUNSUPPORTED otherwise); the limits of moe_gemm_gate_up_gathered with
 * row_token. Results of rows outside [offsets[0], offsets[E]) are not written, here
 * and below. */
moe_status moe_gemm_gate_up_ckpt8(moe_shape s, const void* x_rows, const int32_t* row_token, const int32_t* offsets,
                                  const void* w_gate, const void* w_up, int8_t* gq, float* g_scale, int8_t* uq,
                                  float* u_scale, void* a, hipStream_t stream);

/* The down projection's data gradient from the kept g and u (their values code *
 * scale, in fp32). For each expert e and sorted row p of it, t = row_token[p], w =
 * row_weight[p], s = sigmoid(g):
 *   dA = dy[t] W_down[e],  a = silu(g) u
 *   dgu[p] = [w dA u s (1 + g (1 - s)) | w dA silu(g)]   (bf16 [T*k,2I])
 *   a_w[p] = w a                                         (bf16 [T*k,I], for moe_gemm_down_wgrad_dy)
 *   d_topk_w[sorted_to_flat[p]] = <dA, a>                (f32 [T,k])
 * Workspace: ws of ws_bytes >= moe_ckpt8_workspace_bytes(s) (0 for a shape this
 * call rejects; moe_workspace_bytes(s) covers it). bf16 only, T*H*2 and I*H*2
 * below 2^31, H and I below 2^22 (MOE_EUNSUPPORTED otherwise). */
size_t moe_ckpt8_workspace_bytes(moe_shape s);
moe_status moe_gemm_down_dgrad_ckpt8(moe_shape s, const void* dy, const int32_t* row_token, const float* row_weight,
                                     const int32_t* sorted_to_flat, const int32_t* offsets, const void* w_down,
                                     const int8_t* gq, const float* g_scale, const int8_t* uq, const float* u_scale,
                                     void* dgu, void* a_w, float* d_topk_w, void* ws, size_t ws_bytes,
                                     hipStream_t stream);

/* The weight-gradient half of moe_gemm_down_bwd_dy on its own:
 *   dW_down[e] = sum over p of dy[row_token[p]]^T a_w[p]   (f32 [E,H,I]; += if accumulate_dw)
 * bf16 only, T*H*2 and 4*(T*k+256) below 2^31 (MOE_EUNSUPPORTED otherwise); ws of
 * ws_bytes >= moe_workspace_bytes(s). */
moe_status moe_gemm_down_wgrad_dy(moe_shape s, const void* dy, const int32_t* row_token, const void* a_w,
                                  const int32_t* offsets, float* dw_down, int accumulate_dw, void* ws, size_t ws_bytes,
                                  hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_CKPT8_H_ */
