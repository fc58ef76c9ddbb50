/* moe_serve.h — serving operators of libmoe beside those of moe.h: matrix
 * products and the expert stage on 8-bit weights with one scale per block of
 * 128, and the whole MoE layer for a few tokens (decoding).
 *
 * The conventions of moe.h hold here too: device pointers to dense row-major
 * arrays, int32 indices, caller-owned buffers, nothing allocated, nothing
 * synchronised, every argument checked on the host before any HIP call,
 * results deterministic. Arrays of no rows (rows or M of 0) may be NULL; nothing
 * is done then. Every other array starts at a multiple of 16 bytes (as
 * allocations do; MOE_EINVAL otherwise where the kernels depend on it).
 *
 *   prefill: moe_forward_fused_fp8_block = moe_route -> moe_experts_fp8_block
 *            moe_experts_fp8_block = moe_permute_fused ->
 *              moe_quantize_fp8_block_rows (x) -> moe_gemm_gate_up_fp8_block ->
 *              the down product -> the per-token sum
 *   decode:  moe_forward_few (bf16 weights), moe_forward_few_fp8_block
 */
#ifndef MOE_SERVE_H_
#define MOE_SERVE_H_

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Block-scaled 8-bit operands. Elements are OCP E4M3 codes (bias 7,
 * largest finite 448, 0x7F/0xFF NaN); a block of 128 along the reduction axis
 * shares one float32 scale: activations 1 x 128, weights 128 x 128 (the
 * format in which 8-bit checkpoints of these models are published). With
 * amax the block's largest magnitude,
 *   scale = amax / 448,   code = E4M3(448 v / amax), nearest, ties to even
 * (0 and 0 for a block of zeros); 448 v / amax is rounded once, so for bf16 v
 * the codes are those of exact arithmetic. Blocks at the end of a row, or of
 * a weight, may be short. A NaN element gives a NaN code; an infinite one
 * makes its block's finite elements zeros, its own code NaN and the scale
 * infinite. */

/* Rows [rows, K] of bf16 -> codes q [rows, K], scale [rows, ceil(K/128)].
 * rows >= 0 and K > 0, K % 8 == 0 (MOE_EINVAL otherwise); rows * ceil(K/128)
 * at most 2^28 - 16 (MOE_EUNSUPPORTED otherwise). */
moe_status moe_quantize_fp8_block_rows(int32_t rows, int32_t K, const void* in, uint8_t* q, float* scale,
                                       hipStream_t stream);

/* A stacked weight w [E, N, K] of bf16 -> codes q [E, N, K] and
 * scale [E, ceil(N/128), ceil(K/128)]. K % 8 == 0 (MOE_EINVAL otherwise);
 * E * ceil(N/128) * ceil(K/128) below 2^24 (MOE_EUNSUPPORTED otherwise). */
moe_status moe_quantize_fp8_block_weights(int32_t E, int32_t N, int32_t K, const void* w, uint8_t* q, float* scale,
                                          hipStream_t stream);

/* Grouped product of block-scaled operands: for each expert e and row p in
 * [offsets[e], offsets[e+1]),
 *   out[p,n] = bf16(row_weight[p] * sum over blocks b of
 *                   a_scale[p,b] w_scale[e,n/128,b] sum_{k in b} aq[p,k] wq[e,n,k])
 * in fp32. aq [M,K], a_scale [M,ceil(K/128)], wq [E,N,K],
 * w_scale [E,ceil(N/128),ceil(K/128)], out [M,N] bf16. offsets [E+1] int32
 * with 0 <= offsets[0] <= ... <= offsets[E] <= M (not checked on the device);
 * rows outside [offsets[0], offsets[E]) are not written. offsets may be NULL
 * when E == 1 (every row: the dense product). row_weight [M] f32 or NULL (1).
 * 0 <= M < 2^30; N % 8 == 0, K % 16 == 0, E <= 1024, N K, 256 K and 512 N below 2^31
 * (MOE_EUNSUPPORTED otherwise). */
moe_status moe_gemm_fp8_block(int32_t M, int32_t E, int32_t N, int32_t K, const uint8_t* aq, const float* a_scale,
                              const int32_t* offsets, const uint8_t* wq, const float* w_scale, const float* row_weight,
                              void* out, hipStream_t stream);

/* Gathered gate/up GEMM with the SwiGLU epilogue, its result quantised:
 *   a = silu(g) * u,  g = deq(xq[row_token[p]]) deq(Wg[e])^T, u likewise (fp32),
 *   aq [T*k,I], a_scale [T*k,ceil(I/128)]: a in blocks of 1 x 128, from fp32.
 * xq [T,H], x_scale [T,ceil(H/128)]; wq_gate, wq_up [E,I,H] with scales
 * [E,ceil(I/128),ceil(H/128)]. A layer's shape, here and below: shape.dtype
 * MOE_BF16, H and I multiples of 64 below 2^22, I H and T H below 2^31, T k below
 * 2^30 (MOE_EUNSUPPORTED otherwise), k <= E <= 1024; no limit on E I H, unlike
 * the calls of moe.h. */
moe_status moe_gemm_gate_up_fp8_block(moe_shape s, const uint8_t* xq, const float* x_scale, const int32_t* row_token,
                                      const int32_t* offsets, const uint8_t* wq_gate, const float* w_gate_scale,
                                      const uint8_t* wq_up, const float* w_up_scale, uint8_t* aq, float* a_scale,
                                      hipStream_t stream);

/* The expert stage on block-scaled weights for routing that the caller
 * computed (topk_idx [T,k] in [0,E), topk_w [T,k] f32): moe_permute_fused,
 * the quantisation of x, the two GEMMs and the per-token sum (y [T,H] bf16).
 * o_perm [T*k,H], 2 bytes per element, is scratch: the rows of the down
 * product times row_weight, eight columns to 16 bytes with a common exponent,
 * so that only y is rounded to bf16. A number in it is off by at most 2^-8 of
 * itself, as in bf16 (from 2^-62 of the largest of the eight down it fades to
 * zero), and by at most 2^-13 of the largest where that is 2^-114 or more.
 * Every buffer is caller-owned and overwritten; wq_down [E,H,I] with scales
 * [E,ceil(H/128),ceil(I/128)]; ws of ws_bytes >=
 * MOE_FP8_BLOCK_WORKSPACE_BYTES(T, k, E), which moe_workspace_bytes(s) covers
 * where it is not 0. */
#define MOE_FP8_BLOCK_WORKSPACE_BYTES(T, k, E) \
  ((((size_t)(T) * (size_t)(k) + 1023) / 1024 * (size_t)(E) * 4 + 255) / 256 * 256)
moe_status moe_experts_fp8_block(moe_shape s, const void* x, const int32_t* topk_idx, const float* topk_w,
                                 const uint8_t* wq_gate, const float* w_gate_scale, const uint8_t* wq_up,
                                 const float* w_up_scale, const uint8_t* wq_down, const float* w_down_scale,
                                 int32_t* counts, int32_t* offsets, int32_t* sorted_to_flat, int32_t* flat_to_sorted,
                                 int32_t* row_token, float* row_weight, uint8_t* xq, float* x_scale, uint8_t* aq,
                                 float* a_scale, void* o_perm, void* y, void* ws, size_t ws_bytes, hipStream_t stream);

/* moe_route (logits, topk_idx, topk_w), then moe_experts_fp8_block. */
moe_status moe_forward_fused_fp8_block(moe_shape s, const void* x, const void* w_router, const float* logit_bias,
                                       const uint8_t* wq_gate, const float* w_gate_scale, const uint8_t* wq_up,
                                       const float* w_up_scale, const uint8_t* wq_down, const float* w_down_scale,
                                       float* logits, int32_t* topk_idx, float* topk_w, int32_t* counts,
                                       int32_t* offsets, int32_t* sorted_to_flat, int32_t* flat_to_sorted,
                                       int32_t* row_token, float* row_weight, uint8_t* xq, float* x_scale, uint8_t* aq,
                                       float* a_scale, void* o_perm, void* y, void* ws, size_t ws_bytes,
                                       hipStream_t stream);

/* ---- The whole layer for a few tokens (decoding), in two launches: the
 * router's logits, then one kernel that selects the experts, streams each
 * selected expert's weights once and sums the result per token.
 *   logits[t,e] = the sum over h of x[t,h] w_router[e,h], plus bias[e], in
 *     float64, rounded once to float32;
 *   topk_idx, topk_w from them as moe_route (largest first, ties to the lower
 *     index, NaN below every number);
 *   a[t,j] = bf16(topk_w[t,j] * silu(g) * u), g = x[t] W_gate[e]^T, u likewise;
 *   y[t] = bf16(sum over j of a[t,j] W_down[e]^T)     (fp32 accumulation).
 * It equals moe_forward_fused up to rounding (there the logits are an fp32
 * chain and the weight multiplies the down product). T <= 64, k <= 16,
 * T k I below 2^30 (MOE_EUNSUPPORTED otherwise: moe_forward_fused).
 * logits [T,E] f32, topk_idx [T,k], topk_w [T,k] f32 and y [T,H] bf16 are
 * outputs. Workspace: ws of ws_bytes >= moe_few_workspace_bytes(s), its
 * contents arbitrary; calls that share one must not overlap in time (their
 * results are then undefined; a wait inside the kernel that is never answered
 * ends after some seconds of running, and y is NaN there). */
size_t moe_few_workspace_bytes(moe_shape s);
moe_status moe_forward_few(moe_shape s, const void* x, const void* w_router, const float* logit_bias,
                           const void* w_gate, const void* w_up, const void* w_down, float* logits, int32_t* topk_idx,
                           float* topk_w, void* y, void* ws, size_t ws_bytes, hipStream_t stream);

/* The same on block-scaled 8-bit weights (moe_quantize_fp8_block_weights):
 * codes convert to bf16 exactly, and the activations stay in bf16 (not
 * quantised, unlike moe_forward_fused_fp8_block, to which it is close
 * within their rounding). */
moe_status moe_forward_few_fp8_block(moe_shape s, const void* x, const void* w_router, const float* logit_bias,
                                     const uint8_t* wq_gate, const float* w_gate_scale, const uint8_t* wq_up,
                                     const float* w_up_scale, const uint8_t* wq_down, const float* w_down_scale,
                                     float* logits, int32_t* topk_idx, float* topk_w, void* y, void* ws,
                                     size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_SERVE_H_ */
