// C ABI of the serving operators (moe_serve.h, moe_i8.h): argument checks on the host,
// then kernel launches. Every check runs before any HIP call, so a rejected
// call enqueues nothing.
#include "moe_internal.h"

namespace {

moe_status from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }

template <class... P>
bool any_null(P... p) {
  return ((p == nullptr) || ...);
}

// The kernels move 16 bytes at a time.
template <class... P>
bool misaligned(P... p) {
  return (((reinterpret_cast<uintptr_t>(p) & 15) != 0) || ...);
}

constexpr int64_t k2G = static_cast<int64_t>(1) << 31;
constexpr int64_t kMaxThreads = static_cast<int64_t>(1) << 32;  // of one launch
constexpr int64_t kMaxRows = static_cast<int64_t>(1) << 30;     // rows are counted in int32, rounded up to tiles

// What the serving kernels need: 16-byte rows in whole half steps, offsets
// within one expert's weights, x, and a tile's rows in 32 bits (an expert's
// base is formed in 64). Sums over the experts have no limit here.
moe_status check_serve_shape(const moe_shape& s) {
  if (s.T <= 0 || s.H <= 0 || s.E <= 0 || s.k <= 0 || s.I <= 0) return MOE_EINVAL;
  if (s.k > s.E || s.E > 1024 || static_cast<int64_t>(s.T) * s.k >= k2G) return MOE_EINVAL;
  if (s.dtype != MOE_BF16 || s.H % 64 != 0 || s.I % 64 != 0) return MOE_EUNSUPPORTED;
  if (static_cast<int64_t>(s.T) * s.k >= kMaxRows || static_cast<int64_t>(s.I) * s.H >= k2G) return MOE_EUNSUPPORTED;
  if (static_cast<int64_t>(s.T) * s.H >= k2G || 512 * static_cast<int64_t>(s.H) >= k2G ||
      512 * static_cast<int64_t>(s.I) >= k2G)
    return MOE_EUNSUPPORTED;
  return MOE_OK;
}

// The sort's counts: E per block of 1024 (token, slot) pairs.
size_t fp8_block_workspace_bytes(const moe_shape& s) {
  static_assert(moe::kPermBlock == 1024, "the header's formula");
  return MOE_FP8_BLOCK_WORKSPACE_BYTES(s.T, s.k, s.E);
}

// The integer stage's workspace: the sort's counts, then silu(g) u in 16 and 8
// bits and its maxima per 128 columns.
struct I8Layout {
  size_t v16, v8, amax, total;
};
I8Layout i8_layout(const moe_shape& s) {
  auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
  const size_t M = static_cast<size_t>(s.T) * s.k;
  I8Layout l;
  l.v16 = fp8_block_workspace_bytes(s);
  l.v8 = up(l.v16 + M * s.I * 2);
  l.amax = up(l.v8 + M * s.I);
  l.total = up(l.amax + M * moe::ceil_div(s.I, 128) * 4);
  return l;
}

// K products of at most 2^14 each, summed in int32.
constexpr int64_t kMaxI8K = static_cast<int64_t>(1) << 17;
moe_status check_i8_shape(const moe_shape& s) {
  const moe_status st = check_serve_shape(s);
  if (st != MOE_OK) return st;
  if (s.H >= kMaxI8K || s.I >= kMaxI8K) return MOE_EUNSUPPORTED;
  return static_cast<int64_t>(s.T) * s.k * (s.I / 8) + 256 >= kMaxThreads ? MOE_EUNSUPPORTED : MOE_OK;
}

moe_status check_few(const moe_shape& s) {
  const moe_status st = check_serve_shape(s);
  if (st != MOE_OK) return st;
  if (s.T > moe::kFewMaxT || s.k > moe::kFewMaxK) return MOE_EUNSUPPORTED;
  return static_cast<int64_t>(s.T) * s.k * s.I * 2 >= k2G ? MOE_EUNSUPPORTED : MOE_OK;  // 32-bit offsets into a
}

}  // namespace

extern "C" {

moe_status moe_quantize_fp8_block_rows(int32_t rows, int32_t K, const void* in, uint8_t* q, float* scale,
                                       hipStream_t stream) {
  if (rows < 0 || K <= 0 || K % 8 != 0) return MOE_EINVAL;
  if (rows == 0) return MOE_OK;
  if (any_null(in, q, scale) || misaligned(in, q)) return MOE_EINVAL;
  // 16 threads per block of 128, in workgroups of 256
  if (moe::ceil_div64(static_cast<int64_t>(rows) * moe::ceil_div64(K, 128), 16) * 256 >= kMaxThreads) return MOE_EUNSUPPORTED;
  return from_hip(moe::launch_quantize_fp8_block_rows(rows, K, in, q, scale, stream));
}

moe_status moe_quantize_fp8_block_weights(int32_t E, int32_t N, int32_t K, const void* w, uint8_t* q, float* scale,
                                          hipStream_t stream) {
  if (E <= 0 || N <= 0 || K <= 0 || K % 8 != 0) return MOE_EINVAL;
  if (any_null(w, q, scale) || misaligned(w, q)) return MOE_EINVAL;
  const int64_t most = kMaxThreads / 256, bands = E * moe::ceil_div64(N, 128);  // a workgroup per block
  if (bands >= most || bands * moe::ceil_div64(K, 128) >= most) return MOE_EUNSUPPORTED;
  return from_hip(moe::launch_quantize_fp8_block_weights(E, N, K, w, q, scale, stream));
}

moe_status moe_gemm_fp8_block(int32_t M, int32_t E, int32_t N, int32_t K, const uint8_t* aq, const float* a_scale,
                              const int32_t* offsets, const uint8_t* wq, const float* w_scale, const float* row_weight,
                              void* out, hipStream_t stream) {
  if (M < 0 || E <= 0 || N <= 0 || K <= 0) return MOE_EINVAL;
  if (any_null(wq, w_scale) || (offsets == nullptr && E != 1)) return MOE_EINVAL;
  if (M > 0 && any_null(aq, a_scale, out)) return MOE_EINVAL;
  if (misaligned(aq, wq, out)) return MOE_EINVAL;
  if (N % 8 != 0 || K % 16 != 0 || E > 1024 || M >= kMaxRows) return MOE_EUNSUPPORTED;
  if (static_cast<int64_t>(N) * K >= k2G || 256 * static_cast<int64_t>(K) >= k2G || 512 * static_cast<int64_t>(N) >= k2G)
    return MOE_EUNSUPPORTED;
  moe::BlockGemmArgs g{};
  g.M = g.arows = M;
  g.E = E;
  g.N = N;
  g.K = K;
  g.a = aq;
  g.a_scale = a_scale;
  g.offsets = offsets;
  g.w0 = wq;
  g.w0_scale = w_scale;
  g.row_weight = row_weight;
  g.out = out;
  return from_hip(moe::launch_gemm_fp8_block(g, stream));
}

moe_status moe_gemm_gate_up_fp8_block(moe_shape s, const uint8_t* xq, const float* x_scale, const int32_t* row_token,
                                      const int32_t* offsets, const uint8_t* wq_gate, const float* w_gate_scale,
                                      const uint8_t* wq_up, const float* w_up_scale, uint8_t* aq, float* a_scale,
                                      hipStream_t stream) {
  const moe_status st = check_serve_shape(s);
  if (st != MOE_OK) return st;
  if (any_null(xq, x_scale, row_token, offsets, wq_gate, w_gate_scale, wq_up, w_up_scale, aq, a_scale))
    return MOE_EINVAL;
  if (misaligned(xq, wq_gate, wq_up, aq)) return MOE_EINVAL;
  moe::BlockGemmArgs g{};
  g.M = s.T * s.k;
  g.arows = s.T;
  g.E = s.E;
  g.N = s.I;
  g.K = s.H;
  g.a = xq;
  g.a_scale = x_scale;
  g.row_token = row_token;
  g.offsets = offsets;
  g.w0 = wq_gate;
  g.w0_scale = w_gate_scale;
  g.w1 = wq_up;
  g.w1_scale = w_up_scale;
  g.aq = aq;
  g.a_out_scale = a_scale;
  return from_hip(moe::launch_gemm_fp8_block(g, stream));
}

moe_status moe_experts_fp8_block(moe_shape s, const void* x, const int32_t* topk_idx, const float* topk_w,
                                 const uint8_t* wq_gate, const float* w_gate_scale, const uint8_t* wq_up,
                                 const float* w_up_scale, const uint8_t* wq_down, const float* w_down_scale,
                                 int32_t* counts, int32_t* offsets, int32_t* sorted_to_flat, int32_t* flat_to_sorted,
                                 int32_t* row_token, float* row_weight, uint8_t* xq, float* x_scale, uint8_t* aq,
                                 float* a_scale, void* o_perm, void* y, void* ws, size_t ws_bytes,
                                 hipStream_t stream) {
  moe_status st = check_serve_shape(s);
  if (st != MOE_OK) return st;
  if (any_null(x, topk_idx, topk_w, wq_gate, w_gate_scale, wq_up, w_up_scale, wq_down, w_down_scale, counts, offsets,
               sorted_to_flat, flat_to_sorted, row_token, row_weight, xq, x_scale, aq, a_scale, o_perm, y, ws))
    return MOE_EINVAL;
  if (misaligned(x, wq_gate, wq_up, wq_down, xq, aq, o_perm, y)) return MOE_EINVAL;
  if (ws_bytes < fp8_block_workspace_bytes(s)) return MOE_EWORKSPACE;
  if ((st = from_hip(moe::launch_permute_fused(s, topk_idx, topk_w, counts, offsets, sorted_to_flat, flat_to_sorted,
                                               row_token, row_weight, ws, stream))) != MOE_OK)
    return st;
  if ((st = moe_quantize_fp8_block_rows(s.T, s.H, x, xq, x_scale, stream)) != MOE_OK) return st;
  if ((st = moe_gemm_gate_up_fp8_block(s, xq, x_scale, row_token, offsets, wq_gate, w_gate_scale, wq_up, w_up_scale, aq,
                                       a_scale, stream)) != MOE_OK)
    return st;
  moe::BlockGemmArgs g{};
  g.M = g.arows = s.T * s.k;
  g.E = s.E;
  g.N = s.H;
  g.K = s.I;
  g.a = aq;
  g.a_scale = a_scale;
  g.offsets = offsets;
  g.w0 = wq_down;
  g.w0_scale = w_down_scale;
  g.row_weight = row_weight;
  g.out = o_perm;
  g.shared8 = true;
  if ((st = from_hip(moe::launch_gemm_fp8_block(g, stream))) != MOE_OK) return st;
  return from_hip(moe::launch_sum_shared8(s, o_perm, flat_to_sorted, y, stream));
}

moe_status moe_forward_fused_fp8_block(moe_shape s, const void* x, const void* w_router, const float* logit_bias,
                                       const uint8_t* wq_gate, const float* w_gate_scale, const uint8_t* wq_up,
                                       const float* w_up_scale, const uint8_t* wq_down, const float* w_down_scale,
                                       float* logits, int32_t* topk_idx, float* topk_w, int32_t* counts,
                                       int32_t* offsets, int32_t* sorted_to_flat, int32_t* flat_to_sorted,
                                       int32_t* row_token, float* row_weight, uint8_t* xq, float* x_scale, uint8_t* aq,
                                       float* a_scale, void* o_perm, void* y, void* ws, size_t ws_bytes,
                                       hipStream_t stream) {
  moe_status st = check_serve_shape(s);
  if (st != MOE_OK) return st;
  if (any_null(x, w_router, wq_gate, w_gate_scale, wq_up, w_up_scale, wq_down, w_down_scale, logits, topk_idx, topk_w,
               counts, offsets, sorted_to_flat, flat_to_sorted, row_token, row_weight, xq, x_scale, aq, a_scale, o_perm,
               y, ws))
    return MOE_EINVAL;
  if (misaligned(x, w_router, wq_gate, wq_up, wq_down, xq, aq, o_perm, y)) return MOE_EINVAL;
  if (ws_bytes < fp8_block_workspace_bytes(s)) return MOE_EWORKSPACE;
  if ((st = from_hip(moe::launch_route(s, x, w_router, logit_bias, logits, topk_idx, topk_w, stream))) != MOE_OK) return st;
  return moe_experts_fp8_block(s, x, topk_idx, topk_w, wq_gate, w_gate_scale, wq_up, w_up_scale, wq_down, w_down_scale,
                               counts, offsets, sorted_to_flat, flat_to_sorted, row_token, row_weight, xq, x_scale, aq,
                               a_scale, o_perm, y, ws, ws_bytes, stream);
}

moe_status moe_quantize_i8_rows(int32_t rows, int32_t K, const void* in, int8_t* q, float* scale, hipStream_t stream) {
  if (rows < 0 || K <= 0 || K % 8 != 0) return MOE_EINVAL;
  if (rows == 0) return MOE_OK;
  if (any_null(in, q, scale) || misaligned(in, q)) return MOE_EINVAL;
  // 16, 64 or 256 threads per row, in workgroups of 256
  const int64_t per_row = K <= 512 ? 16 : K <= 2048 ? 64 : 256;
  if (rows * per_row + 256 >= kMaxThreads) return MOE_EUNSUPPORTED;
  return from_hip(moe::launch_quantize_i8_rows(rows, K, in, q, scale, stream));
}

moe_status moe_gemm_i8(int32_t M, int32_t E, int32_t N, int32_t K, const int8_t* aq, const float* a_scale,
                       const int32_t* offsets, const int8_t* wq, const float* w_scale, const float* row_weight, void* out,
                       hipStream_t stream) {
  if (M < 0 || E <= 0 || N <= 0 || K <= 0) return MOE_EINVAL;
  if (any_null(wq, w_scale) || (offsets == nullptr && E != 1)) return MOE_EINVAL;
  if (M > 0 && any_null(aq, a_scale, out)) return MOE_EINVAL;
  if (misaligned(aq, wq, out)) return MOE_EINVAL;
  if (N % 8 != 0 || K % 16 != 0 || K >= kMaxI8K || E > 1024 || M >= kMaxRows) return MOE_EUNSUPPORTED;
  if (static_cast<int64_t>(N) * K >= k2G || 512 * static_cast<int64_t>(N) >= k2G) return MOE_EUNSUPPORTED;
  moe::I8GemmArgs g{};
  g.M = g.arows = M;
  g.E = E;
  g.N = N;
  g.K = K;
  g.a = aq;
  g.a_scale = a_scale;
  g.offsets = offsets;
  g.w0 = wq;
  g.w0_scale = w_scale;
  g.row_weight = row_weight;
  g.out = out;
  return from_hip(moe::launch_gemm_i8(g, stream));
}

size_t moe_i8_workspace_bytes(moe_shape s) { return check_i8_shape(s) != MOE_OK ? 0 : i8_layout(s).total; }

moe_status moe_gemm_gate_up_i8(moe_shape s, const int8_t* xq, const float* x_scale, const int32_t* row_token,
                               const int32_t* offsets, const int8_t* wq_gate, const float* w_gate_scale,
                               const int8_t* wq_up, const float* w_up_scale, int8_t* aq, float* a_scale, void* ws,
                               size_t ws_bytes, hipStream_t stream) {
  const moe_status st = check_i8_shape(s);
  if (st != MOE_OK) return st;
  if (any_null(xq, x_scale, row_token, offsets, wq_gate, w_gate_scale, wq_up, w_up_scale, aq, a_scale, ws))
    return MOE_EINVAL;
  if (misaligned(xq, wq_gate, wq_up, aq, ws)) return MOE_EINVAL;
  const I8Layout l = i8_layout(s);
  if (ws_bytes < l.total) return MOE_EWORKSPACE;
  moe::I8GemmArgs g{};
  g.M = s.T * s.k;
  g.arows = s.T;
  g.E = s.E;
  g.N = s.I;
  g.K = s.H;
  g.a = xq;
  g.a_scale = x_scale;
  g.row_token = row_token;
  g.offsets = offsets;
  g.w0 = wq_gate;
  g.w0_scale = w_gate_scale;
  g.w1 = wq_up;
  g.w1_scale = w_up_scale;
  g.v16 = reinterpret_cast<int16_t*>(static_cast<char*>(ws) + l.v16);
  g.v8 = static_cast<uint8_t*>(ws) + l.v8;
  g.amax = reinterpret_cast<float*>(static_cast<char*>(ws) + l.amax);
  const moe_status done = from_hip(moe::launch_gemm_i8(g, stream));
  if (done != MOE_OK) return done;
  return from_hip(moe::launch_requantize_i8_rows(g.M, s.I, s.E, offsets, g.v16, g.v8, g.amax, aq, a_scale, stream));
}

moe_status moe_experts_i8(moe_shape s, const void* x, const int32_t* topk_idx, const float* topk_w,
                          const int8_t* wq_gate, const float* w_gate_scale, const int8_t* wq_up, const float* w_up_scale,
                          const int8_t* wq_down, const float* w_down_scale, int32_t* counts, int32_t* offsets,
                          int32_t* sorted_to_flat, int32_t* flat_to_sorted, int32_t* row_token, float* row_weight,
                          int8_t* xq, float* x_scale, int8_t* aq, float* a_scale, void* o_perm, void* y, void* ws,
                          size_t ws_bytes, hipStream_t stream) {
  moe_status st = check_i8_shape(s);
  if (st != MOE_OK) return st;
  if (any_null(x, topk_idx, topk_w, wq_gate, w_gate_scale, wq_up, w_up_scale, wq_down, w_down_scale, counts, offsets,
               sorted_to_flat, flat_to_sorted, row_token, row_weight, xq, x_scale, aq, a_scale, o_perm, y, ws))
    return MOE_EINVAL;
  if (misaligned(x, wq_gate, wq_up, wq_down, xq, aq, o_perm, y, ws)) return MOE_EINVAL;
  if (ws_bytes < i8_layout(s).total) return MOE_EWORKSPACE;
  if ((st = from_hip(moe::launch_permute_quantize_i8(s, topk_idx, topk_w, x, counts, offsets, sorted_to_flat,
                                                     flat_to_sorted, row_token, row_weight, xq, x_scale, ws,
                                                     stream))) != MOE_OK)
    return st;
  if ((st = moe_gemm_gate_up_i8(s, xq, x_scale, row_token, offsets, wq_gate, w_gate_scale, wq_up, w_up_scale, aq, a_scale,
                                ws, ws_bytes, stream)) != MOE_OK)
    return st;
  moe::I8GemmArgs g{};
  g.M = g.arows = s.T * s.k;
  g.E = s.E;
  g.N = s.H;
  g.K = s.I;
  g.a = aq;
  g.a_scale = a_scale;
  g.offsets = offsets;
  g.w0 = wq_down;
  g.w0_scale = w_down_scale;
  g.row_weight = row_weight;
  g.out = o_perm;
  g.shared8 = true;
  if ((st = from_hip(moe::launch_gemm_i8(g, stream))) != MOE_OK) return st;
  return from_hip(moe::launch_sum_shared8(s, o_perm, flat_to_sorted, y, stream));
}

moe_status moe_forward_fused_i8(moe_shape s, const void* x, const void* w_router, const float* logit_bias,
                                const int8_t* wq_gate, const float* w_gate_scale, const int8_t* wq_up,
                                const float* w_up_scale, const int8_t* wq_down, const float* w_down_scale, float* logits,
                                int32_t* topk_idx, float* topk_w, int32_t* counts, int32_t* offsets,
                                int32_t* sorted_to_flat, int32_t* flat_to_sorted, int32_t* row_token, float* row_weight,
                                int8_t* xq, float* x_scale, int8_t* aq, float* a_scale, void* o_perm, void* y, void* ws,
                                size_t ws_bytes, hipStream_t stream) {
  moe_status st = check_i8_shape(s);
  if (st != MOE_OK) return st;
  if (any_null(x, w_router, wq_gate, w_gate_scale, wq_up, w_up_scale, wq_down, w_down_scale, logits, topk_idx, topk_w,
               counts, offsets, sorted_to_flat, flat_to_sorted, row_token, row_weight, xq, x_scale, aq, a_scale, o_perm,
               y, ws))
    return MOE_EINVAL;
  if (misaligned(x, w_router, wq_gate, wq_up, wq_down, xq, aq, o_perm, y, ws)) return MOE_EINVAL;
  if (ws_bytes < i8_layout(s).total) return MOE_EWORKSPACE;
  if ((st = from_hip(moe::launch_route(s, x, w_router, logit_bias, logits, topk_idx, topk_w, stream))) != MOE_OK) return st;
  return moe_experts_i8(s, x, topk_idx, topk_w, wq_gate, w_gate_scale, wq_up, w_up_scale, wq_down, w_down_scale, counts,
                        offsets, sorted_to_flat, flat_to_sorted, row_token, row_weight, xq, x_scale, aq, a_scale, o_perm,
                        y, ws, ws_bytes, stream);
}

size_t moe_few_workspace_bytes(moe_shape s) {
  if (check_few(s) != MOE_OK) return 0;
  return moe::few_layout(s).total;
}

moe_status moe_forward_few(moe_shape s, const void* x, const void* w_router, const float* logit_bias,
                           const void* w_gate, const void* w_up, const void* w_down, float* logits, int32_t* topk_idx,
                           float* topk_w, void* y, void* ws, size_t ws_bytes, hipStream_t stream) {
  const moe_status st = check_few(s);
  if (st != MOE_OK) return st;
  if (any_null(x, w_router, w_gate, w_up, w_down, logits, topk_idx, topk_w, y, ws)) return MOE_EINVAL;
  if (misaligned(x, w_router, w_gate, w_up, w_down, y, ws)) return MOE_EINVAL;
  if (ws_bytes < moe::few_layout(s).total) return MOE_EWORKSPACE;
  moe::FewArgs a{};
  a.x = x;
  a.w_router = w_router;
  a.bias = logit_bias;
  a.w_gate = w_gate;
  a.w_up = w_up;
  a.w_down = w_down;
  a.logits = logits;
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.y = y;
  return from_hip(moe::launch_few(s, a, ws, stream));
}

moe_status moe_forward_few_fp8_block(moe_shape s, const void* x, const void* w_router, const float* logit_bias,
                                     const uint8_t* wq_gate, const float* w_gate_scale, const uint8_t* wq_up,
                                     const float* w_up_scale, const uint8_t* wq_down, const float* w_down_scale,
                                     float* logits, int32_t* topk_idx, float* topk_w, void* y, void* ws,
                                     size_t ws_bytes, hipStream_t stream) {
  const moe_status st = check_few(s);
  if (st != MOE_OK) return st;
  if (any_null(x, w_router, wq_gate, w_gate_scale, wq_up, w_up_scale, wq_down, w_down_scale, logits, topk_idx, topk_w, y,
               ws))
    return MOE_EINVAL;
  if (misaligned(x, w_router, wq_gate, wq_up, wq_down, y, ws)) return MOE_EINVAL;
  if (ws_bytes < moe::few_layout(s).total) return MOE_EWORKSPACE;
  moe::FewArgs a{};
  a.x = x;
  a.w_router = w_router;
  a.bias = logit_bias;
  a.w_gate = wq_gate;
  a.w_up = wq_up;
  a.w_down = wq_down;
  a.gate_scale = w_gate_scale;
  a.up_scale = w_up_scale;
  a.down_scale = w_down_scale;
  a.logits = logits;
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.y = y;
  return from_hip(moe::launch_few(s, a, ws, stream));
}

moe_status moe_forward_few_i8(moe_shape s, const void* x, const void* w_router, const float* logit_bias,
                              const int8_t* wq_gate, const float* w_gate_scale, const int8_t* wq_up,
                              const float* w_up_scale, const int8_t* wq_down, const float* w_down_scale, float* logits,
                              int32_t* topk_idx, float* topk_w, void* y, void* ws, size_t ws_bytes, hipStream_t stream) {
  const moe_status st = check_few(s);
  if (st != MOE_OK) return st;
  if (any_null(x, w_router, wq_gate, w_gate_scale, wq_up, w_up_scale, wq_down, w_down_scale, logits, topk_idx, topk_w, y,
               ws))
    return MOE_EINVAL;
  if (misaligned(x, w_router, wq_gate, w_gate_scale, wq_up, w_up_scale, wq_down, w_down_scale, y, ws)) return MOE_EINVAL;
  if (ws_bytes < moe::few_layout(s).total) return MOE_EWORKSPACE;
  moe::FewArgs a{};
  a.x = x;
  a.w_router = w_router;
  a.bias = logit_bias;
  a.w_gate = wq_gate;
  a.w_up = wq_up;
  a.w_down = wq_down;
  a.gate_scale = w_gate_scale;
  a.up_scale = w_up_scale;
  a.down_scale = w_down_scale;
  a.logits = logits;
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.y = y;
  return from_hip(moe::launch_few_i8(s, a, ws, stream));
}

}  // extern "C"
