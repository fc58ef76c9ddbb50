// 8-bit integer codes of bf16 rows: one fp32 scale per row (tokens, output
// channels of a weight), or one per 64 columns (activations kept for the
// backward pass) and back; and the second half of the gate/up product's
// quantisation. See i8.h for the codes.
//
// All are bound by memory (3 bytes per element, 4 in the last): every value
// is read once and stays in registers between its row's maximum and its code.
#include "i8.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// LPR lanes per row, CPL chunks of 8 columns in each one's registers: rows of up
// to 8 LPR CPL columns. Longer ones (LPR = 256 only) are read twice, the second
// time from cache.
template <int LPR, int CPL>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(int rows, int K, const uint4* __restrict__ in,
                                                                 uint2* __restrict__ q, float* __restrict__ scale) {
  __shared__ uint32_t part[kThreads / kWave];
  constexpr int RPB = kThreads / LPR;
  const int n = threadIdx.x % LPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + threadIdx.x / LPR;
  const bool active = row < rows;
  const int chunks = K / 8;
  const uint4* from = in + (active ? row : 0) * chunks;
  uint4 v[CPL];
  u16x2 m{0, 0};
#pragma unroll
  for (int i = 0; i < CPL; ++i) {
    const int c = n + i * LPR;
    v[i] = active && c < chunks ? from[c] : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < CPL; ++i) m = amax_bits(m, v[i]);
  if constexpr (LPR == kThreads)
    for (int c = n + CPL * LPR; c < chunks; c += LPR) m = amax_bits(m, from[c]);
  uint32_t bits = group_max<16>(amax_bits(m));
  if constexpr (LPR >= kWave) {
    bits = max(max(__builtin_amdgcn_readlane(bits, 0), __builtin_amdgcn_readlane(bits, 16)),
               max(__builtin_amdgcn_readlane(bits, 32), __builtin_amdgcn_readlane(bits, 48)));
  }
  if constexpr (LPR == kThreads) {
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = bits;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / kWave; ++w) bits = max(bits, part[w]);
  }
  const CodeFactor f(bits);
  if (!active) return;
  uint2* to = q + row * chunks;
#pragma unroll
  for (int i = 0; i < CPL; ++i) {
    const int c = n + i * LPR;
    if (c < chunks) to[c] = codes8(v[i], f);
  }
  if constexpr (LPR == kThreads)
    for (int c = n + CPL * LPR; c < chunks; c += LPR) to[c] = codes8(from[c], f);
  if (n == 0) scale[row] = f.scale;
}

// One 1 x 64 block per 8 lanes.
__global__ __launch_bounds__(kThreads) void quantize_ckpt8_kernel(uint32_t blocks, int K, uint32_t KB,
                                                                  const uint4* __restrict__ in, uint2* __restrict__ q,
                                                                  float* __restrict__ scale) {
  const uint32_t j = blockIdx.x * (kThreads / 8) + threadIdx.x / 8;
  const int n = threadIdx.x % 8, chunks = K / 8;
  const bool active = j < blocks;
  const uint32_t row = active ? j / KB : 0;
  const int c = static_cast<int>(active ? j - row * KB : 0) * 8 + n;
  const bool in_row = active && c < chunks;
  const int64_t at = static_cast<int64_t>(row) * chunks + c;
  const uint4 v = in_row ? in[at] : make_uint4(0u, 0u, 0u, 0u);
  const CodeFactor f(group_max<8>(amax_bits(amax_bits(u16x2{0, 0}, v))));
  if (in_row) q[at] = codes8(v, f);
  if (active && n == 0) scale[j] = f.scale;
}

__global__ __launch_bounds__(kThreads) void dequantize_ckpt8_kernel(uint32_t blocks, int K, uint32_t KB,
                                                                    const uint2* __restrict__ q,
                                                                    const float* __restrict__ scale,
                                                                    uint4* __restrict__ out) {
  const uint32_t j = blockIdx.x * (kThreads / 8) + threadIdx.x / 8;
  const int n = threadIdx.x % 8, chunks = K / 8;
  if (j >= blocks) return;
  const uint32_t row = j / KB;
  const int c = static_cast<int>(j - row * KB) * 8 + n;
  if (c >= chunks) return;
  const int64_t at = static_cast<int64_t>(row) * chunks + c;
  const uint2 w = q[at];
  const float s = scale[j];
  uint4 o;
  o.x = pack_bf16x2(code_value(w.x, 0) * s, code_value(w.x, 1) * s);
  o.y = pack_bf16x2(code_value(w.x, 2) * s, code_value(w.x, 3) * s);
  o.z = pack_bf16x2(code_value(w.y, 0) * s, code_value(w.y, 1) * s);
  o.w = pack_bf16x2(code_value(w.y, 2) * s, code_value(w.y, 3) * s);
  out[at] = o;
}

// Rows of 24-bit codes with a maximum per 128 columns (amax, NT per row) -> 8-bit
// codes with a scale per row, for the rows that some expert has.
__global__ __launch_bounds__(kThreads) void requantize_rows_kernel(uint32_t total, uint32_t chunks, int NT, int E,
                                                                   const int32_t* __restrict__ offsets,
                                                                   const uint4* __restrict__ v16,
                                                                   const uint2* __restrict__ v8,
                                                                   const float* __restrict__ amax,
                                                                   uint2* __restrict__ q, float* __restrict__ scale) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= total) return;
  const uint32_t first = static_cast<uint32_t>(offsets[0]), rows = static_cast<uint32_t>(offsets[E]) - first;
  const uint32_t row = i / chunks, c = i - row * chunks;
  const float* a = amax + static_cast<int64_t>(row) * NT;
  const uint4 v = v16[i];
  const uint2 lo = v8[i];
  float m = 0.0f;
  for (int t = 0; t < NT; ++t) m = __builtin_elementwise_maximum(m, a[t]);  // NaN if one is
  const bool finite = m < __builtin_inff();
  const float f = finite && m > 0.0f ? a[c / 16] / m * (127.0f / kFull24) : 0.0f;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t k[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t l = (j < 2 ? lo.x : lo.y) >> 16 * (j & 1);
    const int even = static_cast<int>(static_cast<int16_t>(w[j])) * 256 + static_cast<int>(l & 0xff);
    const int odd = (static_cast<int>(w[j]) >> 16) * 256 + static_cast<int>(l >> 8 & 0xff);
    k[2 * j] = code_bits(static_cast<float>(even) * f);
    k[2 * j + 1] = code_bits(static_cast<float>(odd) * f);
  }
  if (row - first >= rows) return;  // asked last: the loads do not wait for it
  q[i] = make_uint2(bytes4(k[0], k[1], k[2], k[3]), bytes4(k[4], k[5], k[6], k[7]));
  if (c == 0) scale[row] = finite ? m / 127.0f : __builtin_nanf("");
}

template <int LPR, int CPL>
hipError_t rows_launch(int rows, int K, const void* in, int8_t* q, float* scale, hipStream_t st) {
  const unsigned grid = static_cast<unsigned>(ceil_div64(rows, kThreads / LPR));
  quantize_rows_kernel<LPR, CPL><<<grid, kThreads, 0, st>>>(rows, K, static_cast<const uint4*>(in),
                                                            reinterpret_cast<uint2*>(q), scale);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_i8_rows(int rows, int K, const void* in, int8_t* q, float* scale, hipStream_t st) {
  // Lanes per row: as few as hold it in 64 bytes each, so that short rows leave
  // no lane idle and a long one's loads are all in flight at once.
  if (K <= 16 * 4 * 8) return rows_launch<16, 4>(rows, K, in, q, scale, st);
  if (K <= 64 * 4 * 8) return rows_launch<64, 4>(rows, K, in, q, scale, st);
  return rows_launch<256, 4>(rows, K, in, q, scale, st);
}

hipError_t launch_quantize_ckpt8(int rows, int K, const void* in, int8_t* q, float* scale, hipStream_t st) {
  const uint32_t KB = static_cast<uint32_t>(ceil_div(K, kCkptBlock)), blocks = static_cast<uint32_t>(rows) * KB;
  quantize_ckpt8_kernel<<<(blocks + kThreads / 8 - 1) / (kThreads / 8), kThreads, 0, st>>>(
      blocks, K, KB, static_cast<const uint4*>(in), reinterpret_cast<uint2*>(q), scale);
  return hipGetLastError();
}

hipError_t launch_dequantize_ckpt8(int rows, int K, const int8_t* q, const float* scale, void* out, hipStream_t st) {
  const uint32_t KB = static_cast<uint32_t>(ceil_div(K, kCkptBlock)), blocks = static_cast<uint32_t>(rows) * KB;
  dequantize_ckpt8_kernel<<<(blocks + kThreads / 8 - 1) / (kThreads / 8), kThreads, 0, st>>>(
      blocks, K, KB, reinterpret_cast<const uint2*>(q), scale, static_cast<uint4*>(out));
  return hipGetLastError();
}

hipError_t launch_requantize_i8_rows(int rows, int K, int E, const int32_t* offsets, const void* v16, const void* v8,
                                     const float* amax, int8_t* q, float* scale, hipStream_t st) {
  const uint32_t chunks = static_cast<uint32_t>(K / 8), total = static_cast<uint32_t>(rows) * chunks;
  requantize_rows_kernel<<<(total + kThreads - 1) / kThreads, kThreads, 0, st>>>(
      total, chunks, ceil_div(K, 128), E, offsets, static_cast<const uint4*>(v16), static_cast<const uint2*>(v8), amax,
      reinterpret_cast<uint2*>(q), scale);
  return hipGetLastError();
}

}  // namespace moe
