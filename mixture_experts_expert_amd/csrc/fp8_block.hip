// bf16 -> OCP E4M3 with one fp32 scale per block of 128: rows (activations)
// in 1 x 128 blocks, stacked weights in 128 x 128 blocks.
//
//   scale = amax / 448,  code = E4M3(448 v / amax)     (zeros for amax = 0)
//
// For bf16 v and amax the codes are those of exact arithmetic, ties to even
// included, without a division per element. The quotient q = 448 v / amax is
// taken as v * (448 / amax) in fp32, off by at most 2^-22 of q. A rounding
// boundary m of E4M3 has at most 5 significant bits M, and v and amax have 8 (V,
// A), so q - m is a multiple of 1 / (M A) of m: either zero or more than
// 2^-13 of it (31 * 255 < 2^13). Rounding the product to 13 fraction bits
// moves it by at most 2^-14 and leaves m itself in place, so a tie lands on
// the boundary exactly and everything else stays on its side of it.
//
// Both kernels are bound by memory (3 bytes per element): a lane takes 16
// bytes, the 16 lanes of a DPP row one 1 x 128 block; a workgroup holds a
// 128 x 128 weight block in registers between its maximum and its codes, so
// everything is read once.
#include "moe_internal.h"
#include "select.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void unpack8(const uint4& v, float* o) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = __uint_as_float(w[i] << 16);
    o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ float amax8(const uint4& v) {
  float f[8];
  unpack8(v, f);
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(f[i]));
  return a;
}

// Eight codes. `up` lifts blocks below 2^-64 by 2^64 (exact), so that
// 448 / amax stays finite.
__device__ __forceinline__ uint2 codes8(const uint4& v, float amax) {
  const float up = amax < 0x1p-64f ? 0x1p64f : 1.0f;
  const float r = amax > 0.0f ? 448.0f / (amax * up) : 0.0f;
  float f[8];
  unpack8(v, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = f[i] * up * r;
    const uint32_t b = __float_as_uint(t);
    f[i] = t == t ? __uint_as_float((b + 0x200u) & ~0x3ffu) : t;
  }
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], hi, true);
  return make_uint2(static_cast<uint32_t>(lo), static_cast<uint32_t>(hi));
}

__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __uint_as_float(dpp32<0xB1>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp32<0x4E>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp32<0x141>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp32<0x140>(__float_as_uint(v))));
  return v;
}

// One 1 x 128 block per 16 lanes; blocks = rows * KB (below 2^31).
__global__ __launch_bounds__(kThreads) void quantize_block_rows_kernel(uint32_t blocks, int K, uint32_t KB,
                                                                       const uint4* __restrict__ in,
                                                                       uint2* __restrict__ q,
                                                                       float* __restrict__ scale) {
  const uint32_t j = blockIdx.x * (kThreads / 16) + threadIdx.x / 16;
  const int n = threadIdx.x % 16;
  const bool active = j < blocks;
  const uint32_t row = active ? j / KB : 0, b = active ? j - row * KB : 0;
  const int chunks = K / 8, c = static_cast<int>(b) * 16 + n;
  const bool in_row = active && c < chunks;
  const int64_t at = static_cast<int64_t>(row) * chunks + c;
  const uint4 v = in_row ? in[at] : make_uint4(0u, 0u, 0u, 0u);
  const float amax = row_max(amax8(v));
  if (in_row) q[at] = codes8(v, amax);
  if (active && n == 0) scale[j] = amax / 448.0f;
}

// One 128 x 128 block per workgroup: 16 lanes along k, 16 rows at a time.
// Neighbouring workgroups hold neighbouring blocks of the same rows, so that
// together they walk whole rows: 128 x 768 x 2048 in 110 us (5.5 TB/s), 142 with
// the blocks below one another side by side.
__global__ __launch_bounds__(kThreads) void quantize_block_weights_kernel(int N, int K, int NB, int KB,
                                                                          const uint4* __restrict__ w,
                                                                          uint2* __restrict__ q,
                                                                          float* __restrict__ scale) {
  __shared__ float part[kThreads / kWave];
  const int rows_of = blockIdx.x / KB, b = blockIdx.x - rows_of * KB, e = rows_of / NB, nb = rows_of - e * NB;
  const int chunks = K / 8, c = b * 16 + static_cast<int>(threadIdx.x) % 16;
  const int r0 = nb * 128 + static_cast<int>(threadIdx.x) / 16;
  const int64_t base = (static_cast<int64_t>(e) * N + r0) * chunks + c;
  uint4 v[8];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = c < chunks && r0 + 16 * i < N ? w[base + static_cast<int64_t>(16 * i) * chunks] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, amax8(v[i]));
  amax = wave_max(amax);
  if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / kWave; ++i) amax = fmaxf(amax, part[i]);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c < chunks && r0 + 16 * i < N) q[base + static_cast<int64_t>(16 * i) * chunks] = codes8(v[i], amax);
  if (threadIdx.x == 0) scale[blockIdx.x] = amax / 448.0f;
}

}  // namespace

hipError_t launch_quantize_fp8_block_rows(int rows, int K, const void* in, uint8_t* q, float* scale, hipStream_t st) {
  const uint32_t KB = static_cast<uint32_t>(ceil_div(K, 128));
  const uint32_t blocks = static_cast<uint32_t>(rows) * KB;
  const unsigned grid = (blocks + kThreads / 16 - 1) / (kThreads / 16);
  quantize_block_rows_kernel<<<grid, kThreads, 0, st>>>(blocks, K, KB, static_cast<const uint4*>(in),
                                                        reinterpret_cast<uint2*>(q), scale);
  return hipGetLastError();
}

hipError_t launch_quantize_fp8_block_weights(int E, int N, int K, const void* w, uint8_t* q, float* scale,
                                             hipStream_t st) {
  const int NB = ceil_div(N, 128), KB = ceil_div(K, 128);
  const unsigned grid = static_cast<unsigned>(E) * static_cast<unsigned>(NB) * static_cast<unsigned>(KB);
  quantize_block_weights_kernel<<<grid, kThreads, 0, st>>>(N, K, NB, KB, static_cast<const uint4*>(w),
                                                           reinterpret_cast<uint2*>(q), scale);
  return hipGetLastError();
}

}  // namespace moe
