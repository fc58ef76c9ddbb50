// 8-bit integer codes: scale = amax / 127, code = the whole number nearest to
// 127 v / amax, halves to even (0 and 0 for amax = 0).
//
// For bf16 v the codes are those of exact arithmetic, without a division per
// element: q = 127 v / amax is taken as v * (127 / amax) in fp32, off by less
// than 2^-22 of q. A border between codes is a half m = odd / 2 below 127. With V
// and A the 8-bit significands of v and amax, q - m is a multiple of
// 1 / (2 A 2^s) where q = 127 V / (A 2^s), so it is zero or at least
// 1 / (254 V) > 2^-16 of q. Rounding the product to 18 fraction bits moves it by
// at most 2^-19 of itself and leaves m (8 bits) in place: a half lands on the
// border exactly, and everything else stays on its side of it.
#pragma once
#include "moe_internal.h"
#include "select.h"

namespace moe {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// The largest magnitude's bits among bf16 values: without the sign they order
// like the values, infinities and then NaN above every number.
__device__ __forceinline__ u16x2 amax_bits(u16x2 m, const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
  return m;
}
__device__ __forceinline__ uint32_t amax_bits(u16x2 m) { return max(static_cast<uint32_t>(m.x), static_cast<uint32_t>(m.y)); }

// What a block's largest magnitude (bits of its bf16) makes of its values. A
// block with an infinity or a NaN has codes 0 and scale NaN, so that whatever is
// computed from it is NaN.
struct CodeFactor {
  float up, r, scale;  // up lifts blocks below 2^-64 by 2^64 (exact), so that 127 / amax stays finite
  __device__ __forceinline__ explicit CodeFactor(uint32_t bits) {
    const float amax = __uint_as_float(bits << 16);
    const bool finite = bits < 0x7f80u;
    up = amax < 0x1p-64f ? 0x1p64f : 1.0f;
    r = finite && amax > 0.0f ? 127.0f / (amax * up) : 0.0f;
    scale = finite ? amax / 127.0f : __builtin_nanf("");
  }
};

// The code of t = 127 v / amax in the low byte: adding 1.5 * 2^23 rounds to a
// whole number, halves to even. NaN (a non-finite value times r = 0) gives 0.
__device__ __forceinline__ uint32_t code_bits(float t) { return __float_as_uint(t + 12582912.0f); }
__device__ __forceinline__ float snap18(float t) { return __uint_as_float((__float_as_uint(t) + 0x10u) & ~0x1fu); }
__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0c0c0400u), __builtin_amdgcn_perm(b, a, 0x0c0c0400u),
                               0x05040100u);
}

__device__ __forceinline__ uint2 codes8(const uint4& v, const CodeFactor& f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[2 * i] = code_bits(snap18(__uint_as_float(w[i] << 16) * f.up * f.r));
    c[2 * i + 1] = code_bits(snap18(__uint_as_float(w[i] & 0xffff0000u) * f.up * f.r));
  }
  return make_uint2(bytes4(c[0], c[1], c[2], c[3]), bytes4(c[4], c[5], c[6], c[7]));
}

// The same for a block of fp32 sums whose largest magnitude is m (NaN if one is).
// The hardware's reciprocal is off by about 1 ulp, which moves a value's code only
// if it is that close to a border: the code is off by less than 0.5 + 2^-15 still.
// It does not return subnormal numbers, which from 2^126 on its result would be:
// blocks above 2^64 are brought down by 2^64, as those below 2^-64 are lifted.
struct SumFactor {
  float up, r, scale;
  __device__ __forceinline__ explicit SumFactor(float m) {
    const bool finite = m < __builtin_inff();
    up = m < 0x1p-64f ? 0x1p64f : m > 0x1p64f ? 0x1p-64f : 1.0f;
    r = finite && m > 0.0f ? 127.0f * __builtin_amdgcn_rcpf(m * up) : 0.0f;
    scale = finite ? m * (1.0f / 127.0f) : __builtin_nanf("");
  }
  __device__ __forceinline__ uint32_t code(float v) const { return code_bits(v * up * r); }
};

// Code i (0 to 3) of a word as a number.
__device__ __forceinline__ float code_value(uint32_t w, int i) {
  return static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
}

// One row [K] of bf16 by a wavefront: codes and scale. The first 4096 columns
// stay in registers between the maximum and the codes.
template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v);
__device__ __forceinline__ void quantize_row(int K, const uint4* __restrict__ in, uint2* __restrict__ q,
                                             float* __restrict__ scale) {
  constexpr int CPL = 8;
  const int lane = threadIdx.x % kWave, chunks = K / 8;
  uint4 v[CPL];
  u16x2 m{0, 0};
#pragma unroll
  for (int i = 0; i < CPL; ++i) v[i] = lane + i * kWave < chunks ? in[lane + i * kWave] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < CPL; ++i) m = amax_bits(m, v[i]);
  for (int c = lane + CPL * kWave; c < chunks; c += kWave) m = amax_bits(m, in[c]);
  const uint32_t r = group_max<16>(amax_bits(m));
  const CodeFactor f(max(max(__builtin_amdgcn_readlane(r, 0), __builtin_amdgcn_readlane(r, 16)),
                         max(__builtin_amdgcn_readlane(r, 32), __builtin_amdgcn_readlane(r, 48))));
#pragma unroll
  for (int i = 0; i < CPL; ++i)
    if (lane + i * kWave < chunks) q[lane + i * kWave] = codes8(v[i], f);
  for (int c = lane + CPL * kWave; c < chunks; c += kWave) q[c] = codes8(in[c], f);
  if (lane == 0) *scale = f.scale;
}

// Maximum over the 8 or 16 neighbouring lanes of a group, in every lane of it.
template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  v = max(v, dpp32<0xB1>(v));
  v = max(v, dpp32<0x4E>(v));
  v = max(v, dpp32<0x141>(v));
  if constexpr (LANES == 16) v = max(v, dpp32<0x140>(v));
  return v;
}

}  // namespace moe
