// Eight numbers in 16 bytes: 15 bits each and one exponent, for results that
// are only summed again (a token's k expert results): as many bytes as bf16,
// and an error of at most 2^-14 of the largest of the eight where bf16 has 2^-8 of
// each.
//
// With s the exponent field of the largest magnitude m (m < 2^(s-126)), number
// j is q_j 2^(s-125) / 32767, q_j = round(v_j 2^(125-s) 32767) / 2 in 15 bits,
// in the upper 15 bits of its half word; the half words' lowest bits are s (bit
// i of it in the low half of word i, bit i + 4 in the high half). s = 255, where
// m is 2^125 or more, infinite or NaN: the upper 15 bits of each one's bf16.
// s below 20 (m under 2^-106) counts as 20.
#pragma once
#include "moe_internal.h"

namespace moe {

constexpr uint32_t kShared8Mask = 0xfffefffeu;

// s of eight numbers whose largest magnitude is m (NaN if one is), and the factor for shared8_word.
__device__ __forceinline__ uint32_t shared8_exponent(float m, float& f) {
  const uint32_t e = max(__float_as_uint(m) >> 23, 20u), s = e > 251 ? 255 : e;
  f = __uint_as_float((252u - min(s, 251u)) << 23);  // 2^(125-s)
  return s;
}

// Word i: numbers 2 i (low half) and 2 i + 1.
__device__ __forceinline__ uint32_t shared8_word(float a, float b, uint32_t s, float f, int i) {
  uint32_t v = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pknorm_i16(a * f, b * f)) << 1;
  if (s == 255) v = pack_bf16x2(a, b);
  return (v & kShared8Mask) | (((s | s << 12) >> i) & ~kShared8Mask);
}

__device__ __forceinline__ void shared8_unpack(const uint4& v, float* o) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) bits |= (w[i] & ~kShared8Mask) << i;
  const uint32_t s = (bits & 0xf) | (bits >> 12 & 0xf0);
  const float f = __uint_as_float((s + 2) << 23) * (1.0f / 32767.0f);  // 2^(s-125) / 32767
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = static_cast<float>(static_cast<int32_t>(w[i] << 16) >> 17) * f;
    o[2 * i + 1] = static_cast<float>(static_cast<int32_t>(w[i]) >> 17) * f;
    if (s == 255) {
      o[2 * i] = __uint_as_float((w[i] & kShared8Mask) << 16);
      o[2 * i + 1] = __uint_as_float(w[i] & 0xfffe0000u);
    }
  }
}

}  // namespace moe
