// Eight numbers in 16 bytes, for results that are only summed again (a token's
// k expert results): as many bytes as bf16, each number off by no more than in
// bf16 (2^-8 of itself), and by at most 2^-13 of the largest of the eight if
// that is 2^-114 or more.
//
// With s the exponent field of the largest magnitude m (m < 2^(s-126)), number
// v is held as L = |v| 2^(139-s) < 8192: from 128 on as a whole number (off
// by 2^-14 of 2^(s-126) at most), below as bf16. Both grow by 1 from code to code, the
// second by 128 per octave, and meet at 128, so one 14-bit code u holds them:
//   u <= kLow: the bf16 with bits u + kBf16Base, less the one for u = 0 (which
//     matters from 2^-62 of the largest down),   u > kLow: L = u - kLow + 128.
// A half word is the sign, u, and one bit of s (bit i of s in the low half of
// word i, bit i + 4 in the high half). s = 255, where m is infinite or NaN: the
// upper 15 bits of each one's bf16. s below 13 (m under 2^-114) counts as 13.
//
// One step for all eight (15 bits and the exponent) costs half the operations
// (4096 skewed tokens 379 us instead of 390, 192 tokens 149 instead of 152) and
// loses the small ones: beside a column 1024 times the others, as residual
// streams have, those are off by 2.7% where bf16 gives 0.17%. bf16 rows cost
// less still, and leave y off by 0.0025 instead of 0.0020.
#pragma once
#include "moe_internal.h"

namespace moe {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
constexpr uint32_t kShared8Mask = 0xfffefffeu;
constexpr uint32_t kBf16Of128 = 0x4300, kLow = 0x3fff - (8192 - 128), kBf16Base = kBf16Of128 - kLow;

// s of eight numbers whose largest magnitude is m (NaN if one is), and the factor for shared8_word.
__device__ __forceinline__ uint32_t shared8_exponent(float m, float& f) {
  const uint32_t e = max(__float_as_uint(m) >> 23, 13u), s = min(e, 255u);
  f = __uint_as_float(s == 255 ? 127u << 23 : (266u - s) << 23);  // 2^(139-s)
  return s;
}

// Word i: numbers 2 i (low half) and 2 i + 1.
__device__ __forceinline__ uint32_t shared8_word(float a, float b, uint32_t s, float f, int i) {
  const float x = a * f, y = b * f;
  const uint32_t h = pack_bf16x2(x, y);
  // |x| + 2^23: the whole number nearest to |x| in the lower bits
  const uint32_t n = __builtin_amdgcn_perm(__float_as_uint(fabsf(y) + 0x1p23f), __float_as_uint(fabsf(x) + 0x1p23f),
                                           0x05040100u);
  constexpr uint16_t k128 = 2 * kBf16Of128, kBase = 2 * kBf16Base;
  const u16x2 whole = __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, n), u16x2{128, 128});
  const u16x2 bits = __builtin_bit_cast(u16x2, h) << 1;  // without the sign
  const u16x2 low = __builtin_elementwise_sub_sat(__builtin_elementwise_min(bits, u16x2{k128, k128}), u16x2{kBase, kBase});
  const u16x2 u = whole * static_cast<uint16_t>(2) + low;  // 2 u
  uint32_t v = __builtin_bit_cast(uint32_t, u) | (h & 0x80008000u);
  asm("" : "+v"(v));  // a select, not a branch around all of this
  v = s == 255 ? h : v;
  return (v & kShared8Mask) | (((s | s << 12) >> i) & ~kShared8Mask);
}

__device__ __forceinline__ float shared8_number(uint32_t u) {
  const float low = __uint_as_float((u + kBf16Base) << 16) - __uint_as_float(kBf16Base << 16);  // u = 0 is zero
  return u > kLow ? static_cast<float>(u - (kLow - 128)) : low;
}

__device__ __forceinline__ void shared8_unpack(const uint4& v, float* o) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) bits |= (w[i] & ~kShared8Mask) << i;
  const uint32_t s = (bits & 0xf) | (bits >> 12 & 0xf0);
  const uint32_t f = (s - 12) << 23;  // 2^(s-139)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = shared8_number(w[i] >> 1 & 0x3fff) * __uint_as_float(f | (w[i] << 16 & 0x80000000u));
    o[2 * i + 1] = shared8_number(w[i] >> 17 & 0x3fff) * __uint_as_float(f | (w[i] & 0x80000000u));
  }
  if (s == 255) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __uint_as_float((w[i] & kShared8Mask) << 16);
      o[2 * i + 1] = __uint_as_float(w[i] & 0xfffe0000u);
    }
  }
}

}  // namespace moe
