// Top-k selection on 16-lane DPP rows, shared by the router's kernels.
#pragma once

#include "moe_internal.h"

namespace moe {

// A selection key orders (logit, index): the logit's order bits (NaN lowest;
// -0 counted as +0, so equal logits tie on the index) above the complement of
// the index. Keys are unique and above 0; the largest is the next expert.
__device__ __forceinline__ uint64_t sel_key(float v, int e) {
  const float c = v + 0.0f;  // -0 -> +0
  const uint32_t b = __float_as_uint(c);
  const uint32_t o = (c != c) ? 0u : ((b & 0x80000000u) ? ~b : (b | 0x80000000u));
  return (static_cast<uint64_t>(o) << 32) | static_cast<uint32_t>(~e);
}

__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);  // o = 0: a NaN
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp32(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, false));
}

// Quad swaps (quad_perm [1,0,3,2] and [2,3,0,1]), then half-row and row
// mirrors: every lane of a 16-lane row ends with the row's maximum (or sum).
__device__ __forceinline__ uint64_t row_max_key(uint64_t k) {
#define RM_STEP(CTRL)                                                                                      \
  {                                                                                                        \
    const uint64_t o = (static_cast<uint64_t>(dpp32<CTRL>(static_cast<uint32_t>(k >> 32))) << 32) |       \
                       dpp32<CTRL>(static_cast<uint32_t>(k));                                              \
    k = o > k ? o : k;                                                                                     \
  }
  RM_STEP(0xB1) RM_STEP(0x4E) RM_STEP(0x141) RM_STEP(0x140)
#undef RM_STEP
  return k;
}

__device__ __forceinline__ float row_sum(float v) {
  v += __uint_as_float(dpp32<0xB1>(__float_as_uint(v)));
  v += __uint_as_float(dpp32<0x4E>(__float_as_uint(v)));
  v += __uint_as_float(dpp32<0x141>(__float_as_uint(v)));
  v += __uint_as_float(dpp32<0x140>(__float_as_uint(v)));
  return v;
}

}  // namespace moe
