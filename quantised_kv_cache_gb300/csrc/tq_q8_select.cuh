// Scores of blocks as ordered numbers, for the kernels that form and compare them (tq_q8_select).
#pragma once

#include "tq_q8.cuh"

namespace tq {

constexpr uint32_t kAlways = 0xffffffffu;  // a block that is taken whatever its score

// order-preserving; never kAlways; 0 below all numbers
__device__ __forceinline__ uint32_t score_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

}  // namespace tq
