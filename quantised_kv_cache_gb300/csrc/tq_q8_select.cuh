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

// Four signed bytes as fp16 numbers: 1024 + (b + 128) has b + 128 as its lowest bits.
__device__ __forceinline__ uint2 bytes_h4(uint32_t w) {
  w ^= 0x80808080u;
  uint32_t p = __byte_perm(w, 0x64646464u, 0x4140), q = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 base = __half2half2(__ushort_as_half(0x6480));  // 1152
  const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&p), base), y = __hsub2(*reinterpret_cast<__half2 *>(&q), base);
  return make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
}

}  // namespace tq
