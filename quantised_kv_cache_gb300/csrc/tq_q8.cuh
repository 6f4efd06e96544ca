// Shared by the 8-bit cache's kernels (TQ_SCHEME_Q8) and the rotary kernels: the block layout,
// e4m3 conversions, block scales, and the sines and cosines of rotary positions.
//
// A block holds 64 tokens' keys, then values, as e4m3 codes (include/tq.h, "Q8 records"): token t,
// coordinate c of a plane at 1024 (t / 8) + 128 (c / 16) + 16 (t % 8) + c % 16. Groups of 8 tokens x
// 16 bytes are the tensor cores' core matrices, so a key plane is a K-major operand (128 bytes from
// one 16-coordinate column to the next, 1024 from one token group to the next) and a value plane an
// MN-major one (the same two strides) without any rearrangement.
#pragma once

#include "tq_ptx.cuh"
#include "tq_q8.h"

namespace tq {

constexpr float kQ8Largest = 3.1901471898837980e38f;  // 1.875 * 2^127: 240 * 2^120

__device__ __forceinline__ int q8_off(int t, int c) { return (t >> 3) * 1024 + (c >> 4) * 128 + (t & 7) * 16 + (c & 15); }

// Physical block of virtual block `v` (= sequence-head * blocks per sequence + j), -1 (and the error
// word set) for a table entry outside the pool.
__device__ __forceinline__ long long q8_block(const int32_t *btab, int pool_blocks, long long v, int *error) {
  if (btab == nullptr) return v;
  const int pb = __ldg(btab + v);
  if (pb < 0 || pb >= pool_blocks) {
    set_error(error, TQ_ERR_ARG);
    return -1;
  }
  return pb;
}

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127
__device__ __forceinline__ int log2i(float p) { return (__float_as_int(p) >> 23) - 127; }   // p = 2^e > 0

// The least e >= kQ8MinExp with amax <= 448 * 2^e (448 = 1.75 * 2^8; amax >= 0 finite, given by its bits).
__device__ __forceinline__ int q8_exponent(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, kQ8MinExp);  // zero and subnormal numbers have a small exponent field: the minimum
}

// (lo, hi) -> two e4m3 bytes (lo in the low one), to nearest even, saturated to +-448
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t cvt_e5m2x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// two e4m3 / e5m2 bytes -> floats (exact)
__device__ __forceinline__ float2 e4m3x2_f(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Four e4m3 codes times 2^shift, rounded to e4m3 again.
__device__ __forceinline__ uint32_t e4m3x4_scaled(uint32_t w, float f) {
  const float2 a = e4m3x2_f(w & 0xffffu), b = e4m3x2_f(w >> 16);
  return cvt_e4m3x2(a.x * f, a.y * f) | (cvt_e4m3x2(b.x * f, b.y * f) << 16);
}

// Elements of the input types as float, N consecutive ones from an address aligned to N elements.
template <typename T, int N>
__device__ __forceinline__ void load_vec(const T *p, float (&v)[N]) {
  constexpr int kBytes = N * (int)sizeof(T);
  static_assert(kBytes % 8 == 0, "");
  uint32_t w[kBytes / 4];
  if constexpr (kBytes % 16 == 0) {
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) {
      const uint4 x = reinterpret_cast<const uint4 *>(p)[i];
      w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kBytes / 8; ++i) {
      const uint2 x = reinterpret_cast<const uint2 *>(p)[i];
      w[2 * i] = x.x, w[2 * i + 1] = x.y;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (sizeof(T) == 4) {
      v[i] = __uint_as_float(w[i]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      v[i] = __uint_as_float((i & 1) ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
    } else {
      const __half2 h = *reinterpret_cast<const __half2 *>(&w[i / 2]);
      v[i] = (i & 1) ? __high2float(h) : __low2float(h);
    }
  }
}
template <typename T>
__device__ __forceinline__ T to_type(float x) {
  if constexpr (sizeof(T) == 4) return x;
  else if constexpr (std::is_same<T, __nv_bfloat16>::value) return __float2bfloat16_rn(x);
  else return __float2half_rn(x);
}
template <typename T, int N>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[N]) {
  alignas(16) T x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = to_type<T>(v[i]);
  constexpr int kBytes = N * (int)sizeof(T);
  if constexpr (kBytes % 16 == 0) {
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(x)[i];
  } else {
#pragma unroll
    for (int i = 0; i < kBytes / 8; ++i) reinterpret_cast<uint2 *>(p)[i] = reinterpret_cast<const uint2 *>(x)[i];
  }
}

// cos and sin of 2 pi (pos * freq mod 1), freq in units of 2^-64 turns: the 64-bit product wraps at
// whole turns, so the angle is off by less than 2^-32 turns from its cut and 2^-34, half a unit of freq 2^31 times, at any position. The top 2 bits (rounded) are the
// quadrant; the rest, |x| <= pi / 4, is kept in two parts (x + lo: the integer and 2 pi / 2^32 each split where
// float32 ends) and goes through the Taylor polynomials of sine (to x^9, the next
// term is below 2e-9) and cosine (to x^10, below 2e-10), so that little more than the last rounding is lost.
__device__ __forceinline__ void rope_sincos(int pos, unsigned long long freq, float *c, float *s) {
  const uint32_t u = (uint32_t)(((unsigned long long)(long long)pos * freq) >> 32);
  const uint32_t q = (u + 0x20000000u) >> 30;
  const int r = (int)(u - (q << 30));
  const float kUnit = 1.46291811e-9f, kUnitLo = -4.07094027e-17f;  // 2 pi / 2^32 and what float32 drops of it
  const float rh = (float)(r & ~63), rl = (float)(r & 63);
  const float x = __fmul_rn(rh, kUnit);
  const float lo = fmaf(rh, kUnit, -x) + fmaf(rl, kUnit, rh * kUnitLo);
  const float z = x * x;
  float sn = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
  sn = fmaf(z, sn, 8.3333333e-3f);
  sn = fmaf(z, sn, -1.6666667e-1f);
  sn = fmaf(x * z, sn, lo) + x;
  float cs = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
  cs = fmaf(z, cs, -1.3888889e-3f);
  cs = fmaf(z, cs, 4.1666667e-2f);
  cs = fmaf(z, cs, -0.5f);
  cs = fmaf(z, cs, -x * lo) + 1.f;
  const bool swap = q & 1;
  const float a = swap ? cs : sn, b = swap ? sn : cs;
  *s = (q & 2) ? -a : a;
  *c = ((q + 1) & 2) ? -b : b;
}

// One coordinate of a rotated pair: x cos + other * (-sin or +sin), with one rounding of its own in
// the product and one in the sum, so that every kernel rotates to the same bits.
__device__ __forceinline__ float rope_turn(float x, float other, float c, float s) {
  return __fmaf_rn(other, s, __fmul_rn(x, c));
}

}  // namespace tq
