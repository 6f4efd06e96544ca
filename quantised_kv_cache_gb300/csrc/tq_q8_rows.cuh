// Query rows of the 8-bit cache's attention kernels: their key ranges and their 8-bit terms.
#pragma once

#include "tq_q8_attend.cuh"

namespace tq {

// A row's key range: query token i of sequence b, whose length is len and whose query tokens number m.
__device__ __forceinline__ int2 row_range(const Q8AttnArgs &a, int b, int i, int len, int m) {
  if (i >= m) return make_int2(0, 0);
  int beg = 0, end = len - m + i + 1;
  if (a.kbeg) beg = max(0, __ldg(a.kbeg + (long long)b * a.n_q + i));
  if (a.kend) end = __ldg(a.kend + (long long)b * a.n_q + i);
  end = min(end, len);
  return end > beg ? make_int2(beg, end) : make_int2(0, 0);
}

__device__ __forceinline__ void seq_sizes(const Q8AttnArgs &a, int b, int *len, int *m, bool report) {
  int n = __ldg(a.seq_lens + b), q = a.new_lens ? __ldg(a.new_lens + b) : a.n_q;
  if (report && (n < 0 || n > a.max_len || q < 0 || q > a.n_q)) set_error(a.error, TQ_ERR_ARG);
  *len = min(max(n, 0), a.max_len);
  *m = min(max(q, 0), a.n_q);
}

// The bits of a row's largest magnitude, a lane holding four of its coordinates.
__device__ __forceinline__ uint32_t row_top(const float (&x)[4]) {
  uint32_t amax = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) amax = max(amax, __float_as_uint(x[k]) & 0x7fffffffu);
  return __reduce_max_sync(kFull, amax);
}

// A row's terms, four bytes each, of its coordinates times 2^-e (e is returned); a whole warp. A row with an infinity or a
// NaN becomes all NaN. Many rows: e4m3, e4m3, e5m2.
__device__ __forceinline__ int row_terms(const float (&x)[4], uint32_t (&w)[3]) {
  const uint32_t amax = row_top(x);
  const int e = row_exponent(amax, 7);
  const float f = pow2i(-e);
  uint32_t lo[3], hi[3];
  split_terms(x[0] * f, x[1] * f, lo);
  split_terms(x[2] * f, x[3] * f, hi);
#pragma unroll
  for (int k = 0; k < 3; ++k) w[k] = amax >= 0x7f800000u ? 0x7f7f7f7fu : lo[k] | (hi[k] << 16);
  return e;
}
// Few rows: T e5m2 terms.
template <int T>
__device__ __forceinline__ int row_e5m2(const Q8AttnArgs &a, int b, int hq, int i, bool live, int lane, uint32_t (&w)[T]) {
  float x[4] = {0.f, 0.f, 0.f, 0.f};  // coordinates 4 lane .. 4 lane + 3 of row (head hq, query token i) of sequence b
  if (live) {
    const long long off = b * a.qs.b + hq * a.qs.h + i * a.qs.t + 4 * lane;
    if (a.q_dtype == TQ_F32) load_vec<float, 4>(static_cast<const float *>(a.q) + off, x);
    else if (a.q_dtype == TQ_BF16) load_vec<__nv_bfloat16, 4>(static_cast<const __nv_bfloat16 *>(a.q) + off, x);
    else load_vec<__half, 4>(static_cast<const __half *>(a.q) + off, x);
  }
  const uint32_t amax = row_top(x);
  const int e = row_exponent(amax, 14);
  const float f = pow2i(-e);
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] *= f;
  uint32_t lo[T], hi[T];
  split_e5m2<T>(x[0], x[1], lo);
  split_e5m2<T>(x[2], x[3], hi);
#pragma unroll
  for (int k = 0; k < T; ++k) w[k] = amax >= 0x7f800000u ? 0x7f7f7f7fu : lo[k] | (hi[k] << 16);
  return e;
}

// Many rows: 4 coordinates a lane of eight rows of 16-bit queries from first_row on, their loads in flight at once: no branch in their
// way, a row that is not there loads another (and counts as 0).
__device__ __forceinline__ void load_rows(const Q8AttnArgs &a, int b, int h, int m, int first_row, int lane, uint2 (&raw)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int row = min(first_row + k, a.group * a.n_q - 1), i = row / a.group;
    const long long off = b * a.qs.b + (h * a.group + row - i * a.group) * a.qs.h + min(i, max(m - 1, 0)) * a.qs.t + 4 * lane;
    raw[k] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.q) + off));
  }
}
__device__ __forceinline__ void row_floats(const Q8AttnArgs &a, uint2 raw, bool live, float (&x)[4]) {
  if (a.q_dtype == TQ_BF16) {
    x[0] = __uint_as_float(raw.x << 16), x[1] = __uint_as_float(raw.x & 0xffff0000u);
    x[2] = __uint_as_float(raw.y << 16), x[3] = __uint_as_float(raw.y & 0xffff0000u);
  } else {
    const float2 lo = __half22float2(*reinterpret_cast<const __half2 *>(&raw.x));
    const float2 hi = __half22float2(*reinterpret_cast<const __half2 *>(&raw.y));
    x[0] = lo.x, x[1] = lo.y, x[2] = hi.x, x[3] = hi.y;
  }
  if (!live) x[0] = x[1] = x[2] = x[3] = 0.f;
}

// Few rows: term k of row r is operand row k NR + r. An accumulator's columns are summed over the terms, the small ones first.
__host__ __device__ constexpr int stacked_rows(int NR, int T) { return T * NR < 16 ? 16 : T * NR; }
template <int NR, int T>
__device__ __forceinline__ void tmem_term_sums(uint32_t taddr, float (&out)[NR]) {
  constexpr int C = NR * T < 32 ? NR * T : 32, kParts = NR * T / C;
#pragma unroll
  for (int part = kParts - 1; part >= 0; --part) {
    float v[C];
    tmem_ld_cols<C>(taddr + part * C, v);
#pragma unroll
    for (int k = C / NR - 1; k >= 0; --k)
#pragma unroll
      for (int r = 0; r < NR; ++r)
        out[r] = part == kParts - 1 && k == C / NR - 1 ? v[k * NR + r] : out[r] + v[k * NR + r];
  }
}

__device__ __forceinline__ void bar_wg(int wg) { asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory"); }

}  // namespace tq
