// Query rows of the 8-bit cache's attention kernels that hold 16 rows per operand: their key ranges and
// their 8-bit terms.
#pragma once

#include "tq_q8_attend.cuh"

namespace tq {

constexpr int kRows = 16;           // rows of an operand = N of the MMAs
constexpr int kTerm = kRows * 128;  // bytes of one 8-bit term of a Q or P operand

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

// Row (head hq, query token i) of sequence b, a whole warp: coordinates 4 lane .. 4 lane + 3 scaled by the row's power of
// two 2^-e and split into terms, four bytes each; returns e. A row with an infinity or a NaN becomes all NaN.
template <int GR>
__device__ __forceinline__ int row_terms(const Q8AttnArgs &a, int b, int hq, int i, bool live, int lane,
                                         uint32_t (&w)[GR][3]) {
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  if (live) {
    const long long off = b * a.qs.b + hq * a.qs.h + i * a.qs.t + 4 * lane;
    if (a.q_dtype == TQ_F32) load_vec<float, 4>(static_cast<const float *>(a.q) + off, x);
    else if (a.q_dtype == TQ_BF16) load_vec<__nv_bfloat16, 4>(static_cast<const __nv_bfloat16 *>(a.q) + off, x);
    else load_vec<__half, 4>(static_cast<const __half *>(a.q) + off, x);
  }
  uint32_t amax = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) amax = max(amax, __float_as_uint(x[k]) & 0x7fffffffu);
  amax = __reduce_max_sync(kFull, amax);
  const int e = row_exponent(amax);
  if (amax >= 0x7f800000u) {
#pragma unroll
    for (int gr = 0; gr < GR; ++gr)
#pragma unroll
      for (int k = 0; k < 3; ++k) w[gr][k] = 0x7f7f7f7fu;
    return e;
  }
  const float f = pow2i(-e);
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] *= f;
#pragma unroll
  for (int gr = 0; gr < GR; ++gr) {
    uint32_t lo[3], hi[3];
    split_terms(x[0], x[1], lo);
    split_terms(x[2], x[3], hi);
#pragma unroll
    for (int k = 0; k < 3; ++k) w[gr][k] = lo[k] | (hi[k] << 16);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] *= kGroupScale;
  }
  return e;
}

__device__ __forceinline__ void bar_wg(int wg) { asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory"); }

}  // namespace tq
