// Query rows of the 8-bit cache's attention kernels: their key ranges and their 8-bit terms.
#pragma once

#include "tq_q8_attend.cuh"

namespace tq {

// Query token i of a kPrefix call: of which sequence, its number in it, the sequence's lengths (prefix, own, query tokens).
struct Folded {
  int b, i, prefix, len, m;
};
__device__ __forceinline__ Folded folded(const Q8AttnArgs &a, int i) {
  Folded f;
  f.b = i / a.fold, f.i = i - f.b * a.fold;
  f.prefix = min(max(latest(a.prefix_lens + f.b), 0), a.max_prefix);
  f.len = min(max(latest(a.seq_lens + f.b), 0), a.own_max);
  f.m = a.new_lens ? min(max(latest(a.new_lens + f.b), 0), a.fold) : a.fold;
  return f;
}

// A row's key range: query token i of sequence b, whose length is len and whose query tokens number m.
template <int KIND = kWhole>
__device__ __forceinline__ int2 row_range(const Q8AttnArgs &a, int b, int i, int len, int m) {
  if (i >= m) return make_int2(0, 0);
  int beg = 0, end;
  if constexpr (KIND == kPrefix) {
    const Folded f = folded(a, i);
    if (f.i >= f.m) return make_int2(0, 0);
    end = f.prefix + f.len - f.m + f.i + 1;
    if (a.kbeg) beg = max(0, latest(a.kbeg + i));
    if (a.kend) end = latest(a.kend + i);
    end = min(end, f.prefix);
  } else {
    end = len - m + i + 1;
    if (a.kbeg) beg = max(0, latest(a.kbeg + (long long)b * a.n_q + i));
    if (a.kend) end = latest(a.kend + (long long)b * a.n_q + i);
    if constexpr (KIND == kOwn) {  // ranges count the prefix's slots
      const int prefix = min(max(latest(a.prefix_lens + b), 0), a.max_prefix);
      beg = max(0, beg - prefix);
      if (a.kend) end = max(end, 0) - prefix;
    }
    end = min(end, len);
  }
  return end > beg ? make_int2(beg, end) : make_int2(0, 0);
}

template <int KIND = kWhole>
__device__ __forceinline__ void seq_sizes(const Q8AttnArgs &a, int b, int *len, int *m, bool report) {
  if constexpr (KIND == kPrefix) {
    *len = a.max_len, *m = a.n_q;
  } else {
    int n = latest(a.seq_lens + b), q = a.new_lens ? latest(a.new_lens + b) : a.n_q;
    [[maybe_unused]] int prefix = 0;
    if constexpr (KIND == kOwn || KIND == kBoth) prefix = latest(a.prefix_lens + b);
    if (report && (n < 0 || n > a.max_len || q < 0 || q > a.n_q || prefix < 0 || prefix > a.max_prefix)) set_error(a.error, TQ_ERR_ARG);
    *len = min(max(n, 0), a.max_len);
    if constexpr (KIND == kBoth) *len += min(max(prefix, 0), a.max_prefix);
    *m = min(max(q, 0), a.n_q);
  }
}

// A query's slot, among those that its keys' slots count in.
template <int KIND>
__device__ __forceinline__ int query_slot(const Q8AttnArgs &a, int i, int len, int m) {
  if constexpr (KIND == kPrefix) {
    const Folded f = folded(a, i);
    return f.prefix + f.len - f.m + f.i;
  }
  return len - m + i;
}

template <int KIND>
__device__ __forceinline__ long long query_offset(const Q8AttnArgs &a, int b, int hq, int i) {
  if constexpr (KIND == kPrefix) b = i / a.fold, i -= b * a.fold;
  return b * a.qs.b + hq * a.qs.h + i * a.qs.t;
}

// a / b of numbers that are not negative: in 32 bits where they fit (64-bit divisions take some 100 instructions).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// The rows [r0, end) of unit x of a sequence, units of `unit` rows; kListed: of list *list.
template <int KIND>
__device__ __forceinline__ void unit_span(const Q8AttnArgs &a, int x, int unit, int *r0, int *end, int *list) {
  *list = 0, *r0 = x * unit, *end = a.group * a.n_q;
  if constexpr (KIND == kListed) {
    const int rows = a.group * a.span, units = (rows + unit - 1) / unit;
    *list = x / units;
    *r0 = *list * rows + (x - *list * units) * unit;
    *end = (int)min((long long)*end, ((long long)*list + 1) * rows);
  }
}
// kBoth: the prefix's length of sequence b, and a unit's tiles of 128 of its slots, the first one that its rows see (those of slots from lo to
// hi - 1), then of the sequence's own.
__device__ __forceinline__ int prefix_of(const Q8AttnArgs &a, int b) { return min(max(latest(a.prefix_lens + b), 0), a.max_prefix); }
struct BothTiles {
  int prefix, first, own;  // tiles of the prefix; the first of them; the first of the own ones
  int total;
};
__device__ __forceinline__ BothTiles both_tiles(int prefix, int lo, int hi) {
  BothTiles t;
  t.first = lo / 128, t.own = max(lo - prefix, 0) / 128;
  t.prefix = max(0, (min(hi, prefix) + 127) / 128 - t.first);
  if (lo >= prefix) t.prefix = 0;
  t.total = t.prefix + (hi > prefix ? (hi - prefix + 127) / 128 - t.own : 0);
  return t;
}
// Tiles of 128 slots that a unit goes through whose rows see slots from lo to hi - 1 (kListed: of two list entries each; a block of
// number j is among the first j + 1 of its list).
template <int KIND>
__device__ __forceinline__ int unit_tiles(const Q8AttnArgs &a, int b, int lo, int hi) {
  if constexpr (KIND == kListed) return (min(a.n_blocks, (hi + kQ8Block - 1) / kQ8Block) + 1) / 2;
  if constexpr (KIND == kBoth) return both_tiles(prefix_of(a, b), lo, hi).total;
  return (hi + 127) / 128 - lo / 128;
}
// The blocks of entries k and k + 1 (k even) of list `list` of (sequence, head) bh, -1 for none that counts.
__device__ __forceinline__ void list_entries(const Q8AttnArgs &a, long long bh, int list, int k, int (&blk)[2]) {
  const int32_t *p = a.blocks + (bh * a.lists + list) * a.n_blocks + k;
  int e[3];
#pragma unroll
  for (int j = 0; j < 3; ++j) e[j] = k + j > 0 && k + j <= a.n_blocks ? latest(p + j - 1) : -1;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    blk[j] = e[j + 1] > e[j] && e[j + 1] < a.c.nblk && (e[j] >= 0 || k + j == 0) ? e[j + 1] : -1;
    bad |= e[j + 1] >= 0 && blk[j] < 0;
  }
  if (bad) set_error(a.error, TQ_ERR_ARG);
}
// The sources of a unit's tile whose rows see slots from lo to hi - 1: of its blocks blk[k], the first at slot `base` of the rows' count, which
// slots they begin at, where they lie (src, -1 for one of which no row sees a token) and how many bytes of a plane are copied: whole
// K-steps of the value product.
__device__ __forceinline__ float4 tile_sources(const Q8AttnArgs &a, const Q8Cache &c, long long bh, const int (&blk)[2], int base, int lo, int hi,
                                               long long (&src)[2], int (&bytes)[2], int (&at)[2]) {
  long long v[2];
  bool use[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    at[k] = base + max(blk[k], 0) * kQ8Block;
    const int m = min(kQ8Block, hi - at[k]);
    use[k] = blk[k] >= 0 && m > 0 && at[k] + kQ8Block > lo;
    v[k] = bh * c.nblk + blk[k];
    bytes[k] = (m + 31) / 32 * 32 * kD;
  }
  q8_two_blocks(c, v, use, a.error, src);
#pragma unroll
  for (int k = 0; k < 2; ++k) bytes[k] = src[k] < 0 ? 0 : bytes[k];
  return q8_two_scales(c, src);
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
// Coordinates 4 lane .. 4 lane + 3 of row (head hq, query token i) of sequence b; zeros for a row that is not live.
template <int KIND = kWhole>
__device__ __forceinline__ void row_coords(const Q8AttnArgs &a, int b, int hq, int i, bool live, int lane, float (&x)[4]) {
  x[0] = x[1] = x[2] = x[3] = 0.f;
  if (!live) return;
  const long long off = query_offset<KIND>(a, b, hq, i) + 4 * lane;
  if (a.q_dtype == TQ_F32) load_vec<float, 4>(static_cast<const float *>(a.q) + off, x);
  else if (a.q_dtype == TQ_BF16) load_vec<__nv_bfloat16, 4>(static_cast<const __nv_bfloat16 *>(a.q) + off, x);
  else load_vec<__half, 4>(static_cast<const __half *>(a.q) + off, x);
}
// Few rows: T e5m2 terms.
template <int T, int KIND = kWhole>
__device__ __forceinline__ int row_e5m2(const Q8AttnArgs &a, int b, int hq, int i, bool live, int lane, uint32_t (&w)[T]) {
  float x[4];
  row_coords<KIND>(a, b, hq, i, live, lane, x);
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
template <int KIND = kWhole>
__device__ __forceinline__ void load_rows(const Q8AttnArgs &a, int b, int h, int m, int first_row, int lane, uint2 (&raw)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int row = min(first_row + k, a.group * a.n_q - 1), i = row / a.group;
    const long long off = query_offset<KIND>(a, b, h * a.group + row - i * a.group, min(i, max(m - 1, 0))) + 4 * lane;
    raw[k] = latest(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.q) + off));
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

// A row's part of the prefix (coordinates d .. d + N - 1), as it lies: asked for before results are stored, behind which it would wait.
template <int N>
struct Prior {
  float x[N], was, l, lr;
};
template <int KIND, int N>
__device__ __forceinline__ Prior<N> prior_of(const Q8AttnArgs &a, int b, int hq, int i, int d) {
  Prior<N> p{};
  if constexpr (KIND == kOwn) {
    const float *row = a.prior + (((long long)hq * a.batch + b) * a.n_q + i) * kPriorRow;
    if constexpr (N == 1) p.x[0] = latest(row + d);
    else load_vec<float, N>(row + d, p.x);
    p.was = latest(row + kD), p.l = latest(row + kD + 1), p.lr = latest(row + kD + 2);
  }
  return p;
}
// The reference of a row's own part (its sums are relative to 2^m) and that of the prefix, and the factors that bring either to it.
struct Joined {
  float m, by, own;  // the reference, the prefix part's factor, the own part's
};
__device__ __forceinline__ Joined joined(float was, float m) {
  Joined p;
  p.m = fmaxf(m, was);
  p.by = was == -INFINITY ? 1.f : ex2_approx(was - p.m);  // without a maximum: zeros (or NaN)
  p.own = m == -INFINITY ? 1.f : ex2_approx(m - p.m);
  return p;
}

// Coordinate d of a row: x = sum 2^(t - top + shift) v, l and lr the same of 1 (lr of the numbers as they entered x). Written to where the kind's
// results go, joined with the prefix's part where there is one.
template <int KIND>
__device__ __forceinline__ void finish_row(const Q8AttnArgs &a, int b, int hq, int i, int d, float x, float top, float l, float lr, float shift,
                                           const Prior<1> &prior) {
  if constexpr (KIND == kPrefix) {
    float *row = a.prior + ((long long)hq * a.n_q + i) * kPriorRow;
    row[d] = x;
    if (d == 0) row[kD] = top - shift, row[kD + 1] = l, row[kD + 2] = lr;
    return;
  }
  float m = top;
  if constexpr (KIND == kOwn) {
    const Joined p = joined(prior.was, top - shift);
    x = fmaf(prior.x[0], p.by, x * p.own);
    l = fmaf(prior.l, p.by, l * p.own);
    lr = fmaf(prior.lr, p.by, lr * p.own);
    m = p.m + shift;
  }
  const float y = lr == 0.f ? 0.f : x / lr;
  const long long off = b * a.os.b + hq * a.os.h + i * a.os.t + d;
  if (a.out_dtype == TQ_F32) static_cast<float *>(a.out)[off] = y;
  else if (a.out_dtype == TQ_BF16) static_cast<__nv_bfloat16 *>(a.out)[off] = __float2bfloat16_rn(y);
  else static_cast<__half *>(a.out)[off] = __float2half_rn(y);
  if (a.lse && d == 0) a.lse[((long long)b * a.heads_q + hq) * a.n_q + i] = (m + log2f(l) - shift) * kLn2;
}

__device__ __forceinline__ void bar_wg(int wg) { asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory"); }

}  // namespace tq
