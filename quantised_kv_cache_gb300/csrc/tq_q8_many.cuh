// Attention over the 8-bit cache for many query rows per KV head (tq_q8_attention): prompts. Results of 16 bits.
//
// Here a row (query token, head of the group) is an accumulator lane: S = Q K^T for 128 rows x 128 tokens, keys as
// the K-major B operand and values as the MN-major B operand as they lie in the cache; the queries' 8-bit terms
// sit in shared memory for the whole unit, the probabilities' terms take the place of the scores they came from in tensor memory
// (A operand). Two row tiles of 128 share a CTA and its key / value ring; each has two
// threads a row, one for each 64-token block of a tile, and runs its own chain (scores, softmax, value
// sums), so that one tile's tensor work hides behind the other's exponentials. O stays in registers (64
// coordinates a thread), where the running maximum's corrections and the blocks' value scales multiply it. MMAs and
// copies are issued by warps of their own: an issue waits while the tensor cores' queue is full.
//
// Bound by issue, then the tensor cores: per 128 x 128 tile two products of TERMS passes (540 clocks a
// product and two passes) and about 7 instructions an element. Measured: the last 2048 of 8192 tokens, 32 query and 8 KV heads: 292 us in
// bf16 (824 TFLOP/s of the formula's products, 0.43 of a plain bf16 matrix product), 348 us
// in fp16; ALU 57 % and tensor cores 37 % busy, the rest the wait of each for the other. Capped 492 us (three
// exponentials or reciprocals an element), caps above 128, whose small scores go through a series, 589 us; biased 426 us. Both store their scores and
// read them again, without loads ahead and without turns. TERMS = 2 for bf16 (8 significant bits of
// q and p, down to 2^-18 of the largest of either), 3 for fp16 (11). A term costs half an instruction to make: the probabilities go
// through fp16 pairs, in which the differences to the terms are exact.
//
// Two blocks of a tile share one value sum, the smaller scale folded into its probabilities; where the scales are more than
// 2^4 apart that would cost precision, and the blocks' sums are formed one after the other. The terms of a probability end at a fixed
// step (2^-17 of 2^8 for two of them), so it is relative to the row's largest of its own sum, not to the running maximum: the smaller ones of a
// tile after a heavy key keep their bits, and what a tile's terms drop is below 2^-8 of its own mass. The way to the running maximum is a factor of the
// whole sum, formed while the tensor cores work.
// Work split: as in the kernel for few rows, equal slices of the (sequence, unit of 256 rows, head, tile) space, a unit's start counted
// as tiles, and cut units joined afterwards; small kernels find each unit's tiles and the slices first. Up to 128 rows over many tiles
// are units of one row tile: the two row tiles of a CTA then work on slices of their own (APART).

#pragma once

#include "tq_q8_rows.cuh"

namespace tq {
namespace {

constexpr int kTile = 128;
// Rows of a unit: two row tiles, or, APART, one: then the two row tiles of a CTA hold units of their own, with half of the ring each.
constexpr int unit_rows(bool apart) { return apart ? 128 : 256; }
constexpr int kSoft = 512;              // softmax threads; then a warpgroup of controllers:
constexpr int kThreads = kSoft + 128;   // warps 16 and 17 issue a row tile's MMAs each, warp 18 the copies, warp 19 nothing (APART: the second row tile's)
constexpr int kRegsSoft = 112, kRegsControl = 32;  // 512 * 112 + 128 * 32 = 640 * 96, what the block is launched with
constexpr int kStage = 2 * kTile * kD;
constexpr int kQTerm = 128 * kD;       // one term of a row tile's queries
constexpr int part_of(int unit) { return unit * (kD + 2); }  // a partial record: O as 32 columns of 4 coordinates [column][row][4], then m and l [row]
constexpr float kFold = 0.0625f;       // blocks' value scales within 2^4 share a sum
constexpr float kLowest = -3e38f;      // in place of a maximum of -inf: an unseen score stays -inf beside it, its factor is 0

constexpr int stages_of(int terms, bool apart) { return terms == 2 || apart ? 4 : 3; }

struct Entry {
  int lo, hi;          // first visible slot, one past the last
  int maxbeg, minend;  // slots in [maxbeg, minend) are seen by every row that is written
};

struct Cut {
  int b, pair, h, parts;
};

struct Plan {
  int *pre;       // [entries + 1] tiles (of one head) before each entry
  int *starts;    // [entries + 1] entries with tiles before each
  long long *cut; // [slices + 1] where the slices of the tiles begin (APART: two a CTA, else one)
  Entry *entry;   // [entries]
  Cut *cuts;      // [slices]
  float *parts;   // [slices][2] records
  int entries, pairs, unit;  // pairs: units of a sequence (and head); unit: their rows
};

// An entry (sequence, unit of rows): a warp.
template <int KIND>
__device__ __forceinline__ void make_entry(const Q8AttnArgs &a, const Plan &p, int e, int lane) {
  const int b = e / p.pairs, G = a.group;
  int len, m, r0, end, list;
  unit_span<KIND>(a, e % p.pairs, p.unit, &r0, &end, &list);
  seq_sizes<KIND>(a, b, &len, &m, lane == 0);
  const int i0 = r0 / G, i1 = min(m - 1, (min(end, r0 + p.unit) - 1) / G);
  int lo = 0x7fffffff, hi = 0, maxbeg = 0, minend = 0x7fffffff;
  for (int i = i0 + lane; i <= i1; i += 32) {
    const int2 r = row_range<KIND>(a, b, i, len, m);
    if (r.y > r.x) lo = min(lo, r.x), hi = max(hi, r.y);
    maxbeg = max(maxbeg, r.x);
    minend = min(minend, r.y);  // 0 for a row that sees nothing
  }
  lo = __reduce_min_sync(kFull, lo);
  hi = __reduce_max_sync(kFull, hi);
  maxbeg = __reduce_max_sync(kFull, maxbeg);
  minend = __reduce_min_sync(kFull, minend);
  if (lane == 0) {
    if (hi == 0) lo = 0;
    p.entry[e] = Entry{lo, hi, maxbeg, minend};
    // rows that see nothing keep one tile, so that their zeros are written
    p.pre[e + 1] = i0 < m ? max(1, unit_tiles<KIND>(a, b, lo, hi)) : 0;
  }
}

template <int KIND>
__global__ void __launch_bounds__(256) q8_entries_kernel(const __grid_constant__ Q8AttnArgs a, Plan p) {
  const int e = blockIdx.x * 8 + (threadIdx.x >> 5);
  if constexpr (KIND != kWhole) pdl_trigger();  // each of the call's launches waits for all of the one before
  pdl_wait();
  if (e < p.entries) make_entry<KIND>(a, p, e, threadIdx.x & 31);
}

// What a unit's start (its queries, the first tile's chain alone) costs, in tiles: ragged documents of 1 to 11 tiles a unit take 127 us in
// slices that count tiles alone, 90 us with 2, 91 with 3, 91 with 5; units of up to 64 tiles, 96 tiles a CTA: 333, 304, 304, 310.
constexpr int kStart = 3;

// Prefix sums of the entries' tiles and the slices, one CTA. Slices are equal in tiles and starts, and none is empty (an
// interval of kStart + 1 holds a tile); with fewer than two tiles a CTA, in tiles alone, so that as many CTAs as possible work.
// Up to kPlanned entries are made here as well.
constexpr int kPlanned = 128;
constexpr int kMostSlices = 1023;
constexpr int kJoinTiles = 4;  // what the join costs, in tiles
template <int KIND>
__global__ void __launch_bounds__(1024) q8_prefix_kernel(const __grid_constant__ Q8AttnArgs a, Plan p, int ctas) {
  const int heads = a.heads_kv;
  __shared__ int warp_tiles[32], warp_starts[32];
  __shared__ unsigned long long largest;
  __shared__ long long rounded[KIND == kWhole ? 1 : kMostSlices + 1];
  __shared__ int pre_near[kPlanned + 1], starts_near[kPlanned + 1];  // of few entries
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int base = 0, base_starts = 0;
  if constexpr (KIND != kWhole) pdl_trigger();
  pdl_wait();
  if (KIND != kWhole && p.entries <= kPlanned) {
    for (int e = warp; e < p.entries; e += 32) make_entry<KIND>(a, p, e, lane);
    __syncthreads();
  }
  if (tid == 0) p.pre[0] = 0, p.starts[0] = 0, pre_near[0] = 0, starts_near[0] = 0;
  for (int e0 = 0; e0 < p.entries; e0 += 1024) {
    const int e = e0 + tid;
    int x = e < p.entries ? p.pre[e + 1] : 0, y = x > 0 ? 1 : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x1 = __shfl_up_sync(kFull, x, o), y1 = __shfl_up_sync(kFull, y, o);
      if (lane >= o) x += x1, y += y1;
    }
    if (lane == 31) warp_tiles[warp] = x, warp_starts[warp] = y;
    __syncthreads();
    const int wx = warp_tiles[lane], wy = warp_starts[lane];
    const int before = base + __reduce_add_sync(kFull, lane < warp ? wx : 0), all = base + __reduce_add_sync(kFull, wx);
    const int sbefore = base_starts + __reduce_add_sync(kFull, lane < warp ? wy : 0), sall = base_starts + __reduce_add_sync(kFull, wy);
    if (e < p.entries) p.pre[e + 1] = before + x, p.starts[e + 1] = sbefore + y;
    if (KIND != kWhole && e < p.entries && p.entries <= kPlanned) pre_near[e + 1] = before + x, starts_near[e + 1] = sbefore + y;
    base = all, base_starts = sall;
    __syncthreads();
  }
  const long long tiles = (long long)base * heads;
  // Few units of many slices each: every slice begins with a start of its own then (counted, it would leave the first slice of a unit 3 tiles short).
  const bool few = KIND != kWhole && 4LL * base_starts * heads <= ctas;
  const int start = tiles >= 2LL * ctas && !few ? kStart : 0;
  const bool near = KIND != kWhole && p.entries <= kPlanned;
  const int *const pre = near ? pre_near : p.pre, *const starts = near ? starts_near : p.starts;
  const long long total = tiles + (long long)start * base_starts * heads;
  const long long slices = min((long long)ctas, total / (start + 1));
  // where slice k begins: its weight, and the unit there (its weight, its first tile's number)
  auto begin = [&](int k, long long *unit, int *each, long long *tile) {
    const long long c = quotient(total * k, slices);
    int lo = 0, hi = p.entries - 1;
    while (lo < hi) {  // the last entry that begins at or before c
      const int mid = (lo + hi + 1) >> 1;
      if (((long long)pre[mid] + (long long)start * starts[mid]) * heads <= c) lo = mid;
      else hi = mid - 1;
    }
    const int cnt = pre[lo + 1] - pre[lo];
    *each = cnt + start;
    const long long from = ((long long)pre[lo] + (long long)start * starts[lo]) * heads, h = quotient(c - from, *each);
    *unit = from + h * *each, *tile = (long long)pre[lo] * heads + h * cnt;
    return c;
  };
  // Slices of whole units, each slice's begin moved to the nearer end of the unit that it lies in, save the cut units' further starts
  // and the join: taken where the largest costs no more than an even slice with these (16 tiles a unit, 256 units: 130 us cut, 119 whole).
  bool whole = false;
  if (KIND != kWhole && slices > 0 && slices <= kMostSlices && !few) {
    for (int k = tid; k <= slices; k += 1024) {
      long long unit = total, tile, c = total;
      int each = 1;
      if (k < slices) c = begin(k, &unit, &each, &tile);
      rounded[k] = 2 * (c - unit) >= each ? unit + each : unit;
    }
    if (tid == 0) largest = 0;
    __syncthreads();
    for (int k = tid; k < slices; k += 1024) atomicMax(&largest, (unsigned long long)(rounded[k + 1] - rounded[k]));
    __syncthreads();
    whole = (long long)largest <= quotient(total, slices) + kStart + kJoinTiles;
  }
  for (int k = tid; k <= ctas; k += 1024) {
    long long g = tiles;
    if (k < slices) {
      long long unit, tile;
      int each;
      const long long c = begin(k, &unit, &each, &tile);
      g = tile + max(0, (int)(c - unit) - start);
      if (whole) g = 2 * (c - unit) >= each ? tile + each - start : tile;
    }
    p.cut[k] = g;
  }
}

struct Shared {
  uint64_t full[4], empty[4];
  uint64_t bar_q[2], bar_s[2], bar_p[2], bar_o[2];  // of a row tile: queries, scores, probabilities, value sums are there
  float4 info[4];             // of a stage: key scales of the tile's two blocks, value scales (negative: not there)
  int2 at[4];                 // (BLOCKS) their first slots
  float top[2][2][128];       // [row tile][half]: row maxima, then sums
  uint32_t tmem;
  int bad;
};

// The unit of work at tile g of the slice that ends at g1: entry e, KV head h, from tile t0 of its cnt on, up to g = end.
struct Unit {
  int e, h, b, pair, t0, cnt;
  long long end;
};
__device__ __forceinline__ Unit unit_at(const Plan &p, int heads, long long g, long long g1) {
  Unit u;
  int lo = 0, hi = p.entries - 1;
  while (lo < hi) {  // the last entry that begins at or before g
    const int mid = (lo + hi + 1) >> 1;
    if ((long long)p.pre[mid] * heads <= g) lo = mid;
    else hi = mid - 1;
  }
  u.e = lo, u.cnt = p.pre[lo + 1] - p.pre[lo];
  const long long in = g - (long long)p.pre[lo] * heads;
  u.h = (int)quotient(in, u.cnt), u.t0 = (int)(in - (long long)u.h * u.cnt);
  u.b = lo / p.pairs, u.pair = lo % p.pairs;
  u.end = min(g1, g - u.t0 + u.cnt);
  return u;
}

// A tile's two blocks have value scales too far apart to be folded into one sum.
__device__ __forceinline__ bool scales_apart(const float4 &f) {
  return f.z >= 0.f && f.w >= 0.f && fminf(f.z, f.w) < fmaxf(f.z, f.w) * kFold;
}

__device__ __forceinline__ void bar_rt(int rt) { asm volatile("bar.sync %0, 256;" ::"r"(1 + rt) : "memory"); }
// The row tiles take turns at the exponentials: turn_take waits for the other's turn_pass.
__device__ __forceinline__ void turn_take(int rt) { asm volatile("bar.sync %0, 512;" ::"r"(3 + rt) : "memory"); }
__device__ __forceinline__ void turn_pass(int rt) { asm volatile("bar.arrive %0, 512;" ::"r"(4 - rt) : "memory"); }

// D (TMEM) (+)= A (TMEM, four 8-bit K-elements per column) x B (shared); executed by one lane.
__device__ __forceinline__ void tc_mma_f8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st_x4(uint32_t taddr, const uint32_t (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// two e4m3 (e5m2) bytes of an fp16 pair, and back
__device__ __forceinline__ uint32_t h2_e4m3(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t h2_e5m2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_h2(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
  return h;
}
__device__ __forceinline__ uint32_t h2_sub(uint32_t x, uint32_t y) {
  const __half2 r = __hsub2(*reinterpret_cast<__half2 *>(&x), *reinterpret_cast<__half2 *>(&y));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// Coordinates d .. d + N - 1 of a row: o = sum 2^(t - mx + 8) v, l the same of 1. Written to where the kind's results go, joined with the
// prefix's part where there is one.
template <int KIND, int N>
__device__ __forceinline__ void finish_part(const Q8AttnArgs &a, int b, int hq, int i, int d, float (&o)[N], float mx, float l, const Prior<N> &prior) {
  if constexpr (KIND == kPrefix) {
    float *row = a.prior + ((long long)hq * a.n_q + i) * kPriorRow;
#pragma unroll
    for (int q = 0; q < N; q += 4) *reinterpret_cast<float4 *>(row + d + q) = make_float4(o[q], o[q + 1], o[q + 2], o[q + 3]);
    if (d == 0) *reinterpret_cast<float4 *>(row + kD) = make_float4(mx - 8.f, l, l, 0.f);
    return;
  }
  float lr = l, m = mx;
  if constexpr (KIND == kOwn) {
    const Joined p = joined(prior.was, mx - 8.f);
#pragma unroll
    for (int q = 0; q < N; ++q) o[q] = fmaf(prior.x[q], p.by, o[q] * p.own);
    lr = fmaf(prior.lr, p.by, l * p.own);
    l = fmaf(prior.l, p.by, l * p.own);
    m = p.m + 8.f;
  }
  const float inv = lr == 0.f ? 0.f : 1.f / lr;
  const long long off = b * a.os.b + hq * a.os.h + i * a.os.t + d;
  constexpr int V = N < 8 ? N : 8;
#pragma unroll
  for (int q = 0; q < N; q += V) {
    float y[V];
#pragma unroll
    for (int k = 0; k < V; ++k) y[k] = o[q + k] * inv;
    if (a.out_dtype == TQ_BF16) store_vec<__nv_bfloat16, V>(static_cast<__nv_bfloat16 *>(a.out) + off + q, y);
    else store_vec<__half, V>(static_cast<__half *>(a.out) + off + q, y);
  }
  if (a.lse && d == 0) a.lse[((long long)b * a.heads_q + hq) * a.n_q + i] = (m + log2f(l) - 8.f) * kLn2;
}

template <int TERMS, int EXTRA, bool APART, int KIND>
__global__ void __launch_bounds__(kThreads, 1)
q8_prompt_kernel(const __grid_constant__ Q8AttnArgs a, const __grid_constant__ Plan p) {
  constexpr int kStages = stages_of(TERMS, APART), kUnit = unit_rows(APART);
  constexpr bool BLOCKS = KIND == kListed || KIND == kBoth;  // a tile's blocks do not follow each other
  constexpr bool kTurns = !EXTRA && !APART;  // capped or biased scores run without turns (2048 of 8192 tokens, when they took 653 us: 713 with them)
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ Shared sm;
  uint8_t *ring = dyn, *qbuf = dyn + kStages * kStage;  // [row tile][term][128 x 128]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&sm.full[s], 1), mbar_init(&sm.empty[s], APART ? 1 : 2);
    for (int r = 0; r < 2; ++r) {
      mbar_init(&sm.bar_s[r], 1), mbar_init(&sm.bar_o[r], 1);
      mbar_init(&sm.bar_q[r], 8), mbar_init(&sm.bar_p[r], 8);  // a row tile's warps
    }
    mbar_fence_init();
    sm.bad = 0;
  }
  if (warp == kSoft / 32 + 2) {
    tmem_alloc(smem_u32(&sm.tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sm.tmem;
  if constexpr (KIND != kWhole) pdl_trigger();
  pdl_wait();

  // the row tile that a warp belongs to (0 for the copies of both), its slice, and the ring's stage and its phase for the slice's tile `it`
  const int rt = warp < kSoft / 32 ? warp >> 3 : APART || warp < kSoft / 32 + 2 ? warp & 1 : 0;
  const int slice = APART ? rt * gridDim.x + blockIdx.x : blockIdx.x, slices = APART ? 2 * gridDim.x : gridDim.x;
  auto stage = [&](int it) { return APART ? 2 * rt + (it & 1) : it % kStages; };
  auto turn = [&](int it) { return (uint32_t)(APART ? it >> 1 : it / kStages) & 1; };
  const long long g0 = p.cut[slice], g1 = p.cut[slice + 1];
  const bool idle = g0 >= g1;
  auto wait = [&](uint64_t *bar, uint32_t parity) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i)
      if (mbar_try_wait(bar, parity)) return;
    if (*(volatile int *)&sm.bad) return;
    if (!mbar_wait_bounded(bar, parity, a.error)) *(volatile int *)&sm.bad = 1;
  };

  if (warp >= kSoft / 32) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (warp == kSoft / 32 + 2 || (APART && warp == kSoft / 32 + 3)) {
      // ================================ copies: a lane finds the sources of one of a unit's next 32 tiles
      int it = 0;
      for (long long g = g0; g < g1;) {
        const Unit u = unit_at(p, a.heads_kv, g, g1);
        const Entry en = p.entry[u.e];
        const long long bh = (long long)u.b * a.heads_kv + u.h;
        int r0, rend, list;
        unit_span<KIND>(a, u.pair, kUnit, &r0, &rend, &list);
        const int prefix = KIND == kBoth ? prefix_of(a, u.b) : 0;
        const BothTiles both = both_tiles(prefix, en.lo, en.hi);
        for (int k0 = 0; g + k0 < u.end; k0 += 32) {
          const int todo = (int)min(32ll, u.end - g - k0);
          long long src[2] = {-1, -1};
          float4 f = make_float4(-1.f, -1.f, -1.f, -1.f);
          int bytes[2] = {0, 0}, at[2] = {0, 0};
          if (lane < todo) {
            const int j = u.t0 + k0 + lane;
            int blk[2];
            if constexpr (KIND == kBoth) {  // (src: addresses)
              const bool pre = j < both.prefix;
              const Q8Cache &c = pre ? a.pc : a.c;
              blk[0] = 2 * (pre ? both.first + j : both.own + j - both.prefix), blk[1] = blk[0] + 1;
              f = tile_sources(a, c, pre ? u.h : bh, blk, pre ? 0 : prefix, en.lo, pre ? min(prefix, en.hi) : en.hi, src, bytes, at);
#pragma unroll
              for (int k = 0; k < 2; ++k)
                if (src[k] >= 0) src[k] = (long long)(c.records + src[k] * kQ8BlockBytes);
            } else {
              if constexpr (KIND == kListed) list_entries(a, bh, list, 2 * j, blk);
              else blk[0] = 2 * (en.lo / kTile + j), blk[1] = blk[0] + 1;
              f = tile_sources(a, a.c, bh, blk, 0, en.lo, en.hi, src, bytes, at);
            }
          }
          for (int k = 0; k < todo; ++k, ++it) {
            const int s = stage(it);
            const long long s0 = __shfl_sync(kFull, src[0], k), s1 = __shfl_sync(kFull, src[1], k);
            const int n0 = __shfl_sync(kFull, bytes[0], k), n1 = __shfl_sync(kFull, bytes[1], k);
            float4 x;
            x.x = __shfl_sync(kFull, f.x, k), x.y = __shfl_sync(kFull, f.y, k);
            x.z = __shfl_sync(kFull, f.z, k), x.w = __shfl_sync(kFull, f.w, k);
            int2 slots = make_int2(0, 0);
            if constexpr (BLOCKS) slots.x = __shfl_sync(kFull, at[0], k), slots.y = __shfl_sync(kFull, at[1], k);
            if (lane == 0) {
              wait(&sm.empty[s], turn(it) ^ 1);
              if (!*(volatile int *)&sm.bad) {
                sm.info[s] = x;
                if constexpr (BLOCKS) sm.at[s] = slots;
                uint8_t *dst = ring + s * kStage;
                mbar_arrive_expect_tx(&sm.full[s], 2 * (n0 + n1));
                if (n0) {
                  const uint8_t *q = KIND == kBoth ? (const uint8_t *)s0 : a.c.records + s0 * kQ8BlockBytes;
                  tma_load_1d(dst, q, n0, &sm.full[s]);
                  tma_load_1d(dst + kTile * kD, q + kQ8Plane, n0, &sm.full[s]);
                }
                if (n1) {
                  const uint8_t *q = KIND == kBoth ? (const uint8_t *)s1 : a.c.records + s1 * kQ8BlockBytes;
                  tma_load_1d(dst + kQ8Plane, q, n1, &sm.full[s]);
                  tma_load_1d(dst + kTile * kD + kQ8Plane, q + kQ8Plane, n1, &sm.full[s]);
                }
              }
            }
            __syncwarp();
          }
        }
        g = u.end;
      }
      // every copy lands before the CTA's shared memory goes: the last fill of each stage
      if (lane == 0)
        for (int k = max(0, it - (APART ? 2 : kStages)); k < it; ++k)
          mbar_wait_bounded(&sm.full[stage(k)], turn(k), nullptr, kWaitBudgetNs / 8);
      __syncwarp();
    } else if (warp < kSoft / 32 + 2) {
      // ================================ a row tile's MMAs
      {
        const bool issue = elect_lane();
        const uint32_t t_s = warp_uniform(tmem + rt * 256), t_o = t_s + 128, q = warp_uniform(smem_u32(qbuf + rt * TERMS * kQTerm));
        uint32_t units = 0, probs = 0;
        int it = 0;
        for (long long g = g0; g < g1; ++units) {
          const Unit u = unit_at(p, a.heads_kv, g, g1);
          const int first = p.entry[u.e].lo / kTile + u.t0, hi = p.entry[u.e].hi, todo = (int)(u.end - g);
          const int prefix = KIND == kBoth ? prefix_of(a, u.b) : 0;
          wait(&sm.bar_q[rt], units & 1);
          for (int j = 0; j <= todo; ++j) {
            // the value sums of tile j - 1, then the scores of tile j over its probabilities: in this order, as issued
            if (j > 0) {
              const int s = stage(it + j - 1);
              const float4 f = sm.info[s];
              // the tokens up to the end of either block's (of those that are there)
              int n0 = min(kTile, max(0, hi - (first + j - 1) * kTile)), n1 = n0;
              if constexpr (BLOCKS) {
                const int2 at = sm.at[s];
                n0 = min(kQ8Block, (at.x < prefix ? min(prefix, hi) : hi) - at.x);
                n1 = kQ8Block + min(kQ8Block, (at.y < prefix ? min(prefix, hi) : hi) - at.y);
              }
              const bool apart = scales_apart(f), whole = n0 >= kQ8Block && n1 == kTile && f.z >= 0.f && f.w >= 0.f && !apart;
              const uint32_t vt = warp_uniform(smem_u32(ring + s * kStage) + kTile * kD);
              for (int part = 0; part <= (int)apart; ++part) {  // the two blocks at once, or one after the other
                wait(&sm.bar_p[rt], probs & 1);
                ++probs;
                tc_fence_after_sync();
                if (whole) {  // nothing to decide between the MMAs
#pragma unroll
                  for (int t = 0; t < TERMS; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                      if (issue)
                        tc_mma_f8_ts(t_o, t_s + 32 * k + 8 * t, tc_sdesc_kmajor(vt + 4096 * k, 1024, 128),
                                     tc_idesc_f8(128, 128, t == 2, 0, 0, 1), t > 0 || k > 0);
                } else {
                  bool more = false;
#pragma unroll
                  for (int t = 0; t < TERMS; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                      if (k * 32 >= (k < 2 ? n0 : n1) || (k < 2 ? f.z : f.w) < 0.f || (apart && k / 2 != part)) continue;
                      if (issue)
                        tc_mma_f8_ts(t_o, t_s + 32 * k + 8 * t, tc_sdesc_kmajor(vt + 4096 * k, 1024, 128),
                                     tc_idesc_f8(128, 128, t == 2, 0, 0, 1), more);
                      more = true;
                    }
                }
                if (issue && part == (int)apart) tc_commit(smem_u32(&sm.empty[s]));
                if (issue) tc_commit(smem_u32(&sm.bar_o[rt]));
                __syncwarp();
              }
            }
            if (j < todo) {
              const int s = stage(it + j);
              wait(&sm.full[s], turn(it + j));
              tc_fence_after_sync();
              const uint32_t kt = warp_uniform(smem_u32(ring + s * kStage));
#pragma unroll
              for (int t = 0; t < TERMS; ++t)
#pragma unroll
                for (int k = 0; k < kD / 32; ++k)
                  if (issue) tc_mma_f8(t_s, tc_sdesc_kmajor(q + t * kQTerm + 256 * k, 128, 1024), tc_sdesc_kmajor(kt + 256 * k, 128, 1024),
                            tc_idesc_f8(128, 128, t == 2, 0, 0, 0), t > 0 || k > 0);
              if (issue) tc_commit(smem_u32(&sm.bar_s[rt]));
              __syncwarp();
            }
          }
          it += todo;
          g = u.end;
        }
      }
      __syncwarp();
    }
  } else {
    // ================================ softmax and output: two threads a row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    const int half = (tid >> 7) & 1, lrow = tid & 127, in_unit = (APART ? 0 : rt * 128) + lrow;
    const uint32_t t_s = tmem + rt * 256 + ((uint32_t)(32 * (warp & 3)) << 16) + 64 * half, t_o = t_s + 128;
    const ScoreCap sc = EXTRA ? score_cap(a.scale, a.softcap) : ScoreCap{};
    int it = 0;  // tiles done: stages and phases count on
    if (kTurns && rt == 1 && g0 < g1) turn_pass(rt);
    uint32_t sums = 0;
    long long g = g0;
    while (g < g1) {
      const Unit u = unit_at(p, a.heads_kv, g, g1);
      const int first = p.entry[u.e].lo / kTile + u.t0, hi = p.entry[u.e].hi, maxbeg = p.entry[u.e].maxbeg,
                minend = p.entry[u.e].minend;
      const long long bh = (long long)u.b * a.heads_kv + u.h;
      int len, m;
      seq_sizes<KIND>(a, u.b, &len, &m, false);
      const int G = a.group;
      const int prefix = KIND == kBoth ? prefix_of(a, u.b) : 0;
      int unit0, unit1, list;
      unit_span<KIND>(a, u.pair, kUnit, &unit0, &unit1, &list);

      // ---- queries: a warp prepares 16 rows of its row tile (whose score MMAs of the unit before are done)
      bar_rt(rt);
#pragma unroll 1
      for (int k0 = 0; k0 < 16; k0 += 8) {
        uint2 raw[8];
        const int first_row = unit0 + (APART ? 0 : rt * 128) + (warp & 7) * 16 + k0;
        load_rows<KIND>(a, u.b, u.h, m, first_row, lane, raw);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = (warp & 7) * 16 + k0 + k, row = first_row + k;
          float x[4];
          row_floats(a, raw[k], row < unit1 && row / G < m, x);
          uint32_t w[3];
          const int ex = row_terms(x, w);
#pragma unroll
          for (int t = 0; t < TERMS; ++t)
            *reinterpret_cast<uint32_t *>(qbuf + (rt * TERMS + t) * kQTerm + q8_off(r, 4 * lane)) = w[t];
          if (lane == 0) sm.top[rt][0][r] = pow2i(ex);
        }
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.bar_q[rt]);
      bar_rt(rt);
      const float qs = sm.top[rt][0][lrow];
      const int row = unit0 + in_unit, qi = row / G, hq = u.h * G + row % G;
      const bool live = row < unit1 && qi < m;
      const int2 rg = live ? row_range<KIND>(a, u.b, qi, len, m) : make_int2(0, 0);
      const float slope = EXTRA && live && a.slopes ? latest(a.slopes + hq) * kLog2e : 0.f;
      const int qp = !EXTRA || !live ? 0 : a.qpos ? latest(a.qpos + (long long)u.b * a.n_q + qi) : query_slot<KIND>(a, qi, len, m);
      bar_rt(rt);

      float o[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) o[i] = 0.f;
      float mx = -INFINITY, l = 0.f;
      const int todo = (int)(u.end - g);
      for (int j = 0; j < todo; ++j) {
        const int s = stage(it + j);
        int tok0 = (first + j) * kTile, n = min(kTile, max(0, hi - tok0));  // (BLOCKS: of this half's block, below)
        wait(&sm.full[s], turn(it + j));
        const float4 f = sm.info[s];
        const float ks = half ? f.y : f.x;
        bool masked = !(maxbeg <= tok0 && minend >= tok0 + kTile) || f.x < 0.f || f.y < 0.f;
        if constexpr (BLOCKS) {
          const int at = half ? sm.at[s].y : sm.at[s].x;  // of a prefix's block: its last tokens may not be the sequence's
          const int there = ks < 0.f ? 0 : min(kQ8Block, (at < prefix ? min(prefix, hi) : hi) - at);
          tok0 = at - 64 * half, n = 64 * half + there;
          masked = there < kQ8Block || !(maxbeg <= at && minend >= at + kQ8Block);
        }
        int from = 0, to = 64;  // the tokens of this half that the row sees
        if (masked) {
          from = min(max(rg.x - tok0 - 64 * half, 0), 64), to = min(max(rg.y - tok0 - 64 * half, 0), 64);
          if (ks < 0.f) to = 0;
          if constexpr (KIND == kBoth) to = min(to, n - 64 * half);
        }
        // never 0, so that an unseen score of -inf stays -inf (products so small make no difference)
        const float c = EXTRA ? qs * fmaxf(ks, 0.f) * sc.in : fmaxf(qs * fmaxf(ks, 0.f) * (a.scale * kLog2e), 1e-30f);
        // the raw product (the scaling is in c); MASK: unseen ones are -inf
        auto score = [&](float x, int i, auto mask) {
          if constexpr (decltype(mask)::value) x = i >= from && i < to ? x : -INFINITY;
          return x;
        };
        // where keys are at their slots, the distance of slot i of this half is |far - i|
        const int slot0 = tok0 + 64 * half;
        const float far = EXTRA && a.slopes && !a.kpos ? (float)((long long)qp - slot0) : 0.f;
        wait(&sm.bar_s[rt], (it + j) & 1);
        __syncwarp();  // tensor memory is read by whole warps
        tc_fence_after_sync();
        if constexpr (kTurns) turn_take(rt);
        // ---- the row's maximum over this half
        float top = -INFINITY;
        auto maximum = [&](auto mask) {
          float top1 = -INFINITY;
          if constexpr (EXTRA) {  // scaled to log2, capped, biased and masked once, here
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[16];
              tmem_ld_start(t_s + 16 * q, w);  // (the next 16 ahead, as below, would spill: 633 against 528 us capped)
              tmem_ld_done(w);
              float x[16];
              if (sc.cap == 0.f) {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(w[i]) * c;
              } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = capped_log2<EXTRA == kLongCaps>(__uint_as_float(w[i]), c, sc.cap);
              }
              if (a.kpos && a.slopes) {
                const int32_t *kp = a.kpos + bh * a.c.capacity + slot0 + 16 * q;
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = fmaf(-slope, (float)__sad(qp, slot0 + 16 * q + i < hi ? latest(kp + i) : 0, 0u), x[i]);
              } else if (a.slopes) {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = fmaf(-slope, fabsf(far - (float)(16 * q + i)), x[i]);
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                x[i] = score(x[i], 16 * q + i, mask);
                top = fmaxf(top, x[i]);
              }
              tmem_st_x16(t_s + 16 * q, x);
            }
            tmem_st_wait();
          } else {
            uint32_t w[2][16];
            tmem_ld_start(t_s, w[0]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              tmem_ld_done(w[q & 1]);
              if (q < 3) tmem_ld_start(t_s + 16 * (q + 1), w[(q + 1) & 1]);
              float x[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) x[i] = score(__uint_as_float(w[q & 1][i]), 16 * q + i, mask);
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                top = fmaxf(top, fmaxf(x[i], x[i + 1]));
                top1 = fmaxf(top1, fmaxf(x[i + 2], x[i + 3]));
              }
            }
            top = fmaxf(top, top1);
          }
        };
        if (masked) maximum(std::true_type{});
        else maximum(std::false_type{});
        if constexpr (!EXTRA) top = top == -INFINITY ? top : top * c;
        sm.top[rt][half][lrow] = top;
        bar_rt(rt);
        const float other = sm.top[rt][half ^ 1][lrow];
        // ---- the two blocks' value scales, in log2: the smaller is folded into its block's probabilities (`fold` for this block, `fold1`
        // for the other), or each block has a sum of its own. Probabilities are relative to the row's largest (folded) one of their sum
        const bool apart = scales_apart(f);
        float fold = 0.f, fold1 = apart ? -INFINITY : 0.f;
        if (f.z != f.w && f.z >= 0.f && f.w >= 0.f && !apart) {
          const float d = (float)(log2i(half ? f.w : f.z) - log2i(half ? f.z : f.w));
          fold = fminf(d, 0.f), fold1 = fminf(-d, 0.f);
        }
        // This block's scale (the other's where it is not there) is the sum's, beside the way from this block's reference: folded, the two have
        // the same product in both. Kept in place of both scales over the exponentials: 292 us, 301 with them.
        const float own = half ? (f.w < 0.f ? f.z : f.w) : f.z < 0.f ? f.w : f.z;
        const float shift = 8.f + fold - fmaxf(fmaxf(top + fold, other + fold1), kLowest);
        // ---- probabilities times 2^8, their terms over the scores they come from, their sum
        float2 sum = make_float2(0.f, 0.f);
        auto probabilities = [&](auto mask) {
          uint32_t held[4], v[2][16];
          tmem_ld_start(t_s, v[0]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t(&x)[16] = v[q & 1];
            tmem_ld_done(x);
            if (q < 3) tmem_ld_start(t_s + 16 * (q + 1), v[(q + 1) & 1]);
            uint32_t w[TERMS][4];
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              uint32_t t[TERMS][2];
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const int k = i + 2 * u;
                float y0 = __uint_as_float(x[k]), y1 = __uint_as_float(x[k + 1]);
                if constexpr (!EXTRA) y0 = score(y0, 16 * q + k, mask), y1 = score(y1, 16 * q + k + 1, mask);
                const float p0 = ex2_approx(EXTRA ? y0 + shift : fmaf(y0, c, shift));
                const float p1 = ex2_approx(EXTRA ? y1 + shift : fmaf(y1, c, shift));
                sum.x += p0, sum.y += p1;
                const __half2 hp = __floats2half2_rn(p0, p1);
                uint32_t left = *reinterpret_cast<const uint32_t *>(&hp);
                t[0][u] = h2_e4m3(left);
                left = h2_sub(left, e4m3_h2(t[0][u]));
                t[1][u] = h2_e4m3(left);
                if constexpr (TERMS == 3) {
                  left = h2_sub(left, e4m3_h2(t[1][u]));
                  t[2][u] = h2_e5m2(left);
                }
              }
#pragma unroll
              for (int k = 0; k < TERMS; ++k) w[k][i / 4] = __byte_perm(t[k][0], t[k][1], 0x5410);
            }
            // a K-step's 32 tokens have 32 score columns; its term k goes to columns 8 k .. 8 k + 7 of them, where
            // the scores were read by now, but for the third term's first half: that waits for the next 16
            const uint32_t at = t_s + 32 * (q >> 1) + 4 * (q & 1);
            tmem_st_x4(at, w[0]);
            tmem_st_x4(at + 8, w[1]);
            if constexpr (TERMS == 3) {
              if (q & 1) {
                tmem_st_x4(at + 12, held);
                tmem_st_x4(at + 16, w[2]);
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) held[i] = w[2][i];
              }
            }
          }
        };
        if (masked) probabilities(std::true_type{});
        else probabilities(std::false_type{});
        // value rows past the copied tokens, up to a whole K-step, hold what the cache holds there
        if (n & 31) {
          const int t = n + (BLOCKS ? tid & 127 : tid & 255);
          if (t < ((n + 31) & ~31)) {
            uint8_t *vt = ring + s * kStage + kTile * kD;
#pragma unroll
            for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4 *>(vt + q8_off(t, 16 * k)) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_shared();
        }
        if constexpr (kTurns) {
          if (rt == 0 || u.end < g1 || j + 1 < todo) turn_pass(rt);
        }
        tmem_st_wait();
        // O = O corr + vs by D
        auto add = [&](float vs, float by, float corr) {
          if (!__all_sync(kFull, corr == 1.f)) {
#pragma unroll
            for (int i = 0; i < 64; ++i) o[i] *= corr;
          }
          if (!__any_sync(kFull, vs >= 0.f)) return;  // (a vote, which the compiler knows to be the warp's: 305 us where a comparison took 311)
          vs *= by;
          uint32_t d[2][16];
          tmem_ld_start(t_o, d[0]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            tmem_ld_done(d[q & 1]);
            if (q < 3) tmem_ld_start(t_o + 16 * (q + 1), d[(q + 1) & 1]);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[16 * q + i] = fmaf(__uint_as_float(d[q & 1][i]), vs, o[16 * q + i]);
          }
        };
        float corr = 1.f, by = 1.f, use = 0.f;
        for (int blk = 0; blk <= (int)apart; ++blk) {
          const float its = apart ? half ? sm.info[s].z : sm.info[s].w : 0.f;
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.bar_p[rt]);
          if (blk == 0) {  // while the sum is formed: from the probabilities' reference to the running maximum
            const float run = fmaxf(fmaxf(top, other), mx);
            use = fmaxf(run, kLowest);
            corr = ex2_approx(mx - use), by = ex2_approx(8.f - shift - use);
            mx = run;
            l = fmaf(l, corr, (sum.x + sum.y) * by);
          }
          wait(&sm.bar_o[rt], sums & 1);
          ++sums;
          __syncwarp();
          tc_fence_after_sync();
          const bool swap = apart && blk != half;
          add(swap ? its : own, swap ? ex2_approx(other - use) : by, blk ? 1.f : corr);
        }
      }
      it += todo;

      // ---- the unit's rows
      sm.top[rt][half][lrow] = l;
      bar_rt(rt);
      l += sm.top[rt][half ^ 1][lrow];
      const bool whole = u.t0 == 0 && u.end == g + u.cnt;
      if (live) {
        if (whole) {
          finish_part<KIND>(a, u.b, hq, qi, 64 * half, o, mx, l, prior_of<KIND, 64>(a, u.b, hq, qi, 64 * half));
        } else {
          float *part = p.parts + ((long long)slice * 2 + (u.t0 == 0 ? 1 : 0)) * part_of(kUnit);
          const int r = in_unit;
#pragma unroll
          for (int q = 0; q < 16; ++q)
            reinterpret_cast<float4 *>(part)[(16 * half + q) * kUnit + r] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          if (!half) part[kUnit * kD + r] = mx, part[kUnit * (kD + 1) + r] = l;
        }
      }
      if ((APART ? (tid & 255) == 0 : tid == 0) && u.end == g1) {
        const long long stop = g - u.t0 + u.cnt;
        int parts = 0;
        if (u.t0 == 0 && stop > g1) {
          parts = 1;
          for (int k = slice + 1; k < slices && p.cut[k] < stop; ++k) ++parts;
        }
        p.cuts[slice] = Cut{u.b, u.pair, u.h, parts};
      }
      g = u.end;
    }
    if ((APART ? (tid & 255) == 0 : tid == 0) && idle) p.cuts[slice] = Cut{0, 0, 0, 0};
  }
  if (*(volatile int *)&sm.bad) settle();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == kSoft / 32 + 2) tmem_dealloc(tmem, 512);
}

// The rows of a unit that was cut: lane = row, a warp per kJoin times 4 coordinates; 32 rows a CTA.
constexpr int kJoin = 2;  // (2048 of 8192 tokens: 303 us with 1, 299.5 with 2 or 4; 64 rows of 16384 tokens, joined of 18 parts: 44, 44, 47)
template <bool APART, int KIND>
__global__ void __launch_bounds__(1024 / kJoin) q8_prompt_join_kernel(const __grid_constant__ Q8AttnArgs a, const __grid_constant__ Plan p) {
  constexpr int kUnit = unit_rows(APART);
  if constexpr (KIND != kWhole) pdl_trigger();
  pdl_wait();
  const Cut cut = p.cuts[blockIdx.x];
  if (cut.parts < 2) return;
  const int col = threadIdx.x >> 5, r = blockIdx.y * 32 + (threadIdx.x & 31), G = a.group;
  int row, unit1, list;
  unit_span<KIND>(a, cut.pair, kUnit, &row, &unit1, &list);
  row += r;
  int len, m;
  seq_sizes<KIND>(a, cut.b, &len, &m, false);
  const int i = row / G;
  if (row >= unit1 || i >= m) return;
  auto rec = [&](int k) { return p.parts + (((long long)blockIdx.x + k) * 2 + (k == 0 ? 1 : 0)) * part_of(kUnit); };
  float top = -INFINITY;
  float o[kJoin][4], l = 0.f;
#pragma unroll
  for (int j = 0; j < kJoin; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  auto add = [&](float mk, float lk, const float4 (&y)[kJoin]) {
    const float f = mk == -INFINITY ? 1.f : ex2_approx(mk - top);  // without a maximum: zeros (or NaN)
#pragma unroll
    for (int j = 0; j < kJoin; ++j)
      o[j][0] = fmaf(y[j].x, f, o[j][0]), o[j][1] = fmaf(y[j].y, f, o[j][1]), o[j][2] = fmaf(y[j].z, f, o[j][2]), o[j][3] = fmaf(y[j].w, f, o[j][3]);
    l = fmaf(lk, f, l);
  };
  // kPrefix: a unit's parts are many, so that their loads are asked for together (past the last it is the last's again, which is not
  // used): 64 sequences behind 32768 tokens 106 us, 109 without; where they are few that costs (2048 of 8192 tokens 291 -> 294 us)
  constexpr int kTops = KIND == kPrefix ? 16 : 1, kParts = KIND == kPrefix ? 8 : 1;
#pragma unroll(KIND == kPrefix ? 1 : 16)
  for (int k0 = 0; k0 < cut.parts; k0 += kTops) {
    float x[kTops];
#pragma unroll
    for (int k = 0; k < kTops; ++k) x[k] = rec(min(k0 + k, cut.parts - 1))[kUnit * kD + r];
#pragma unroll
    for (int k = 0; k < kTops; ++k) top = fmaxf(top, x[k]);
  }
#pragma unroll(KIND == kPrefix ? 1 : 8)
  for (int k0 = 0; k0 < cut.parts; k0 += kParts) {
    float mk[kParts], lk[kParts];
    float4 y[kParts][kJoin];
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      const float *x = rec(kParts > 1 ? min(k0 + k, cut.parts - 1) : k0);
      mk[k] = x[kUnit * kD + r], lk[k] = x[kUnit * (kD + 1) + r];
#pragma unroll
      for (int j = 0; j < kJoin; ++j) y[k][j] = reinterpret_cast<const float4 *>(x)[(col + 32 / kJoin * j) * kUnit + r];
    }
#pragma unroll
    for (int k = 0; k < kParts; ++k)
      if (k0 + k < cut.parts) add(mk[k], lk[k], y[k]);
  }
  const int hq = cut.h * G + row % G;
  Prior<4> prior[kJoin];
#pragma unroll
  for (int j = 0; j < kJoin; ++j) prior[j] = prior_of<KIND, 4>(a, cut.b, hq, i, 4 * (col + 32 / kJoin * j));
#pragma unroll
  for (int j = 0; j < kJoin; ++j) finish_part<KIND>(a, cut.b, hq, i, 4 * (col + 32 / kJoin * j), o[j], top, l, prior[j]);
}

template <int TERMS, int EXTRA, bool APART, int KIND>
int launch(const Q8AttnArgs &a, const Plan &p, int num_sms, cudaStream_t st) {
  constexpr int smem = stages_of(TERMS, APART) * kStage + 2 * TERMS * kQTerm;
  const int slices = APART ? 2 * num_sms : num_sms;
  if (!allow_shared<q8_prompt_kernel<TERMS, EXTRA, APART, KIND>>(smem)) return TQ_ERR_CUDA;
  cudaError_t e = cudaSuccess;
  if (KIND == kWhole || p.entries > kPlanned) e = launch_overlapped(true, q8_entries_kernel<KIND>, dim3((p.entries + 7) / 8), dim3(256), 0, st, a, p);
  if (e == cudaSuccess) e = launch_overlapped(true, q8_prefix_kernel<KIND>, dim3(1), dim3(1024), 0, st, a, p, slices);
  if (e == cudaSuccess) e = launch_overlapped(true, q8_prompt_kernel<TERMS, EXTRA, APART, KIND>, dim3(num_sms), dim3(kThreads), smem, st, a, p);
  if (e == cudaSuccess)
    e = launch_overlapped(true, q8_prompt_join_kernel<APART, KIND>, dim3(slices, unit_rows(APART) / 32), dim3(1024 / kJoin), 0, st, a, p);
  return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

template <int TERMS, int EXTRA, int KIND>
int launch(const Q8AttnArgs &a, const Plan &p, int num_sms, cudaStream_t st) {
  return p.unit == unit_rows(true) ? launch<TERMS, EXTRA, true, KIND>(a, p, num_sms, st) : launch<TERMS, EXTRA, false, KIND>(a, p, num_sms, st);
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

// Up to 128 rows are one row tile, and the other of a shared unit would have no rows: with units apart every row tile works, but twice as
// many slices are joined and each has half of the ring. So where a CTA has a dozen tiles. 64 rows, 8 KV heads, bf16 (fp16): 8 sequences of
// 16384 tokens (54 tiles a CTA) 121 us apart, 165 us (170, 198) not, capped 178 and 284; 2 of them (13) 59 and 63 (73, 73); one (7) 49 and 45.
bool units_apart(const Q8AttnArgs &a, int num_sms) {
  const long long tiles = (long long)a.batch * a.heads_kv * ((a.max_len + (a.pc.records ? (long long)a.max_prefix : 0) + kTile - 1) / kTile);
  return (long long)a.group * a.n_q <= unit_rows(true) && tiles >= 12LL * num_sms;
}
long long units_of(const Q8AttnArgs &a, bool apart) {
  const long long unit = unit_rows(apart);
  return ((long long)a.group * a.n_q + unit - 1) / unit;
}
// Entries' tiles are counted in 32 bits.
bool many_fits(const Q8AttnArgs &a, int num_sms) {
  const long long entries = units_of(a, units_apart(a, num_sms)) * a.batch, tiles = (a.max_len + kTile - 1) / kTile + (a.pc.records ? (a.max_prefix + kTile - 1) / kTile : 0);
  return entries <= 1 << 24 && entries * tiles <= 0x7fffffff;
}

// Workspace for `entries` units of either kind.
size_t many_bytes(int num_sms, size_t entries) {
  const size_t slices = 2 * (size_t)num_sms;
  return 2 * round16((entries + 1) * sizeof(int)) + round16((slices + 1) * sizeof(long long)) + entries * sizeof(Entry) +
         round16(slices * sizeof(Cut)) + slices * 2 * part_of(unit_rows(true)) * sizeof(float);
}

// Units of `unit` rows, `pairs` of them a sequence; `w`: many_bytes() of workspace.
template <int KIND>
int launch_many(const Q8AttnArgs &a, bool apart, long long pairs, char *w, int num_sms, cudaStream_t st) {
  const long long entries = pairs * a.batch;
  const int slices = apart ? 2 * num_sms : num_sms;
  Plan p;
  p.entries = (int)entries, p.pairs = (int)pairs, p.unit = unit_rows(apart);
  p.pre = (int *)w, w += round16((size_t)(entries + 1) * sizeof(int));
  p.starts = (int *)w, w += round16((size_t)(entries + 1) * sizeof(int));
  p.cut = (long long *)w, w += round16((size_t)(slices + 1) * sizeof(long long));
  p.entry = (Entry *)w, w += (size_t)entries * sizeof(Entry);
  p.cuts = (Cut *)w, w += round16((size_t)slices * sizeof(Cut));
  p.parts = (float *)w;
  const bool extra = a.softcap != 0.f || a.slopes != nullptr || !(a.scale > 0.f), far = a.softcap > kShortCap;
  if (a.q_dtype == TQ_BF16)
    return far ? launch<2, kLongCaps, KIND>(a, p, num_sms, st) : extra ? launch<2, kCapOrBias, KIND>(a, p, num_sms, st) : launch<2, kPlain, KIND>(a, p, num_sms, st);
  return far ? launch<3, kLongCaps, KIND>(a, p, num_sms, st) : extra ? launch<3, kCapOrBias, KIND>(a, p, num_sms, st) : launch<3, kPlain, KIND>(a, p, num_sms, st);
}

}  // namespace
}  // namespace tq
