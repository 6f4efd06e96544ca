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

// One warp per entry (sequence, unit of rows).
__global__ void __launch_bounds__(256) q8_entries_kernel(const __grid_constant__ Q8AttnArgs a, Plan p) {
  const int e = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  pdl_wait();
  if (e >= p.entries) return;
  const int b = e / p.pairs, r0 = (e % p.pairs) * p.unit, G = a.group, R = G * a.n_q;
  int len, m;
  seq_sizes(a, b, &len, &m, lane == 0);
  const int i0 = r0 / G, i1 = min(m - 1, (min(R, r0 + p.unit) - 1) / G);
  int lo = 0x7fffffff, hi = 0, maxbeg = 0, minend = 0x7fffffff;
  for (int i = i0 + lane; i <= i1; i += 32) {
    const int2 r = row_range(a, b, i, len, m);
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
    p.pre[e + 1] = i0 < m ? max(1, (hi + kTile - 1) / kTile - lo / kTile) : 0;
  }
}

// What a unit's start (its queries, the first tile's chain alone) costs, in tiles: ragged documents of 1 to 11 tiles a unit take 127 us in
// slices that count tiles alone, 90 us with 2, 91 with 3, 91 with 5; units of up to 64 tiles, 96 tiles a CTA: 333, 304, 304, 310.
constexpr int kStart = 3;

// Prefix sums of the entries' tiles and the slices, one CTA. Slices are equal in tiles and starts, and none is empty (an
// interval of kStart + 1 holds a tile); with fewer than two tiles a CTA, in tiles alone, so that as many CTAs as possible work.
__global__ void __launch_bounds__(1024) q8_prefix_kernel(Plan p, int heads, int ctas) {
  __shared__ int warp_tiles[32], warp_starts[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int base = 0, base_starts = 0;
  pdl_wait();
  if (tid == 0) p.pre[0] = 0, p.starts[0] = 0;
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
    int before = base, all = base, sbefore = base_starts, sall = base_starts;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += warp_tiles[w], sbefore += warp_starts[w];
      all += warp_tiles[w], sall += warp_starts[w];
    }
    if (e < p.entries) p.pre[e + 1] = before + x, p.starts[e + 1] = sbefore + y;
    base = all, base_starts = sall;
    __syncthreads();
  }
  const long long tiles = (long long)base * heads;
  const int start = tiles >= 2LL * ctas ? kStart : 0;
  const long long total = tiles + (long long)start * base_starts * heads;
  const long long slices = min((long long)ctas, total / (start + 1));
  for (int k = tid; k <= ctas; k += 1024) {
    long long g = tiles;
    if (k < slices) {
      const long long c = total * k / slices;
      int lo = 0, hi = p.entries - 1;
      while (lo < hi) {  // the last entry that begins at or before c
        const int mid = (lo + hi + 1) >> 1;
        if (((long long)p.pre[mid] + (long long)start * p.starts[mid]) * heads <= c) lo = mid;
        else hi = mid - 1;
      }
      const int cnt = p.pre[lo + 1] - p.pre[lo], each = cnt + start;
      const long long in = c - ((long long)p.pre[lo] + (long long)start * p.starts[lo]) * heads;
      g = (long long)p.pre[lo] * heads + in / each * cnt + max(0, (int)(in % each) - start);
    }
    p.cut[k] = g;
  }
}

struct Shared {
  uint64_t full[4], empty[4];
  uint64_t bar_q[2], bar_s[2], bar_p[2], bar_o[2];  // of a row tile: queries, scores, probabilities, value sums are there
  float4 info[4];             // of a stage: key scales of the tile's two blocks, value scales (negative: not there)
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
  u.h = (int)(in / u.cnt), u.t0 = (int)(in - (long long)u.h * u.cnt);
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

template <int TERMS, int EXTRA, bool APART>
__global__ void __launch_bounds__(kThreads, 1)
q8_prompt_kernel(const __grid_constant__ Q8AttnArgs a, const __grid_constant__ Plan p) {
  constexpr int kStages = stages_of(TERMS, APART), kUnit = unit_rows(APART);
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
        const long long blocks = ((long long)u.b * a.heads_kv + u.h) * a.c.nblk;
        for (int k0 = 0; g + k0 < u.end; k0 += 32) {
          const int todo = (int)min(32ll, u.end - g - k0);
          long long src[2] = {-1, -1};
          float4 f = make_float4(-1.f, -1.f, -1.f, -1.f);
          int bytes[2] = {0, 0};
          if (lane < todo) {
            const int tok = (en.lo / kTile + u.t0 + k0 + lane) * kTile, n = min(kTile, max(0, en.hi - tok));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int m = min(kQ8Block, n - k * kQ8Block);
              if (m <= 0 || tok + (k + 1) * kQ8Block <= en.lo) continue;  // no row sees a token of it
              src[k] = q8_block(a.c.btab, a.c.pool_blocks, blocks + tok / kQ8Block + k, a.error);
              if (src[k] < 0) continue;
              bytes[k] = (m + 31) / 32 * 32 * kD;  // whole K-steps of the value MMA
              (k ? f.y : f.x) = __ldg(a.c.ks + src[k]);
              (k ? f.w : f.z) = __ldg(a.c.vs + src[k]);
            }
          }
          for (int k = 0; k < todo; ++k, ++it) {
            const int s = stage(it);
            const long long s0 = __shfl_sync(kFull, src[0], k), s1 = __shfl_sync(kFull, src[1], k);
            const int n0 = __shfl_sync(kFull, bytes[0], k), n1 = __shfl_sync(kFull, bytes[1], k);
            float4 x;
            x.x = __shfl_sync(kFull, f.x, k), x.y = __shfl_sync(kFull, f.y, k);
            x.z = __shfl_sync(kFull, f.z, k), x.w = __shfl_sync(kFull, f.w, k);
            if (lane == 0) {
              wait(&sm.empty[s], turn(it) ^ 1);
              if (!*(volatile int *)&sm.bad) {
                sm.info[s] = x;
                uint8_t *dst = ring + s * kStage;
                mbar_arrive_expect_tx(&sm.full[s], 2 * (n0 + n1));
                if (n0) {
                  const uint8_t *q = a.c.records + s0 * kQ8BlockBytes;
                  tma_load_1d(dst, q, n0, &sm.full[s]);
                  tma_load_1d(dst + kTile * kD, q + kQ8Plane, n0, &sm.full[s]);
                }
                if (n1) {
                  const uint8_t *q = a.c.records + s1 * kQ8BlockBytes;
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
          wait(&sm.bar_q[rt], units & 1);
          for (int j = 0; j <= todo; ++j) {
            // the value sums of tile j - 1, then the scores of tile j over its probabilities: in this order, as issued
            if (j > 0) {
              const int s = stage(it + j - 1), n = min(kTile, max(0, hi - (first + j - 1) * kTile));
              const float4 f = sm.info[s];
              const bool apart = scales_apart(f), whole = n == kTile && f.z >= 0.f && f.w >= 0.f && !apart;
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
                      if (k * 32 >= n || (k < 2 ? f.z : f.w) < 0.f || (apart && k / 2 != part)) continue;
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
      seq_sizes(a, u.b, &len, &m, false);
      const int G = a.group, R = G * a.n_q;

      // ---- queries: a warp prepares 16 rows of its row tile (whose score MMAs of the unit before are done)
      bar_rt(rt);
#pragma unroll 1
      for (int k0 = 0; k0 < 16; k0 += 8) {
        uint2 raw[8];
        const int first_row = u.pair * kUnit + (APART ? 0 : rt * 128) + (warp & 7) * 16 + k0;
        load_rows(a, u.b, u.h, m, first_row, lane, raw);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = (warp & 7) * 16 + k0 + k, row = first_row + k;
          float x[4];
          row_floats(a, raw[k], row < R && row / G < m, x);
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
      const int row = u.pair * kUnit + in_unit, qi = row / G, hq = u.h * G + row % G;
      const bool live = row < R && qi < m;
      const int2 rg = live ? row_range(a, u.b, qi, len, m) : make_int2(0, 0);
      const float slope = EXTRA && live && a.slopes ? __ldg(a.slopes + hq) * kLog2e : 0.f;
      const int qp = !EXTRA || !live ? 0 : a.qpos ? __ldg(a.qpos + (long long)u.b * a.n_q + qi) : len - m + qi;
      bar_rt(rt);

      float o[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) o[i] = 0.f;
      float mx = -INFINITY, l = 0.f;
      const int todo = (int)(u.end - g);
      for (int j = 0; j < todo; ++j) {
        const int s = stage(it + j), tok0 = (first + j) * kTile, n = min(kTile, max(0, hi - tok0));
        wait(&sm.full[s], turn(it + j));
        const float4 f = sm.info[s];
        const float ks = half ? f.y : f.x;
        const bool masked = !(maxbeg <= tok0 && minend >= tok0 + kTile) || f.x < 0.f || f.y < 0.f;
        int from = 0, to = 64;  // the tokens of this half that the row sees
        if (masked) {
          from = min(max(rg.x - tok0 - 64 * half, 0), 64), to = min(max(rg.y - tok0 - 64 * half, 0), 64);
          if (ks < 0.f) to = 0;
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
                for (int i = 0; i < 16; ++i) x[i] = fmaf(-slope, (float)__sad(qp, slot0 + 16 * q + i < hi ? __ldg(kp + i) : 0, 0u), x[i]);
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
          const int t = n + (tid & 255);
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
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const long long off = u.b * a.os.b + hq * a.os.h + qi * a.os.t + 64 * half;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = o[8 * q + i] * inv;
            if (a.out_dtype == TQ_BF16) store_vec<__nv_bfloat16, 8>(static_cast<__nv_bfloat16 *>(a.out) + off + 8 * q, y);
            else store_vec<__half, 8>(static_cast<__half *>(a.out) + off + 8 * q, y);
          }
          if (a.lse && !half) a.lse[((long long)u.b * a.heads_q + hq) * a.n_q + qi] = (mx + log2f(l) - 8.f) * kLn2;
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
template <bool APART>
__global__ void __launch_bounds__(1024 / kJoin) q8_prompt_join_kernel(const __grid_constant__ Q8AttnArgs a, const __grid_constant__ Plan p) {
  constexpr int kUnit = unit_rows(APART);
  pdl_wait();
  const Cut cut = p.cuts[blockIdx.x];
  if (cut.parts < 2) return;
  const int col = threadIdx.x >> 5, r = blockIdx.y * 32 + (threadIdx.x & 31), row = cut.pair * kUnit + r, G = a.group;
  int len, m;
  seq_sizes(a, cut.b, &len, &m, false);
  const int i = row / G;
  if (row >= G * a.n_q || i >= m) return;
  auto rec = [&](int k) { return p.parts + (((long long)blockIdx.x + k) * 2 + (k == 0 ? 1 : 0)) * part_of(kUnit); };
  float top = -INFINITY;
#pragma unroll 8
  for (int k = 0; k < cut.parts; ++k) top = fmaxf(top, rec(k)[kUnit * kD + r]);
  float o[kJoin][4], l = 0.f;
#pragma unroll
  for (int j = 0; j < kJoin; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
#pragma unroll 4
  for (int k = 0; k < cut.parts; ++k) {
    const float *x = rec(k);
    const float mk = x[kUnit * kD + r], f = mk == -INFINITY ? 1.f : ex2_approx(mk - top);  // without a maximum: zeros (or NaN)
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
      const float4 y = reinterpret_cast<const float4 *>(x)[(col + 32 / kJoin * j) * kUnit + r];
      o[j][0] = fmaf(y.x, f, o[j][0]), o[j][1] = fmaf(y.y, f, o[j][1]), o[j][2] = fmaf(y.z, f, o[j][2]), o[j][3] = fmaf(y.w, f, o[j][3]);
    }
    l = fmaf(x[kUnit * (kD + 1) + r], f, l);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int hq = cut.h * G + row % G;
#pragma unroll
  for (int j = 0; j < kJoin; ++j) {
#pragma unroll
    for (int k = 0; k < 4; ++k) o[j][k] *= inv;
    const long long off = cut.b * a.os.b + hq * a.os.h + i * a.os.t + 4 * (col + 32 / kJoin * j);
    if (a.out_dtype == TQ_BF16) store_vec<__nv_bfloat16, 4>(static_cast<__nv_bfloat16 *>(a.out) + off, o[j]);
    else store_vec<__half, 4>(static_cast<__half *>(a.out) + off, o[j]);
  }
  if (a.lse && col == 0) a.lse[((long long)cut.b * a.heads_q + hq) * a.n_q + i] = (top + log2f(l) - 8.f) * kLn2;
}

template <int TERMS, int EXTRA, bool APART>
int launch(const Q8AttnArgs &a, const Plan &p, int num_sms, cudaStream_t st) {
  constexpr int smem = stages_of(TERMS, APART) * kStage + 2 * TERMS * kQTerm;
  const int slices = APART ? 2 * num_sms : num_sms;
  if (cudaFuncSetAttribute(q8_prompt_kernel<TERMS, EXTRA, APART>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return TQ_ERR_CUDA;
  cudaError_t e = launch_overlapped(true, q8_entries_kernel, dim3((p.entries + 7) / 8), dim3(256), 0, st, a, p);
  if (e == cudaSuccess) e = launch_overlapped(true, q8_prefix_kernel, dim3(1), dim3(1024), 0, st, p, a.heads_kv, slices);
  if (e == cudaSuccess) e = launch_overlapped(true, q8_prompt_kernel<TERMS, EXTRA, APART>, dim3(num_sms), dim3(kThreads), smem, st, a, p);
  if (e == cudaSuccess)
    e = launch_overlapped(true, q8_prompt_join_kernel<APART>, dim3(slices, unit_rows(APART) / 32), dim3(1024 / kJoin), 0, st, a, p);
  return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

// Up to 128 rows are one row tile, and the other of a shared unit would have no rows: with units apart every row tile works, but twice as
// many slices are joined and each has half of the ring. So where a CTA has a dozen tiles. 64 rows, 8 KV heads, bf16 (fp16): 8 sequences of
// 16384 tokens (54 tiles a CTA) 121 us apart, 165 us (170, 198) not, capped 178 and 284; 2 of them (13) 59 and 63 (73, 73); one (7) 49 and 45.
bool units_apart(const Q8AttnArgs &a, int num_sms) {
  const long long tiles = (long long)a.batch * a.heads_kv * ((a.max_len + kTile - 1) / kTile);
  return (long long)a.group * a.n_q <= unit_rows(true) && tiles >= 12LL * num_sms;
}
template <int TERMS, int EXTRA>
int launch(const Q8AttnArgs &a, const Plan &p, int num_sms, cudaStream_t st) {
  return p.unit == unit_rows(true) ? launch<TERMS, EXTRA, true>(a, p, num_sms, st) : launch<TERMS, EXTRA, false>(a, p, num_sms, st);
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

}  // namespace

// Enough for either kind of units.
size_t q8_prompt_workspace(int num_sms, int batch, int group, int n_q) {
  const size_t entries = ((size_t)group * n_q + unit_rows(false) - 1) / unit_rows(false) * batch, slices = 2 * (size_t)num_sms;
  return 2 * round16((entries + 1) * sizeof(int)) + round16((slices + 1) * sizeof(long long)) + entries * sizeof(Entry) +
         round16(slices * sizeof(Cut)) + slices * 2 * part_of(unit_rows(true)) * sizeof(float);
}

static long long units_of(const Q8AttnArgs &a, bool apart) {
  const long long unit = unit_rows(apart);
  return ((long long)a.group * a.n_q + unit - 1) / unit;
}

// Entries' tiles are counted in 32 bits.
bool q8_prompt_fits(const Q8AttnArgs &a, int num_sms) {
  const long long entries = units_of(a, units_apart(a, num_sms)) * a.batch, tiles = (a.max_len + kTile - 1) / kTile;
  return entries <= 1 << 24 && entries * tiles <= 0x7fffffff;
}

int launch_q8_prompt(const Q8AttnArgs &a, void *workspace, int num_sms, void *stream) {
  const bool apart = units_apart(a, num_sms);
  const long long unit = unit_rows(apart), pairs = units_of(a, apart), entries = pairs * a.batch;
  const int slices = apart ? 2 * num_sms : num_sms;
  Plan p;
  p.entries = (int)entries, p.pairs = (int)pairs, p.unit = (int)unit;
  char *w = (char *)workspace;
  p.pre = (int *)w, w += round16((size_t)(entries + 1) * sizeof(int));
  p.starts = (int *)w, w += round16((size_t)(entries + 1) * sizeof(int));
  p.cut = (long long *)w, w += round16((size_t)(slices + 1) * sizeof(long long));
  p.entry = (Entry *)w, w += (size_t)entries * sizeof(Entry);
  p.cuts = (Cut *)w, w += round16((size_t)slices * sizeof(Cut));
  p.parts = (float *)w;
  cudaStream_t st = (cudaStream_t)stream;
  const bool extra = a.softcap != 0.f || a.slopes != nullptr || !(a.scale > 0.f), far = a.softcap > kShortCap;
  if (a.q_dtype == TQ_BF16)
    return far ? launch<2, kLongCaps>(a, p, num_sms, st) : extra ? launch<2, kCapOrBias>(a, p, num_sms, st) : launch<2, kPlain>(a, p, num_sms, st);
  return far ? launch<3, kLongCaps>(a, p, num_sms, st) : extra ? launch<3, kCapOrBias>(a, p, num_sms, st) : launch<3, kPlain>(a, p, num_sms, st);
}

}  // namespace tq
