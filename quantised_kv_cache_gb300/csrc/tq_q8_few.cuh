// Attention over the 8-bit cache for few query rows per KV head (tq_q8_attention): decode steps,
// drafts, short prompts. Up to 16 rows (query tokens x heads of the group; 8 for 32-bit results) are one unit of work with
// a (sequence, KV head).
//
// Mathematics, per unit: S = K Q^T for 128 tokens at a time (token = accumulator lane, row = column),
// t = log2(e) score, running maximum m and sum l of 2^(t - m) per row, O = sum 2^(t - m) v. The codes of
// the keys and values are tensor-core operands as they lie in the cache (no conversion, no
// transposition); queries and probabilities enter as 4 e5m2 terms (8 for fp32 results), side by side in
// one operand. A block's scale multiplies the scores of its tokens, and its part of O.
//
// Bound by the cache's bytes: 256 per token and KV head, read once. Per SM a tile of 128 tokens
// (32 KB) may take 1500 clocks at the memory's rate; its 8 MMAs of 128 x (16 .. 64) x 32 take 43 to 50 each, the
// time of reading the 128-row operand. 4 warpgroups work on 4 tiles at once, each alone on its
// tile from the score MMAs to the value sums, so that the chain of a tile (two MMA round trips, three barriers) is hidden by
// the other three. One producer warp keeps a ring of 5
// tiles filled by bulk copies (whole 8 KB planes). Grid: one CTA per SM; the (sequence, row tile, head, tile) space is
// cut into equal slices, so ragged batches and long single sequences load every SM alike. A unit that lies in one
// slice is finished there; one that was cut leaves a partial record per slice, joined by q8_join_kernel.
// The probabilities' sum for the output counts what their terms hold, that of the log-sum the numbers themselves.
// Measured: 16 sequences of 8192 tokens, 32 KV heads, one row each: 158 us, 6.8 TB/s, a plain copy's rate. One sequence of 131072
// tokens, 8 KV heads of 4 rows, capped, paged: 55 us where its bytes take 40: the rest is the launch, the queries, the first tile's
// latency and the join. 32-bit results, 4 sequences of up to 16383 tokens, 8 KV heads of 6 rows: 53 us where the bytes take 13: a CTA has 17 tiles,
// and the chain of each (8 terms to form, 64 operand columns) shows. One sequence of 1000 tokens: 14 us with its weights, all latency.
//
// The same kernel takes listed blocks (a tile is two of a list's), a shared prefix (the batch's rows as one sequence's) and the own tokens behind
// one. There, where the units are few, a cluster's CTAs share a unit (TEAM): they know theirs without the table of entries and the search,
// and join their parts through each other's shared memory, so that there is one launch. Of 9.8 us for 8 KV heads of 4 rows over 64 blocks, 2.5 are
// the launch, 3 the chain from lengths over list, table and scales to the first keys, 2 a tile, 2 the ends.

#pragma once

#include <cooperative_groups.h>

#include <algorithm>

#include "tq_q8_rows.cuh"

namespace tq {
namespace {

constexpr int kTile = 128;              // tokens of a tile
constexpr int kStage = 2 * kTile * kD;  // its keys, then its values
constexpr int kWg = 4;                  // warpgroups, each with a tile of its own
constexpr int kConsumers = kWg * 128;
constexpr int kThreads = kConsumers + 32;
constexpr int kEntries = 512;           // (sequence, row tile) pairs of a launch
// Rows up to which this kernel takes a 16-bit call: one unit. 16 rows of one sequence over 16384 tokens, 8 KV heads: 40 us
// here, 40 (bf16) or 47 (fp16) in the kernel for many rows, 148 against 120 or 169 in a batch of 8; 20 rows (two units, which
// read the cache twice): 64 against 43 or 49, in a batch of 8 243 against 120 or 169. Up to 16 rows also keep 12 bits in both types.
constexpr long long kFewRows = 16;
constexpr int kPartRow = kD + 4;        // a partial record's row: O, m, l, rounded l, pad

constexpr int kStages = 5;
constexpr int kRows = 16;               // rows of a partial record
constexpr int kMostRanks = 8;           // CTAs of a cluster
constexpr int rows_of(int T) { return T == 8 ? 8 : 16; }  // rows of a unit: what tensor memory holds the terms' columns of

struct Entries {
  int pre[kEntries + 1];  // tiles (of one head) before each entry
  int lo[kEntries];       // its first visible slot
  int hi[kEntries];       // one past its last visible slot
};

// What the main kernel tells the join about each CTA's last unit.
struct Cut {
  int b, rt, h, parts;  // parts: CTAs that hold a part of it, 0 when it was not cut (or began elsewhere)
};

struct Shared {
  // A tile's arrival barrier is one of stages x warpgroups, so that its earlier use was the same warpgroup's: a
  // warpgroup that is ahead would take a parity of a stage's older, still incomplete copy for its own.
  uint64_t full[kStages * kWg], empty[kStages], bar_s[kWg], bar_o[kWg];
  float4 info[kStages];      // key scales of the tile's two blocks, value scales (negative: not mapped)
  int2 at[kStages];          // (kListed) their first slots
  float qscale[kRows], slope[kRows];
  int2 range[kRows];
  int qpos[kRows];
  float4 wmax[kWg][kRows];   // row maxima of a warpgroup's four warps
  float m[kWg][kRows], l[kWg][kRows], lr[kWg][kRows];
  float lw[kWg][4][kRows], lrw[kWg][4][kRows];
  uint32_t tmem;
  int bad, scan[kThreads / 32];
  Entries ent;
};

__device__ __forceinline__ void bar_all() { asm volatile("bar.sync 5, %0;" ::"n"(kConsumers) : "memory"); }

// TEAM: a cluster's CTAs share one unit and join its parts through each other's shared memory; the units are numbered [sequence][rts][head].
template <int NR, int T, int KIND, bool TEAM>
__global__ void __launch_bounds__(kThreads, 1)
q8_attend_kernel(const __grid_constant__ Q8AttnArgs a, int b0, int nb, int rt0, int rts, Cut *cuts) {
  constexpr int kUnitRows = TEAM ? NR : rows_of(T), kN = stacked_rows(NR, T), kOp = kN * 128;  // an operand's rows and bytes
  constexpr int kCols = 2 * kN;  // a warpgroup's columns: S, in its place O of the first block, then O of the second
  static_assert(NR <= kUnitRows && kWg * kCols <= 512 && kWg * NR * 512 <= kWg * kOp, "");
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ Shared sm;
  uint8_t *ring = dyn, *qbuf = dyn + kStages * kStage, *pbuf = qbuf + kOp;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.group;
  [[maybe_unused]] const int R = G * a.n_q;

  if (tid == 0) {
    for (int s = 0; s < kStages * kWg; ++s) mbar_init(&sm.full[s], 1);
    for (int s = 0; s < kStages; ++s) mbar_init(&sm.empty[s], 1);
    for (int w = 0; w < kWg; ++w) mbar_init(&sm.bar_s[w], 1), mbar_init(&sm.bar_o[w], 1);
    mbar_fence_init();
    sm.bad = 0;
  }
  if (warp == kThreads / 32 - 1) {
    tmem_alloc(smem_u32(&sm.tmem), kWg * kCols);
    tmem_relinquish();
  }
  if constexpr (KIND != kWhole) pdl_trigger();  // the join waits for all of this grid, but its blocks may come as this one's leave
  pdl_wait();

  namespace cg = cooperative_groups;
  const int ranks = TEAM ? (int)cg::this_cluster().num_blocks() : 1, rank = TEAM ? (int)cg::this_cluster().block_rank() : 0;
  const int team = TEAM ? blockIdx.x / ranks : 0, team_h = team % a.heads_kv, team_x = team / a.heads_kv % rts, team_b = team / a.heads_kv / rts;
  int team_lo = 0x7fffffff, team_hi = 0, team_tiles = 0;
  const int E = nb * rts;
  if constexpr (TEAM) {  // every warp looks for itself, a lane at a token
    int len, m, r0, end, list;
    unit_span<KIND>(a, team_x, kUnitRows, &r0, &end, &list);
    seq_sizes<KIND>(a, team_b, &len, &m, tid == 0);
    const int i0 = r0 / G, i1 = (min(end, r0 + kUnitRows) - 1) / G;
    if (i0 + lane <= i1) {
      const int2 r = row_range<KIND>(a, team_b, i0 + lane, len, m);
      if (r.y > r.x) team_lo = r.x, team_hi = r.y;
    }
    team_lo = __reduce_min_sync(kFull, team_lo), team_hi = __reduce_max_sync(kFull, team_hi);
    if (team_hi == 0) team_lo = 0;
    team_tiles = i0 < m ? max(1, unit_tiles<KIND>(a, team_b, team_lo, team_hi)) : 0;
  } else {
  // ---- the entries' tiles: one thread each
  int count = 0;
  if (KIND != kWhole && E <= kThreads / 32) {  // a warp each: a lane looks at a token (16 rows of a prefix's are as many sequences')
    int most = 0;
    if (warp < E) {
      int len, m, r0, end, list;
      unit_span<KIND>(a, rt0 + warp % rts, kUnitRows, &r0, &end, &list);
      seq_sizes<KIND>(a, b0 + warp / rts, &len, &m, blockIdx.x == 0 && lane == 0);
      const int i0 = r0 / G, i1 = (min(end, r0 + kUnitRows) - 1) / G;
      int lo = 0x7fffffff, hi = 0;
      if (i0 + lane <= i1) {
        const int2 r = row_range<KIND>(a, b0 + warp / rts, i0 + lane, len, m);
        if (r.y > r.x) lo = r.x, hi = r.y;
      }
      lo = __reduce_min_sync(kFull, lo), hi = __reduce_max_sync(kFull, hi);
      if (hi == 0) lo = 0;
      most = i0 < m ? max(1, unit_tiles<KIND>(a, b0 + warp / rts, lo, hi)) : 0;
      if (lane == 0) sm.ent.lo[warp] = lo, sm.ent.hi[warp] = hi, sm.ent.pre[warp] = most;
    }
    __syncthreads();
    if (tid < E) count = sm.ent.pre[tid];
    __syncthreads();
  } else if (tid < E) {
    const int b = b0 + tid / rts;
    int len, m, r0, end, list;
    unit_span<KIND>(a, rt0 + tid % rts, kUnitRows, &r0, &end, &list);
    seq_sizes<KIND>(a, b, &len, &m, blockIdx.x == 0);
    const int i0 = r0 / G, i1 = (min(end, r0 + kUnitRows) - 1) / G;
    int lo = 0x7fffffff, hi = 0;
    for (int i = i0; i <= i1; ++i) {
      const int2 r = row_range<KIND>(a, b, i, len, m);
      if (r.y > r.x) lo = min(lo, r.x), hi = max(hi, r.y);
    }
    if (hi == 0) lo = 0;
    // an entry whose rows see nothing keeps one (empty) tile, so that its zeros are written
    count = i0 < m ? max(1, unit_tiles<KIND>(a, b, lo, hi)) : 0;
    sm.ent.lo[tid] = lo;
    sm.ent.hi[tid] = hi;
  }
  {
    int x = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sm.scan[warp] = x;
    __syncthreads();
    const int before = __reduce_add_sync(kFull, lane < warp ? sm.scan[lane] : 0);
    if (tid < E) sm.ent.pre[tid + 1] = before + x;
    if (tid == 0) sm.ent.pre[0] = 0;
  }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sm.tmem;
  const long long total = TEAM ? team_tiles : (long long)sm.ent.pre[E] * a.heads_kv;
  // slices, none of them empty: CTA c < slices has tiles [total c / slices, total (c + 1) / slices)
  const long long slices = TEAM ? ranks : min((long long)gridDim.x, total), slice = TEAM ? rank : blockIdx.x;
  const bool idle = slice >= slices;
  const long long g0 = idle ? 0 : quotient(total * slice, slices), g1 = idle ? 0 : quotient(total * (slice + 1), slices);
  auto locate = [&](long long g, int &e, int &h, int &t, int &cnt) {
    if constexpr (TEAM) {
      e = 0, h = team_h, t = (int)g, cnt = team_tiles;
      return;
    }
    int lo = 0, hi = E - 1;
    while (lo < hi) {  // the last entry that begins at or before g
      const int mid = (lo + hi + 1) >> 1;
      if ((long long)sm.ent.pre[mid] * a.heads_kv <= g) lo = mid;
      else hi = mid - 1;
    }
    e = lo;
    cnt = sm.ent.pre[e + 1] - sm.ent.pre[e];
    const long long in = g - (long long)sm.ent.pre[e] * a.heads_kv;
    h = (int)quotient(in, cnt);
    t = (int)(in - (long long)h * cnt);
  };
  auto seq_of = [&](int e) { return TEAM ? team_b : b0 + e / rts; };
  auto unit_of = [&](int e) { return TEAM ? team_x : rt0 + e % rts; };
  auto lo_of = [&](int e) { return TEAM ? team_lo : sm.ent.lo[e]; };
  auto hi_of = [&](int e) { return TEAM ? team_hi : sm.ent.hi[e]; };
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (*(volatile int *)&sm.bad) return;
    if (!mbar_wait_bounded(bar, parity, a.error)) *(volatile int *)&sm.bad = 1;
  };

  if (warp == kThreads / 32 - 1) {
    // ================================ producer: one lane finds the sources of one of the next 32 tiles
    int it = 0;
    for (long long g = g0; g < g1; g += 32) {
      long long src[2] = {-1, -1};
      float4 info = make_float4(-1.f, -1.f, -1.f, -1.f);
      int bytes[2] = {0, 0}, at[2] = {0, 0};
      if (g + lane < g1) {
        int e, h, t, cnt, blk[2];
        locate(g + lane, e, h, t, cnt);
        const int lo = lo_of(e);
        const long long bh = (long long)seq_of(e) * a.heads_kv + h;
        if constexpr (KIND == kListed) {
          int r0, end, list;
          unit_span<KIND>(a, unit_of(e), kUnitRows, &r0, &end, &list);
          list_entries(a, bh, list, 2 * t, blk);
        } else {
          blk[0] = 2 * (lo / kTile + t), blk[1] = blk[0] + 1;
        }
        info = tile_sources(a, a.c, bh, blk, 0, lo, hi_of(e), src, bytes, at);
      }
      const int todo = (int)min(32ll, g1 - g);
      for (int k = 0; k < todo; ++k, ++it) {
        const int s = it % kStages;
        const long long s0 = __shfl_sync(kFull, src[0], k), s1 = __shfl_sync(kFull, src[1], k);
        const int n0 = __shfl_sync(kFull, bytes[0], k), n1 = __shfl_sync(kFull, bytes[1], k);
        float4 f;
        f.x = __shfl_sync(kFull, info.x, k), f.y = __shfl_sync(kFull, info.y, k);
        f.z = __shfl_sync(kFull, info.z, k), f.w = __shfl_sync(kFull, info.w, k);
        int2 first = make_int2(0, 0);
        if constexpr (KIND == kListed) first.x = __shfl_sync(kFull, at[0], k), first.y = __shfl_sync(kFull, at[1], k);
        if (lane == 0) {
          wait(&sm.empty[s], ((it / kStages) & 1) ^ 1);
          if (!*(volatile int *)&sm.bad) {
            sm.info[s] = f;
            if constexpr (KIND == kListed) sm.at[s] = first;
            uint8_t *dst = ring + s * kStage;
            uint64_t *full = &sm.full[it % (kStages * kWg)];
            mbar_arrive_expect_tx(full, 2 * (n0 + n1));
            if (n0) {
              const uint8_t *p = a.c.records + s0 * kQ8BlockBytes;
              tma_load_1d(dst, p, n0, full);
              tma_load_1d(dst + kTile * kD, p + kQ8Plane, n0, full);
            }
            if (n1) {
              const uint8_t *p = a.c.records + s1 * kQ8BlockBytes;
              tma_load_1d(dst + kQ8Plane, p, n1, full);
              tma_load_1d(dst + kTile * kD + kQ8Plane, p + kQ8Plane, n1, full);
            }
          }
        }
        __syncwarp();
      }
    }
    // every copy lands before the CTA's shared memory goes: the last fill of each stage
    if (lane == 0) {
      for (int k = max(0, it - kStages); k < it; ++k)
        mbar_wait_bounded(&sm.full[k % (kStages * kWg)], (k / (kStages * kWg)) & 1, nullptr, kWaitBudgetNs / 8);
    }
    __syncwarp();
  } else {
    // ================================ consumers
    const int wg = warp >> 2, wt = tid & 127, w4 = warp & 3;
    const uint32_t t_s = tmem + wg * kCols;
    const uint32_t lanes = (uint32_t)(32 * w4) << 16;
    uint8_t *const pmine = pbuf + wg * kOp;
    uint8_t *const pbyte = pmine + (wt >> 4) * 128 + (wt & 15);
    const bool issue = elect_lane();  // of the warpgroup's first warp
    const uint32_t u_s = warp_uniform(t_s), u_q = smem_u32(qbuf), u_p = warp_uniform(smem_u32(pmine));
    const Q8Score sc{a.scale, a.softcap, a.softcap != 0.f ? 1.f / a.softcap : 0.f};
    uint32_t phase = 0;  // of this warpgroup's two barriers: its tiles so far
    long long g = g0;
    while (g < g1 || (TEAM && total > 0)) {
      int e, h, t0, cnt;
      locate(g, e, h, t0, cnt);
      const int b = seq_of(e);
      int row0, row_end, list;
      unit_span<KIND>(a, unit_of(e), kUnitRows, &row0, &row_end, &list);
      const long long end = min(g1, g - t0 + cnt);
      const int first = lo_of(e) / kTile, hi = hi_of(e);

      // ---- the unit's queries: warp w prepares row w
      {
        const int row = row0 + warp, i = row / G, hq = h * G + row % G;
        int len, m;
        seq_sizes<KIND>(a, b, &len, &m, false);
        const bool live = warp < NR && row < row_end && i < m;
        // (asked for with the query: behind the barrier it would be one more wait)
        const int2 rg = live ? row_range<KIND>(a, b, i, len, m) : make_int2(0, 0);
        const float slope = live && a.slopes ? latest(a.slopes + hq) : 0.f;
        const int qpos = !live ? 0 : a.qpos ? latest(a.qpos + (long long)b * a.n_q + i) : query_slot<KIND>(a, i, len, m);
        uint32_t w[T];
        const int ex = row_e5m2<T, KIND>(a, b, hq, i, live, lane, w);
        bar_all();  // everyone is done with the unit before
        if (warp < NR) {
#pragma unroll
          for (int k = 0; k < T; ++k) *reinterpret_cast<uint32_t *>(qbuf + q8_off(k * NR + warp, 4 * lane)) = w[k];
          if (lane == 0) {
            sm.qscale[warp] = pow2i(ex);
            sm.range[warp] = rg;
            sm.slope[warp] = slope * kLog2e;
            sm.qpos[warp] = qpos;
          }
        }
        fence_proxy_async_shared();
        bar_all();
      }

      float m[NR], l[NR], lr[NR], o[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) m[r] = -INFINITY, l[r] = 0.f, lr[r] = 0.f, o[r] = 0.f;

      for (long long gt = g + ((wg - (int)(g - g0)) & (kWg - 1)); gt < end; gt += kWg) {
        const int it = (int)(gt - g0), s = it % kStages;
        int tok0 = (first + t0 + (int)(gt - g)) * kTile, n = min(kTile, max(0, hi - tok0));  // (kListed: of the thread's block, below)
        wait(&sm.full[it % (kStages * kWg)], (it / (kStages * kWg)) & 1);
        if (w4 == 0) {
          __syncwarp();
          tc_fence_after_sync();
          const uint32_t ring_k = warp_uniform(smem_u32(ring + s * kStage));
#pragma unroll
          for (int ks = 0; ks < kD / 32; ++ks)
            if (issue)
              tc_mma_f8(u_s, tc_sdesc_kmajor(ring_k + 256 * ks, 128, 1024), tc_sdesc_kmajor(u_q + 256 * ks, 128, 1024),
                        tc_idesc_f8(128, kN, 0, 1, 0, 0), ks > 0);
          if (issue) tc_commit(smem_u32(&sm.bar_s[wg]));
          __syncwarp();
        }
        const float4 info = sm.info[s];
        const float ks = wt < kQ8Block ? info.x : info.y;
        int2 at = make_int2(0, 0);
        if constexpr (KIND == kListed) {  // the thread's block begins 64 threads before the second one's do
          at = sm.at[s];
          tok0 = wt < kQ8Block ? at.x : at.y - kQ8Block;
          n = (wt & kQ8Block) + (ks < 0.f ? 0 : min(kQ8Block, hi - tok0 - (wt & kQ8Block)));
        }
        // value rows of the last K-step past the copied tokens hold whatever the cache holds there
        if (wt >= n && wt < ((n + 31) & ~31)) {
          uint8_t *row = ring + s * kStage + kTile * kD + q8_off(wt, 0);
#pragma unroll
          for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(row + 128 * c) = make_uint4(0, 0, 0, 0);
        }
        const int slot = tok0 + wt;
        int kp = slot;
        if (a.kpos && slot < hi) kp = latest(a.kpos + ((long long)b * a.heads_kv + h) * a.c.capacity + slot);
        wait(&sm.bar_s[wg], phase & 1);
        __syncwarp();  // the loads from tensor memory are a warp's
        tc_fence_after_sync();
        float t[NR];
        tmem_term_sums<NR, T>(t_s + lanes, t);
        // ---- scores, and the rows' maxima over the tile
        float mine = -INFINITY;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const int2 rg = sm.range[r];
          t[r] = q8_score_log2(t[r] * (sm.qscale[r] * ks), sc);
          if (a.slopes) t[r] = fmaf(-sm.slope[r], (float)__sad(sm.qpos[r], kp, 0u), t[r]);
          if (slot < rg.x || slot >= rg.y || ks < 0.f) t[r] = -INFINITY;
          if (KIND == kWhole && a.scores && row0 + r < R) a.scores[((((long long)b * a.heads_kv + h) * R + row0 + r) * a.scores_ld) + slot] = t[r];
          const float w = warp_fmax(t[r]);
          if (lane == r) mine = w;
        }
        if (lane < NR) reinterpret_cast<float *>(&sm.wmax[wg][lane])[w4] = mine;
        bar_wg(wg);
        // ---- probabilities (times 2^15), their terms, the sums
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float4 x = sm.wmax[wg][r];
          const float top = fmaxf(fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)), m[r]);
          const float use = top == -INFINITY ? 0.f : top;
          const float corr = ex2_approx(m[r] - use);
          m[r] = top;
          t[r] = ex2_approx(t[r] - use + 15.f);
          l[r] = fmaf(l[r], corr, t[r]);
          lr[r] = fmaf(lr[r], corr, t[r]);
          o[r] *= corr;
        }
#pragma unroll
        for (int r = 0; r < NR; r += 2) {
          const int r1 = r + 1 < NR ? r + 1 : r;
          float p0 = t[r], p1 = t[r1];
          uint32_t term[T];
          split_e5m2<T>(p0, p1, term);
#pragma unroll
          for (int k = 0; k < T; ++k) {
            const int n0 = k * NR + r, n1 = k * NR + r1;
            pbyte[(n0 >> 3) * 1024 + (n0 & 7) * 16] = (uint8_t)term[k];
            if (r1 > r) pbyte[(n1 >> 3) * 1024 + (n1 & 7) * 16] = (uint8_t)(term[k] >> 8);
          }
          lr[r] -= p0;  // what the terms do not hold
          if (r1 > r) lr[r1] -= p1;
        }
        fence_proxy_async_shared();
        tc_fence_before_sync();
        bar_wg(wg);
        const bool use0 = info.z >= 0.f, use1 = info.w >= 0.f;  // the blocks that were copied
        if (w4 == 0) {
          tc_fence_after_sync();
          const uint32_t ring_v = warp_uniform(smem_u32(ring + s * kStage + kTile * kD));
#pragma unroll
          for (int blk = 0; blk < 2; ++blk) {
            if (!(blk ? use1 : use0)) continue;
            const bool two = (KIND == kListed ? hi - (blk ? at.y : at.x) : n - blk * kQ8Block) > 32;  // K-steps of 32 tokens
#pragma unroll
            for (int st = 0; st < 2; ++st)
              if (issue && (st == 0 || two))
                tc_mma_f8(u_s + blk * kN, tc_sdesc_kmajor(ring_v + blk * kQ8Plane + st * 4096, 1024, 128),
                          tc_sdesc_kmajor(u_p + blk * 512 + 256 * st, 128, 1024), tc_idesc_f8(128, kN, 0, 1, 1, 0), st > 0);
          }
          if (issue) {
            tc_commit(smem_u32(&sm.empty[s]));
            tc_commit(smem_u32(&sm.bar_o[wg]));
          }
          __syncwarp();
        }
        wait(&sm.bar_o[wg], phase & 1);
        __syncwarp();
        tc_fence_after_sync();
        ++phase;
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
          if (!(blk ? use1 : use0)) continue;
          const float vs = blk ? info.w : info.z;
          float d[NR];
          tmem_term_sums<NR, T>(t_s + blk * kN + lanes, d);
#pragma unroll
          for (int r = 0; r < NR; ++r) o[r] = fmaf(d[r], vs, o[r]);
        }
        tc_fence_before_sync();
        bar_wg(wg);  // the next scores take the place of these sums
      }

      // ---- join the four warpgroups (thread = coordinate of O)
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float x = warp_sum(l[r]), y = warp_sum(lr[r]);
        if (lane == 0) sm.lw[wg][w4][r] = x, sm.lrw[wg][w4][r] = y;
      }
      if (wt == 0) {
#pragma unroll
        for (int r = 0; r < NR; ++r) sm.m[wg][r] = m[r];
      }
      bar_all();
      if (wt < NR) {
        sm.l[wg][wt] = sm.lw[wg][0][wt] + sm.lw[wg][1][wt] + sm.lw[wg][2][wt] + sm.lw[wg][3][wt];
        sm.lr[wg][wt] = sm.lrw[wg][0][wt] + sm.lrw[wg][1][wt] + sm.lrw[wg][2][wt] + sm.lrw[wg][3][wt];
      }
      float *mix = reinterpret_cast<float *>(pbuf);  // [kWg][NR][128]; every MMA that read the terms is done
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float top = fmaxf(fmaxf(sm.m[0][r], sm.m[1][r]), fmaxf(sm.m[2][r], sm.m[3][r]));
        const float f = m[r] == -INFINITY ? 0.f : ex2_approx(m[r] - top);
        mix[(wg * NR + r) * 128 + wt] = o[r] * f;
      }
      bar_all();
      const bool whole = t0 == 0 && end == g + cnt;
      // TEAM: where the ring was (no copy is under way, and the products that read it are done)
      float *part = TEAM ? reinterpret_cast<float *>(ring) : a.parts + ((long long)blockIdx.x * 2 + (t0 == 0 ? 1 : 0)) * kRows * kPartRow;
      int len, mm;
      seq_sizes<KIND>(a, b, &len, &mm, false);
#pragma unroll 1
      for (int r = wg; r < NR; r += kWg) {  // a warpgroup finishes every fourth row
        const float top = fmaxf(fmaxf(sm.m[0][r], sm.m[1][r]), fmaxf(sm.m[2][r], sm.m[3][r]));
        float x = mix[r * 128 + wt], sl = 0.f, slr = 0.f;
#pragma unroll
        for (int w = 0; w < kWg; ++w) {
          const float mw = sm.m[w][r], f = mw == -INFINITY ? 0.f : ex2_approx(mw - top);
          // a warpgroup without a maximum adds 0, or the NaN of a row whose query is not finite
          sl = fmaf(sm.l[w][r], mw == -INFINITY && sm.l[w][r] == 0.f ? 0.f : (mw == -INFINITY ? 1.f : f), sl);
          slr = fmaf(sm.lr[w][r], mw == -INFINITY && sm.lr[w][r] == 0.f ? 0.f : (mw == -INFINITY ? 1.f : f), slr);
          if (w) x += mix[(w * NR + r) * 128 + wt];
        }
        const int row = row0 + r, i = row / G;
        if (row >= row_end || i >= mm) continue;
        if (whole && (!TEAM || ranks == 1)) {
          const int hq = h * G + row % G;
          finish_row<KIND>(a, b, hq, i, wt, x, top, sl, slr, 15.f, prior_of<KIND, 1>(a, b, hq, i, wt));
        } else {
          part[r * kPartRow + wt] = x;
          if (wt == 0) {
            part[r * kPartRow + kD] = top;
            part[r * kPartRow + kD + 1] = sl;
            part[r * kPartRow + kD + 2] = slr;
          }
        }
      }
      if constexpr (TEAM) break;
      if (tid == 0 && end == g1) {
        // the CTA's last unit: if it goes on beyond this slice and began in it, the join starts here
        const long long stop = g - t0 + cnt;  // slices c with total c / slices < stop hold parts of it
        const int parts = t0 == 0 && stop > g1 ? (int)((stop * slices + total - 1) / total) - (int)blockIdx.x : 0;
        cuts[blockIdx.x] = Cut{b, unit_of(e), h, parts};
      }
      g = end;
    }
    if (!TEAM && tid == 0 && g0 >= g1) cuts[blockIdx.x] = Cut{0, 0, 0, 0};
  }
  if constexpr (TEAM) {
    if (ranks > 1 && total > 0) {  // the parts of a row: thread = coordinate, the ranks and their warpgroups take turns at the rows
      cg::cluster_group cl = cg::this_cluster();
      __syncwarp();  // a warp's lanes come to the barriers together
      cl.sync();
      int len, m, row0, row_end, list;
      unit_span<KIND>(a, team_x, kUnitRows, &row0, &row_end, &list);
      seq_sizes<KIND>(a, team_b, &len, &m, false);
#pragma unroll 1
      for (int r = rank + ranks * (warp >> 2); warp < kConsumers / 32 && r < NR; r += ranks * kWg) {
        const int row = row0 + r, i = row / G, d = tid & 127;
        if (row >= row_end || i >= m) continue;
        const int hq = team_h * G + row % G;
        const Prior<1> prior = prior_of<KIND, 1>(a, team_b, hq, i, d);
        float x[kMostRanks], mk[kMostRanks], lk[kMostRanks], lrk[kMostRanks], top = -INFINITY;
#pragma unroll
        for (int k = 0; k < kMostRanks; ++k) {
          const float *rec = cl.map_shared_rank(reinterpret_cast<float *>(ring), min(k, ranks - 1)) + r * kPartRow;
          x[k] = rec[d], mk[k] = rec[kD], lk[k] = rec[kD + 1], lrk[k] = rec[kD + 2];
        }
#pragma unroll
        for (int k = 0; k < kMostRanks; ++k) top = fmaxf(top, mk[k]);
        float o = 0.f, l = 0.f, lr = 0.f;
#pragma unroll
        for (int k = 0; k < kMostRanks; ++k) {
          if (k >= ranks) break;
          const float f = mk[k] == -INFINITY ? 1.f : ex2_approx(mk[k] - top);  // without a maximum: zeros (or NaN)
          o = fmaf(x[k], f, o), l = fmaf(lk[k], f, l), lr = fmaf(lrk[k], f, lr);
        }
        finish_row<KIND>(a, team_b, hq, i, d, o, top, l, lr, 15.f, prior);
      }
      __syncwarp();
      cl.sync();  // the others have read this CTA's parts
    }
  }
  if (*(volatile int *)&sm.bad) settle();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == kThreads / 32 - 1) tmem_dealloc(tmem, kWg * kCols);
}

// One CTA per (CTA of the main kernel, row): the parts of the unit that was cut there. Four groups of
// 128 threads (thread = coordinate) take every fourth part; its maximum, sums and O are joined in shared memory.
template <int KIND>
__global__ void __launch_bounds__(512) q8_join_kernel(const __grid_constant__ Q8AttnArgs a, int unit_rows, const Cut *cuts) {
  __shared__ float so[4][kD], sl[4], slr[4], stop[4];
  if constexpr (KIND != kWhole) pdl_trigger();
  pdl_wait();
  const Cut cut = cuts[blockIdx.x];
  const int r = blockIdx.y, G = a.group;
  int row, row_end, list;
  unit_span<KIND>(a, cut.rt, unit_rows, &row, &row_end, &list);
  row += r;
  if (cut.parts < 2 || row >= row_end) return;
  int len, m;
  seq_sizes<KIND>(a, cut.b, &len, &m, false);
  const int i = row / G;
  if (i >= m) return;
  const int d = threadIdx.x & 127, grp = threadIdx.x >> 7, hq = cut.h * G + row % G;
  const Prior<1> prior = prior_of<KIND, 1>(a, cut.b, hq, i, d);
  auto rec = [&](int p) {
    return a.parts + (((long long)blockIdx.x + p) * 2 + (p == 0 ? 1 : 0)) * kRows * kPartRow + r * kPartRow;
  };
  float top = -INFINITY;
  for (int p = grp; p < cut.parts; p += 4) top = fmaxf(top, rec(p)[kD]);
  if (d == 0) stop[grp] = top;
  __syncthreads();
  top = fmaxf(fmaxf(stop[0], stop[1]), fmaxf(stop[2], stop[3]));
  float o = 0.f, l = 0.f, lr = 0.f;
#pragma unroll 4
  for (int p = grp; p < cut.parts; p += 4) {
    const float *x = rec(p);
    const float f = x[kD] == -INFINITY ? 1.f : ex2_approx(x[kD] - top);  // without a maximum: zeros (or NaN)
    o = fmaf(x[d], f, o);
    l = fmaf(x[kD + 1], f, l);
    lr = fmaf(x[kD + 2], f, lr);
  }
  so[grp][d] = o;
  if (d == 0) sl[grp] = l, slr[grp] = lr;
  __syncthreads();
  if (grp) return;
  o = so[0][d] + so[1][d] + so[2][d] + so[3][d];
  l = sl[0] + sl[1] + sl[2] + sl[3];
  lr = slr[0] + slr[1] + slr[2] + slr[3];
  finish_row<KIND>(a, cut.b, hq, i, d, o, top, l, lr, 15.f, prior);
}

template <int NR, int T, int KIND>
int launch_rows(const Q8AttnArgs &a, Cut *cuts, int b0, int nb, int rt0, int rts, int num_sms, cudaStream_t st) {
  constexpr int smem = kStages * kStage + stacked_rows(NR, T) * 128 * (1 + kWg);
  if (!allow_shared<q8_attend_kernel<NR, T, KIND, false>>(smem)) return TQ_ERR_CUDA;
  if (launch_overlapped(true, q8_attend_kernel<NR, T, KIND, false>, dim3(num_sms), dim3(kThreads), smem, st, a, b0, nb, rt0, rts, cuts) != cudaSuccess)
    return TQ_ERR_CUDA;
  if (launch_overlapped(true, q8_join_kernel<KIND>, dim3(num_sms, NR), dim3(512), 0, st, a, rows_of(T), (const Cut *)cuts) != cudaSuccess)
    return TQ_ERR_CUDA;
  return TQ_OK;
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }
size_t few_bytes(int num_sms) { return round16((size_t)num_sms * sizeof(Cut)) + (size_t)num_sms * 2 * kRows * kPartRow * sizeof(float); }

template <int NR, int T, int KIND>
int launch_team_rows(const Q8AttnArgs &a, int units, int ranks, cudaStream_t st) {
  constexpr int smem = kStages * kStage + stacked_rows(NR, T) * 128 * (1 + kWg);
  if (!allow_shared<q8_attend_kernel<NR, T, KIND, true>>(smem)) return TQ_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.batch * units * a.heads_kv * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ranks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, q8_attend_kernel<NR, T, KIND, true>, a, 0, a.batch, 0, units, (Cut *)nullptr) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

// How many clusters of `ranks` CTAs the current device runs at once (their CTAs share a GPC): 15 of 8, 36 of 4, 76 of 2.
template <int KIND>
int clusters_of(int ranks) {
  constexpr int smem = kStages * kStage + stacked_rows(4, 4) * 128 * (1 + kWg);
  static std::atomic<int> known[64][4];  // plus 1
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || !allow_shared<q8_attend_kernel<4, 4, KIND, true>>(smem)) return 0;
  const int k = ranks == 8 ? 3 : ranks == 4 ? 2 : ranks == 2 ? 1 : 0;
  if (device < 64 && known[device][k].load(std::memory_order_relaxed)) return known[device][k].load(std::memory_order_relaxed) - 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr, cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, q8_attend_kernel<4, 4, KIND, true>, &cfg) != cudaSuccess) n = 0;
  if (device < 64) known[device][k].store(n + 1, std::memory_order_relaxed);
  return n;
}

// CTAs that a unit is given where there are few units, 0 where slices do better: one launch instead of two, and no table of entries, but a
// CTA may get up to a quarter and 8 more tiles than an even slice. `tiles` of a unit at most. 8 KV heads of 4 rows over 64 blocks 12.2 us in
// slices, 9.7 in clusters of 8; 8 sequences over 48 blocks 20.4 and 14.2 in clusters of 2.
template <int KIND>
int team_ranks(const Q8AttnArgs &a, long long units, long long tiles, int num_sms) {
  const long long n = a.batch * units * a.heads_kv;
  if (n > num_sms) return 0;
  int ranks = 1;
  for (int k = 8; k > 1 && ranks == 1; k /= 2)
    if (n * k <= num_sms && n <= clusters_of<KIND>(k)) ranks = k;
  return (tiles + ranks - 1) / ranks * 4 <= 5 * n * tiles / num_sms + 32 ? ranks : 0;
}

// What `tiles` tiles of a CTA cost, and a unit's end, in tenths of a microsecond: a round of one tile a warpgroup and the end of units
// of 4 rows 2.2 and 1.4, of 8 4.0 and 1.7, of 16 8.5 and 4.0 (8 KV heads of 16 rows over 64 blocks 19.1 us as one unit a head, 12.2 as four).
inline long long team_cost(int rows, long long tiles) {
  const long long rounds = (tiles + kWg - 1) / kWg;
  return rows <= 4 ? 22 * rounds + 14 : rows <= 8 ? 40 * rounds + 17 : 85 * rounds + 40;
}

// More rows than a unit's, 16-bit results: clusters of 16-row units take them where these are few and short, rather than the kernel for many
// rows, whose plan, start and join cost some 20 us and a tile of 256 rows 3.1 us of an SM. 8 KV heads: 40 rows over 16 blocks 17 us, 22 there, over 64
// blocks 25 and 34; 256 rows over 64 slots 12 us less than there; one head, 132 rows over 128 blocks 25 and 45.
template <int KIND>
bool team_takes(const Q8AttnArgs &a, long long rows, long long lists, long long tiles, int num_sms) {
  const int ranks = team_ranks<KIND>(a, (rows + 15) / 16 * lists, tiles, num_sms);
  const long long there = 200 + 31 * ((rows + 255) / 256 * lists * a.batch * a.heads_kv * tiles) / num_sms;
  return ranks && team_cost(16, (tiles + ranks - 1) / ranks) <= there;
}

// All rows of a call, a few at a time; `units` a sequence, `tiles` at most of each; `w`: few_bytes() of workspace.
template <int KIND>
int launch_few(Q8AttnArgs a, int rows, long long units, long long tiles, char *w, int num_sms, cudaStream_t st) {
  Cut *cuts = (Cut *)w;
  a.parts = (float *)(w + round16((size_t)num_sms * sizeof(Cut)));
  const int all = (int)units;
  if constexpr (KIND != kWhole) {
    const int ranks = team_ranks<KIND>(a, units, tiles, num_sms);
    if (rows > 4 && rows <= (a.out_dtype == TQ_F32 ? 8 : 16)) {  // or as units of 4 rows, which read the list's blocks again (from L2)
      const long long fours = units * ((rows + 3) / 4);
      const int four = team_ranks<KIND>(a, fours, tiles, num_sms);
      if (four && (!ranks || team_cost(4, (tiles + four - 1) / four) <= team_cost(rows, (tiles + ranks - 1) / ranks)))
        return a.out_dtype == TQ_F32 ? launch_team_rows<4, 8, KIND>(a, (int)fours, four, st) : launch_team_rows<4, 4, KIND>(a, (int)fours, four, st);
    }
    if (ranks) {
      if (a.out_dtype == TQ_F32)
        return rows == 1 ? launch_team_rows<1, 8, KIND>(a, all, ranks, st)
               : rows <= 4 ? launch_team_rows<4, 8, KIND>(a, all, ranks, st) : launch_team_rows<8, 8, KIND>(a, all, ranks, st);
      return rows == 1 ? launch_team_rows<1, 4, KIND>(a, all, ranks, st)
             : rows <= 4 ? launch_team_rows<4, 4, KIND>(a, all, ranks, st)
             : rows <= 8 ? launch_team_rows<8, 4, KIND>(a, all, ranks, st) : launch_team_rows<16, 4, KIND>(a, all, ranks, st);
    }
  }
  // (sequence, unit) pairs of a launch: as many as their table holds, and as keep the number of their tiles within 32 bits
  const int most = tiles * kEntries <= 0x7fffffff ? kEntries : (int)(0x7fffffff / tiles);
  const int per = all < most ? most / all : 1;
  for (int b0 = 0; b0 < a.batch; b0 += per)
    for (int rt0 = 0; rt0 < all; rt0 += most) {
      const int nb = a.batch - b0 < per ? a.batch - b0 : per, rts = all - rt0 < most ? all - rt0 : most;
      int s;
      if (a.out_dtype == TQ_F32)
        s = rows == 1 ? launch_rows<1, 8, KIND>(a, cuts, b0, nb, rt0, rts, num_sms, st)
            : rows <= 4 ? launch_rows<4, 8, KIND>(a, cuts, b0, nb, rt0, rts, num_sms, st)
                        : launch_rows<8, 8, KIND>(a, cuts, b0, nb, rt0, rts, num_sms, st);
      else
        s = rows == 1 ? launch_rows<1, 4, KIND>(a, cuts, b0, nb, rt0, rts, num_sms, st)
            : rows <= 4 ? launch_rows<4, 4, KIND>(a, cuts, b0, nb, rt0, rts, num_sms, st)
            : rows <= 8 ? launch_rows<8, 4, KIND>(a, cuts, b0, nb, rt0, rts, num_sms, st)
                        : launch_rows<16, 4, KIND>(a, cuts, b0, nb, rt0, rts, num_sms, st);
      if (s != TQ_OK) return s;
    }
  return TQ_OK;
}

}  // namespace
}  // namespace tq
