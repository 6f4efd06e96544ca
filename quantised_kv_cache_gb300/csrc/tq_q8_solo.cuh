// Attention over the 8-bit cache for few query rows per KV head and many units of work (listed blocks; a batch's own tokens behind a
// shared prefix): up to 4 rows, 16-bit results. The arithmetic of a tile is q8_attend_kernel's (tq_q8_few.cuh). There the four warpgroups
// of a CTA share a unit, and begin and finish it together: its queries' latency, the join of the warpgroups and the results' stores
// stand between two units, 5 to 10 us for 3 us a tile of work. Here every warpgroup has units of its own, with a ring, an operand of queries
// and a slice of the (sequence, list, head, tile) space of its own, so that one's beginning hides behind the others' tiles.
//
// Ring: three places of 16 KB for each warpgroup that its tiles' keys and values take in turn (keys of a tile, its values, keys of the next), so that
// the next tile's keys load while this one's values are used, in 192 KB. One producer warp a warpgroup. A tile's chain is some 3500 clocks, so that
// four at a time are faster than memory; 32 sequences of up to 16383 tokens over 128 blocks each, 4 rows, capped, paged: 66 us, 5.1 TB/s
// (the chosen blocks' 335 MB take 49): some 6 us until the first tile's scores, 5 of join, the rest the slices' unequal ends.
#pragma once

#include "tq_q8_few.cuh"

namespace tq {
namespace {

constexpr int kSoloThreads = kConsumers + 32 * kWg;
constexpr int kPlaces = 3, kPlace = kTile * kD;
constexpr int kSoloRows = 4;  // rows of a partial record
// What a unit's start and end cost, in tiles. 0, 1, 2 and 3 of them: 64 sequences over up to 47 blocks 53, 47, 46 and 46 us, 32 over 16 blocks each
// 24, 22, 23 and 23, 64 sequences' own tokens (1 to 2048) behind a short prefix 73, 68, 66 and 64.
constexpr int kSoloStart = 2;

struct SoloShared {
  uint64_t full[kWg][kPlaces], empty[kWg][kPlaces], bar_s[kWg], bar_o[kWg];
  float4 info[kWg][4];  // of a tile: key scales of its two blocks, value scales (negative: not mapped)
  int2 at[kWg][4];      // (kListed) their first slots
  float qscale[kWg][kSoloRows], slope[kWg][kSoloRows];
  int2 range[kWg][kSoloRows];
  int qpos[kWg][kSoloRows];
  float4 wmax[kWg][kSoloRows];          // row maxima of a warpgroup's four warps
  float4 lw[kWg][kSoloRows], lrw[kWg][kSoloRows];  // row sums of the warps
  uint32_t tmem;
  int bad, scan[kSoloThreads / 32], scan_starts[kSoloThreads / 32];
  Entries ent;
  int starts[kEntries + 1];  // entries with tiles before each
};

template <int NR, int KIND>
__global__ void __launch_bounds__(kSoloThreads, 1)
q8_solo_kernel(const __grid_constant__ Q8AttnArgs a, int b0, int nb, int rt0, int rts, Cut *cuts) {
  constexpr int T = 4, kN = stacked_rows(NR, T), kOp = kN * 128, kCols = 2 * kN;
  static_assert(NR <= kSoloRows && kWg * kCols <= 512 && kEntries <= kSoloThreads, "");
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ SoloShared sm;
  uint8_t *ring = dyn, *qbuf = dyn + kWg * kPlaces * kPlace, *pbuf = qbuf + kWg * kOp;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.group;

  if (tid == 0) {
    for (int w = 0; w < kWg; ++w) {
      for (int s = 0; s < kPlaces; ++s) mbar_init(&sm.full[w][s], 1), mbar_init(&sm.empty[w][s], 1);
      mbar_init(&sm.bar_s[w], 1), mbar_init(&sm.bar_o[w], 1);
    }
    mbar_fence_init();
    sm.bad = 0;
  }
  if (warp == kConsumers / 32) {
    tmem_alloc(smem_u32(&sm.tmem), kWg * kCols);
    tmem_relinquish();
  }
  pdl_trigger();  // the join waits for all of this grid, but its blocks may come as this one's leave
  pdl_wait();

  // ---- the entries' tiles: one thread each
  const int E = nb * rts;
  int count = 0;
  if (tid < E) {
    const int b = b0 + tid / rts;
    int len, m, r0, end, list;
    unit_span<KIND>(a, rt0 + tid % rts, NR, &r0, &end, &list);
    seq_sizes<KIND>(a, b, &len, &m, blockIdx.x == 0);
    const int i0 = r0 / G, i1 = (min(end, r0 + NR) - 1) / G;
    int lo = 0x7fffffff, hi = 0;
    for (int i = i0; i <= i1; ++i) {
      const int2 r = row_range<KIND>(a, b, i, len, m);
      if (r.y > r.x) lo = min(lo, r.x), hi = max(hi, r.y);
    }
    if (hi == 0) lo = 0;
    count = i0 < m ? max(1, unit_tiles<KIND>(a, b, lo, hi)) : 0;
    sm.ent.lo[tid] = lo;
    sm.ent.hi[tid] = hi;
  }
  {
    int x = count;
    const uint32_t some = __ballot_sync(kFull, count > 0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sm.scan[warp] = x, sm.scan_starts[warp] = __popc(some);
    __syncthreads();
    const int before = __reduce_add_sync(kFull, lane < warp ? sm.scan[lane] : 0);
    const int starts = __reduce_add_sync(kFull, lane < warp ? sm.scan_starts[lane] : 0) + __popc(some & (0xffffffffu >> (31 - lane)));
    if (tid < E) sm.ent.pre[tid + 1] = before + x, sm.starts[tid + 1] = starts;
    if (tid == 0) sm.ent.pre[0] = 0, sm.starts[0] = 0;
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sm.tmem;
  const int wg = warp < kConsumers / 32 ? warp >> 2 : warp - kConsumers / 32;
  // Slices are equal in tiles and starts, and none is empty (an interval of kSoloStart + 1 holds a tile).
  auto weight = [&](int e) { return ((long long)sm.ent.pre[e] + (long long)kSoloStart * sm.starts[e]) * a.heads_kv; };
  const long long total = weight(E);
  const int slice = blockIdx.x * kWg + wg;
  const long long slices = min((long long)gridDim.x * kWg, total / (kSoloStart + 1));
  const bool idle = slice >= slices;
  auto tile_at = [&](long long c) {  // the first tile of a slice that begins at weight c
    if (c >= total) return (long long)sm.ent.pre[E] * a.heads_kv;
    int lo = 0, hi = E - 1;
    while (lo < hi) {  // the last entry that begins at or before c
      const int mid = (lo + hi + 1) >> 1;
      if (weight(mid) <= c) lo = mid;
      else hi = mid - 1;
    }
    const int cnt = sm.ent.pre[lo + 1] - sm.ent.pre[lo], each = cnt + kSoloStart;
    const long long in = c - weight(lo), h = quotient(in, each);
    return (long long)sm.ent.pre[lo] * a.heads_kv + h * cnt + max(0, (int)(in - h * each) - kSoloStart);
  };
  const long long g0 = idle ? 0 : tile_at(quotient(total * slice, slices)), g1 = idle ? 0 : tile_at(quotient(total * (slice + 1), slices));
  auto locate = [&](long long g, int &e, int &h, int &t, int &cnt) {
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
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (*(volatile int *)&sm.bad) return;
    if (!mbar_wait_bounded(bar, parity, a.error)) *(volatile int *)&sm.bad = 1;
  };
  // place and phase of a warpgroup's load number k (a tile's keys, then its values)
  auto place = [](int k) { return k % kPlaces; };
  auto turn = [](int k) { return (uint32_t)(k / kPlaces) & 1; };

  if (warp >= kConsumers / 32) {
    // ================================ a warpgroup's producer: one lane finds the sources of one of the next 32 tiles
    uint8_t *const mine = ring + wg * kPlaces * kPlace;
    int it = 0;
    for (long long g = g0; g < g1; g += 32) {
      long long src[2] = {-1, -1};
      float4 info = make_float4(-1.f, -1.f, -1.f, -1.f);
      int bytes[2] = {0, 0}, at[2] = {0, 0};
      if (g + lane < g1) {
        int e, h, t, cnt, blk[2];
        locate(g + lane, e, h, t, cnt);
        const int lo = sm.ent.lo[e];
        const long long bh = (long long)(b0 + e / rts) * a.heads_kv + h;
        if constexpr (KIND == kListed) {
          int r0, end, list;
          unit_span<KIND>(a, rt0 + e % rts, NR, &r0, &end, &list);
          list_entries(a, bh, list, 2 * t, blk);
        } else {
          blk[0] = 2 * (lo / kTile + t), blk[1] = blk[0] + 1;
        }
        const int hi = sm.ent.hi[e];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          at[k] = max(blk[k], 0) * kQ8Block;
          const int m = min(kQ8Block, hi - at[k]);
          if (blk[k] < 0 || m <= 0 || at[k] + kQ8Block <= lo) continue;  // no row sees a token of it
          src[k] = q8_block(a.c.btab, a.c.pool_blocks, bh * a.c.nblk + blk[k], a.error);
          if (src[k] < 0) continue;
          bytes[k] = (m + 31) / 32 * 32 * kD;  // whole K-steps of the value MMA
          (k ? info.y : info.x) = latest(a.c.ks + src[k]);
          (k ? info.w : info.z) = latest(a.c.vs + src[k]);
        }
      }
      const int todo = (int)min(32ll, g1 - g);
      for (int k = 0; k < todo; ++k, ++it) {
        const long long s0 = __shfl_sync(kFull, src[0], k), s1 = __shfl_sync(kFull, src[1], k);
        const int n0 = __shfl_sync(kFull, bytes[0], k), n1 = __shfl_sync(kFull, bytes[1], k);
        const uint8_t *p0 = a.c.records + s0 * kQ8BlockBytes, *p1 = a.c.records + s1 * kQ8BlockBytes;
        uint64_t *fk = &sm.full[wg][place(2 * it)], *fv = &sm.full[wg][place(2 * it + 1)];
        if (lane == 0) {
          wait(&sm.empty[wg][place(2 * it)], turn(2 * it) ^ 1);
          if (!*(volatile int *)&sm.bad) {
            uint8_t *dst = mine + place(2 * it) * kPlace;
            if (n0) tma_load_1d(dst, p0, n0, fk);
            if (n1) tma_load_1d(dst + kQ8Plane, p1, n1, fk);
          }
        }
        __syncwarp();
        float4 f;  // (asked for after the copies: of a batch's first tile the scales are still on their way)
        f.x = __shfl_sync(kFull, info.x, k), f.y = __shfl_sync(kFull, info.y, k);
        f.z = __shfl_sync(kFull, info.z, k), f.w = __shfl_sync(kFull, info.w, k);
        int2 first = make_int2(0, 0);
        if constexpr (KIND == kListed) first.x = __shfl_sync(kFull, at[0], k), first.y = __shfl_sync(kFull, at[1], k);
        if (lane == 0) {
          if (!*(volatile int *)&sm.bad) {
            // the tile four before is done with: its values' place has been loaded twice since
            sm.info[wg][it & 3] = f;
            if constexpr (KIND == kListed) sm.at[wg][it & 3] = first;
            mbar_arrive_expect_tx(fk, n0 + n1);
          }
          wait(&sm.empty[wg][place(2 * it + 1)], turn(2 * it + 1) ^ 1);
          if (!*(volatile int *)&sm.bad) {
            uint8_t *dst = mine + place(2 * it + 1) * kPlace;
            mbar_arrive_expect_tx(fv, n0 + n1);
            if (n0) tma_load_1d(dst, p0 + kQ8Plane, n0, fv);
            if (n1) tma_load_1d(dst + kQ8Plane, p1 + kQ8Plane, n1, fv);
          }
        }
        __syncwarp();
      }
    }
    // every copy lands before the CTA's shared memory goes: the last fill of each place
    if (lane == 0) {
      for (int k = max(0, 2 * it - kPlaces); k < 2 * it; ++k)
        mbar_wait_bounded(&sm.full[wg][place(k)], turn(k), nullptr, kWaitBudgetNs / 8);
    }
    __syncwarp();
  } else {
    // ================================ a warpgroup
    const int wt = tid & 127, w4 = warp & 3;
    const uint32_t t_s = tmem + wg * kCols;
    const uint32_t lanes = (uint32_t)(32 * w4) << 16;
    uint8_t *const mine = ring + wg * kPlaces * kPlace, *const qmine = qbuf + wg * kOp, *const pmine = pbuf + wg * kOp;
    uint8_t *const pbyte = pmine + (wt >> 4) * 128 + (wt & 15);
    const bool issue = elect_lane();  // of the warpgroup's first warp
    const uint32_t u_s = warp_uniform(t_s), u_q = warp_uniform(smem_u32(qmine)), u_p = warp_uniform(smem_u32(pmine)),
                   u_ring = warp_uniform(smem_u32(mine));
    const Q8Score sc{a.scale, a.softcap, a.softcap != 0.f ? 1.f / a.softcap : 0.f};
    int it = 0;  // tiles so far
    long long g = g0;
    while (g < g1) {
      int e, h, t0, cnt;
      locate(g, e, h, t0, cnt);
      const int b = b0 + e / rts;
      int row0, row_end, list;
      unit_span<KIND>(a, rt0 + e % rts, NR, &row0, &row_end, &list);
      const long long end = min(g1, g - t0 + cnt);
      const int first = sm.ent.lo[e] / kTile, hi = sm.ent.hi[e];
      int len, m;
      seq_sizes<KIND>(a, b, &len, &m, false);

      // ---- the unit's queries: warp w prepares row w
      {
        const int row = row0 + w4, i = row / G, hq = h * G + row % G;
        const bool live = w4 < NR && row < row_end && i < m;
        // (asked for with the query: behind the barrier it would be one more wait)
        const int2 rg = live ? row_range<KIND>(a, b, i, len, m) : make_int2(0, 0);
        const float slope = live && a.slopes ? latest(a.slopes + hq) : 0.f;
        const int qpos = !live ? 0 : a.qpos ? latest(a.qpos + (long long)b * a.n_q + i) : query_slot<KIND>(a, i, len, m);
        uint32_t w[T];
        const int ex = row_e5m2<T, KIND>(a, b, hq, i, live, lane, w);
        bar_wg(wg);  // everyone is done with the unit before
        if (w4 < NR) {
#pragma unroll
          for (int k = 0; k < T; ++k) *reinterpret_cast<uint32_t *>(qmine + q8_off(k * NR + w4, 4 * lane)) = w[k];
          if (lane == 0) {
            sm.qscale[wg][w4] = pow2i(ex);
            sm.range[wg][w4] = rg;
            sm.slope[wg][w4] = slope * kLog2e;
            sm.qpos[wg][w4] = qpos;
          }
        }
        fence_proxy_async_shared();
        bar_wg(wg);
      }

      float mx[NR], l[NR], lr[NR], o[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) mx[r] = -INFINITY, l[r] = 0.f, lr[r] = 0.f, o[r] = 0.f;

      for (long long gt = g; gt < end; ++gt, ++it) {
        int tok0 = (first + t0 + (int)(gt - g)) * kTile, n = min(kTile, max(0, hi - tok0));  // (kListed: of the thread's block, below)
        const int pk = place(2 * it), pv = place(2 * it + 1);
        wait(&sm.full[wg][pk], turn(2 * it));
        if (w4 == 0) {
          __syncwarp();
          tc_fence_after_sync();
          const uint32_t u_k = warp_uniform(u_ring + pk * kPlace);
#pragma unroll
          for (int ks = 0; ks < kD / 32; ++ks)
            if (issue)
              tc_mma_f8(u_s, tc_sdesc_kmajor(u_k + 256 * ks, 128, 1024), tc_sdesc_kmajor(u_q + 256 * ks, 128, 1024),
                        tc_idesc_f8(128, kN, 0, 1, 0, 0), ks > 0);
          if (issue) tc_commit(smem_u32(&sm.bar_s[wg]));
          __syncwarp();
        }
        const float4 info = sm.info[wg][it & 3];
        const float ks = wt < kQ8Block ? info.x : info.y;
        int2 at = make_int2(0, 0);
        if constexpr (KIND == kListed) {  // the thread's block begins 64 threads before the second one's do
          at = sm.at[wg][it & 3];
          tok0 = wt < kQ8Block ? at.x : at.y - kQ8Block;
          n = (wt & kQ8Block) + (ks < 0.f ? 0 : min(kQ8Block, hi - tok0 - (wt & kQ8Block)));
        }
        const int slot = tok0 + wt;
        int kp = slot;
        if (a.kpos && slot < hi) kp = latest(a.kpos + ((long long)b * a.heads_kv + h) * a.c.capacity + slot);
        wait(&sm.bar_s[wg], it & 1);
        __syncwarp();  // the loads from tensor memory are a warp's
        tc_fence_after_sync();
        float t[NR];
        tmem_term_sums<NR, T>(t_s + lanes, t);
        // ---- scores, and the rows' maxima over the tile
        float most = -INFINITY;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const int2 rg = sm.range[wg][r];
          t[r] = q8_score_log2(t[r] * (sm.qscale[wg][r] * ks), sc);
          if (a.slopes) t[r] = fmaf(-sm.slope[wg][r], (float)__sad(sm.qpos[wg][r], kp, 0u), t[r]);
          if (slot < rg.x || slot >= rg.y || ks < 0.f) t[r] = -INFINITY;
          const float w = warp_fmax(t[r]);
          if (lane == r) most = w;
        }
        if (lane < NR) reinterpret_cast<float *>(&sm.wmax[wg][lane])[w4] = most;
        // value rows of the last K-step past the copied tokens hold whatever the cache holds there
        wait(&sm.full[wg][pv], turn(2 * it + 1));
        if (wt >= n && wt < ((n + 31) & ~31)) {
          uint8_t *row = mine + pv * kPlace + q8_off(wt, 0);
#pragma unroll
          for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(row + 128 * c) = make_uint4(0, 0, 0, 0);
        }
        bar_wg(wg);
        // The keys are used, and every warp has seen them arrive: a commit behind the products could give the place away, and let the barrier
        // complete a second time, before a warp that is late has looked at the first.
        if (wt == 0) mbar_arrive(&sm.empty[wg][pk]);
        // ---- probabilities (times 2^15), their terms, the sums
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float4 x = sm.wmax[wg][r];
          const float top = fmaxf(fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)), mx[r]);
          const float use = top == -INFINITY ? 0.f : top;
          const float corr = ex2_approx(mx[r] - use);
          mx[r] = top;
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
          const uint32_t u_v = warp_uniform(u_ring + pv * kPlace);
#pragma unroll
          for (int blk = 0; blk < 2; ++blk) {
            if (!(blk ? use1 : use0)) continue;
            const bool two = (KIND == kListed ? hi - (blk ? at.y : at.x) : n - blk * kQ8Block) > 32;  // K-steps of 32 tokens
#pragma unroll
            for (int st = 0; st < 2; ++st)
              if (issue && (st == 0 || two))
                tc_mma_f8(u_s + blk * kN, tc_sdesc_kmajor(u_v + blk * kQ8Plane + st * 4096, 1024, 128),
                          tc_sdesc_kmajor(u_p + blk * 512 + 256 * st, 128, 1024), tc_idesc_f8(128, kN, 0, 1, 1, 0), st > 0);
          }
          if (issue) {
            tc_commit(smem_u32(&sm.bar_o[wg]));
            tc_commit(smem_u32(&sm.empty[wg][pv]));
          }
          __syncwarp();
        }
        wait(&sm.bar_o[wg], it & 1);
        __syncwarp();
        tc_fence_after_sync();
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

      // ---- the rows' sums over the warps (thread = coordinate of O)
      const bool whole = t0 == 0 && end == g + cnt;
      Prior<1> prior[NR];  // of a row that is not there, another's
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const int row = min(row0 + r, row_end - 1), i = row / G;
        prior[r] = prior_of<KIND, 1>(a, b, h * G + row - i * G, i, wt);
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float x = warp_sum(l[r]), y = warp_sum(lr[r]);
        if (lane == 0) reinterpret_cast<float *>(&sm.lw[wg][r])[w4] = x, reinterpret_cast<float *>(&sm.lrw[wg][r])[w4] = y;
      }
      bar_wg(wg);
      float *part = a.parts + ((long long)slice * 2 + (t0 == 0 ? 1 : 0)) * kSoloRows * kPartRow;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float4 x = sm.lw[wg][r], y = sm.lrw[wg][r];
        const float sl = (x.x + x.y) + (x.z + x.w), slr = (y.x + y.y) + (y.z + y.w);
        const int row = row0 + r, i = row / G;
        if (row >= row_end || i >= m) continue;
        if (whole) {
          finish_row<KIND>(a, b, h * G + row % G, i, wt, o[r], mx[r], sl, slr, 15.f, prior[r]);
        } else {
          part[r * kPartRow + wt] = o[r];
          if (wt == 0) part[r * kPartRow + kD] = mx[r], part[r * kPartRow + kD + 1] = sl, part[r * kPartRow + kD + 2] = slr;
        }
      }
      if (wt == 0 && end == g1) {
        // the slice's last unit: if it goes on beyond it and began in it, the join starts here
        const long long stop = g - t0 + cnt;
        int parts = 0;
        if (t0 == 0 && stop > g1) {  // slices that begin before the unit's end, from this one on
          const long long last = weight(e) + (long long)(h + 1) * (cnt + kSoloStart);
          parts = (int)((last * slices + total - 1) / total) - slice;
        }
        cuts[slice] = Cut{b, rt0 + e % rts, h, parts};
      }
      g = end;
    }
    if (wt == 0 && g0 >= g1) cuts[slice] = Cut{0, 0, 0, 0};
  }
  if (*(volatile int *)&sm.bad) settle();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == kConsumers / 32) tmem_dealloc(tmem, kWg * kCols);
}

// One CTA per slice: the rows (128 threads each, thread = coordinate) of the unit that was cut there, its parts in their order.
template <int NR, int KIND>
__global__ void __launch_bounds__(128 * NR) q8_solo_join_kernel(const __grid_constant__ Q8AttnArgs a, const Cut *cuts) {
  pdl_trigger();
  pdl_wait();
  const Cut cut = cuts[blockIdx.x];
  const int d = threadIdx.x & 127, r = threadIdx.x >> 7, G = a.group;
  if (cut.parts < 2) return;
  int row, row_end, list, len, m;
  unit_span<KIND>(a, cut.rt, NR, &row, &row_end, &list);
  row += r;
  seq_sizes<KIND>(a, cut.b, &len, &m, false);
  const int i = row / G;
  if (row >= row_end || i >= m) return;
  const int hq = cut.h * G + row % G;
  const Prior<1> prior = prior_of<KIND, 1>(a, cut.b, hq, i, d);
  const float *rec = a.parts + ((long long)blockIdx.x * 2 + 1) * kSoloRows * kPartRow + r * kPartRow;  // the first part's; then two records a slice
  float top = -INFINITY, o = 0.f, l = 0.f, lr = 0.f;
  for (int p0 = 0; p0 < cut.parts; p0 += 4) {
    float m4[4], o4[4], l4[4], lr4[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int p = min(p0 + u, cut.parts - 1);
      const float *x = rec + (p ? (2ll * p - 1) * kSoloRows * kPartRow : 0);
      m4[u] = x[kD], o4[u] = x[d], l4[u] = x[kD + 1], lr4[u] = x[kD + 2];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (p0 + u >= cut.parts) break;
      const float now = fmaxf(top, m4[u]);
      // without a maximum: zeros (or NaN)
      const float was = top == -INFINITY ? 1.f : ex2_approx(top - now), f = m4[u] == -INFINITY ? 1.f : ex2_approx(m4[u] - now);
      o = fmaf(o4[u], f, o * was), l = fmaf(l4[u], f, l * was), lr = fmaf(lr4[u], f, lr * was);
      top = now;
    }
  }
  finish_row<KIND>(a, cut.b, hq, i, d, o, top, l, lr, 15.f, prior);
}

// Where there is a unit for every SM. 8 KV heads x 4 rows, here and in q8_attend_kernel: 32 sequences over 128 blocks 97 and 99 us (of up to
// 128: 69 and 91), over 16 blocks 23 and 28 us, 128 over 8 blocks 37 and 57 us; 8 sequences over 48 blocks 24 and 22 us, over 128 41 and 36; one
// over 64 27 and 16 us (its unit would lie in 76 slices).
bool solo_wins(const Q8AttnArgs &a, int lists, int num_sms) {
  const long long rows = (long long)a.group * (lists > 1 || a.span ? a.span : a.n_q);
  return a.out_dtype != TQ_F32 && rows <= kSoloRows && (long long)a.batch * a.heads_kv * lists >= num_sms;
}

size_t solo_bytes(int num_sms) {
  return round16((size_t)num_sms * kWg * sizeof(Cut)) + (size_t)num_sms * kWg * 2 * kSoloRows * kPartRow * sizeof(float);
}


template <int NR, int KIND>
int launch_solo_rows(const Q8AttnArgs &a, Cut *cuts, int b0, int nb, int rt0, int rts, int num_sms, cudaStream_t st) {
  constexpr int smem = kWg * (kPlaces * kPlace + 2 * stacked_rows(NR, 4) * 128);
  if (!allow_shared<q8_solo_kernel<NR, KIND>>(smem)) return TQ_ERR_CUDA;
  if (launch_overlapped(true, q8_solo_kernel<NR, KIND>, dim3(num_sms), dim3(kSoloThreads), smem, st, a, b0, nb, rt0, rts, cuts) != cudaSuccess)
    return TQ_ERR_CUDA;
  return launch_overlapped(true, q8_solo_join_kernel<NR, KIND>, dim3(num_sms * kWg), dim3(128 * NR), 0, st, a, (const Cut *)cuts) == cudaSuccess
             ? TQ_OK : TQ_ERR_CUDA;
}

// As launch_few, for 16-bit results and units of up to 4 rows; `w`: solo_bytes() of workspace.
template <int KIND>
int launch_solo(Q8AttnArgs a, int rows, long long units, long long tiles, char *w, int num_sms, cudaStream_t st) {
  Cut *cuts = (Cut *)w;
  a.parts = (float *)(w + round16((size_t)num_sms * kWg * sizeof(Cut)));
  const int all = (int)units;
  const int most = tiles * kEntries <= 0x7fffffff ? kEntries : (int)(0x7fffffff / tiles);
  const int per = all < most ? most / all : 1;
  for (int b0 = 0; b0 < a.batch; b0 += per)
    for (int rt0 = 0; rt0 < all; rt0 += most) {
      const int nb = a.batch - b0 < per ? a.batch - b0 : per, rts = all - rt0 < most ? all - rt0 : most;
      const int s = rows == 1 ? launch_solo_rows<1, KIND>(a, cuts, b0, nb, rt0, rts, num_sms, st)
                              : launch_solo_rows<4, KIND>(a, cuts, b0, nb, rt0, rts, num_sms, st);
      if (s != TQ_OK) return s;
    }
  return TQ_OK;
}

}  // namespace
}  // namespace tq
