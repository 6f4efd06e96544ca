// Accumulated attention weight of the 8-bit cache (tq_q8_attention with d_weights): per slot the sum,
// over the group's heads and the sequence's query tokens, of p = 2^(t - lse), t and lse in log2. No atomics, one fixed
// order of the sum.
//
// q8_kept_kernel: the attention for few rows has kept its scores (4 bytes a row and token, beside the 256 of the cache that it
// reads); a thread adds up 4 tokens' probabilities over the rows. Bound by those scores' bytes: 10 us for 6 rows of 4 x 16383 tokens and 8 heads.
// (Blocks without a place in the pool are reported by the attention, where a row sees them; here they are left out.)
// Else, after the attention has left each row's lse, the scores are formed again from the keys alone: token = accumulator lane =
// thread, which adds its own token's probabilities over all rows in registers.
// q8_weights_many_kernel, 16-bit results: a CTA holds the keys of 256 tokens; row tiles of 128 queries (their terms made once, by
// q8_row_tiles_kernel) pass through a ring, those that see none of the tokens left out. Two accumulators per token tile, so that
// the MMAs of one row tile (66 clocks each, 4 TERMS a tile) run under the exponentials of the other: bound by those, 1024 clocks for 128 x 128
// at 16 a clock. Where tokens alone give too few CTAs the row tiles are split, and the splits' sums added in order. Measured: 2048 query
// tokens over 8192, 32 query and 8 KV heads: 190 us beside the attention's 304, half the exponentials' rate; 16 sequences of 16384
// tokens and 64 rows: 300 us, a CTA's start for one row tile.
// q8_weights_kernel, 32-bit results: one CTA per 128 tokens, its key tile read once; four warpgroups take every fourth tile of 8
// rows: 8 e5m2 terms side by side, one score MMA chain. Row tiles that see none of the tokens are skipped. Measured: 128 query tokens of
// 2048, 32 query and 8 KV heads: 62 us beside the attention's 100.

#include "tq_q8_rows.cuh"

namespace tq {
namespace {

constexpr int kTile = 128;
constexpr int kWg = 4;
constexpr int kThreads = kWg * 128;

constexpr int T = 8, NR = 8;  // terms, rows of a tile: 64 operand rows
constexpr int kN = NR * T, kOp = kN * 128;

struct Shared {
  uint64_t full, bar_s[kWg];
  float qscale[kWg][NR], slope[kWg][NR], lse[kWg][NR];
  int2 range[kWg][NR];
  int qpos[kWg][NR];
  float sum[kWg][kTile];
  uint32_t tmem;
  int bad;
};

__global__ void __launch_bounds__(kThreads) q8_weights_kernel(const __grid_constant__ Q8AttnArgs a) {
  static_assert(stacked_rows(NR, T) == kN, "");
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ Shared sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2, wt = tid & 127, w4 = warp & 3;
  const int tok0 = blockIdx.x * kTile, h = blockIdx.y, b = blockIdx.z;
  int len, m;
  pdl_wait();
  seq_sizes(a, b, &len, &m, false);
  const int n = min(kTile, max(0, len - tok0));
  const long long bh = (long long)b * a.heads_kv + h, at = bh * a.c.capacity + tok0;
  if (n == 0) {  // no token here: the weights as they were
    if (a.weights != a.weights_in && tid < kTile && tok0 + tid < a.c.capacity)
      a.weights[at + tid] = a.weights_in ? a.weights_in[at + tid] : 0.f;
    return;
  }
  uint8_t *ktile = dyn, *qbuf = dyn + kTile * kD + wg * kOp;
  if (tid == 0) {
    mbar_init(&sm.full, 1);
    for (int w = 0; w < kWg; ++w) mbar_init(&sm.bar_s[w], 1);
    mbar_fence_init();
    sm.bad = 0;
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&sm.tmem), kWg * kN);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t t_s = sm.tmem + wg * kN, lanes = (uint32_t)(32 * w4) << 16;
  // the keys of the tile's two blocks; a block that is not mapped stays unread and unseen
  float ks = -1.f;
  if (wt < n) {
    const long long blk = q8_block(a.c.btab, a.c.pool_blocks, bh * a.c.nblk + (tok0 + wt) / kQ8Block, nullptr);
    if (blk >= 0) ks = latest(a.c.ks + blk);
  }
  if (tid == 0) {
    int bytes = 0;
    long long src[2] = {-1, -1};
    for (int k = 0; k < 2 && k * kQ8Block < n; ++k) {
      src[k] = q8_block(a.c.btab, a.c.pool_blocks, bh * a.c.nblk + tok0 / kQ8Block + k, nullptr);
      if (src[k] >= 0) bytes += kQ8Plane;
    }
    mbar_arrive_expect_tx(&sm.full, bytes);
    for (int k = 0; k < 2; ++k)
      if (src[k] >= 0) tma_load_1d(ktile + k * kQ8Plane, a.c.records + src[k] * kQ8BlockBytes, kQ8Plane, &sm.full);
  }
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (*(volatile int *)&sm.bad) return;
    if (!mbar_wait_bounded(bar, parity, a.error)) *(volatile int *)&sm.bad = 1;
  };
  wait(&sm.full, 0);
  const int slot = tok0 + wt;
  const int kp = a.kpos && wt < n ? latest(a.kpos + at + wt) : slot;
  const Q8Score sc{a.scale, a.softcap, a.softcap != 0.f ? 1.f / a.softcap : 0.f};
  const bool issue = elect_lane();  // of the warpgroup's first warp
  const uint32_t u_s = warp_uniform(t_s), u_k = smem_u32(ktile), u_q = warp_uniform(smem_u32(qbuf));
  const int R = a.group * a.n_q, rts = (R + NR - 1) / NR;
  float sum = 0.f;
  uint32_t phase = 0;
  for (int rt = wg; rt < rts; rt += kWg) {
    // ---- the ranges first: does any row of the tile see a token here?
    int2 rg = make_int2(0, 0);
    const int mine = rt * NR + (wt & (NR - 1)), mi = mine / a.group;
    if (mine < R) rg = row_range(a, b, mi, len, m);
    if (!__any_sync(kFull, rg.x < tok0 + n && rg.y > tok0)) continue;  // the same for the four warps
    if (wt < NR) sm.range[wg][wt] = rg;
    for (int k = 0; k < NR / 4; ++k) {
      const int r = w4 * (NR / 4) + k, row = rt * NR + r, i = row / a.group, hq = h * a.group + row % a.group;
      const bool live = row < R && i < m;
      uint32_t w[T];
      const int ex = row_e5m2<T>(a, b, hq, i, live, lane, w);
#pragma unroll
      for (int t = 0; t < T; ++t) *reinterpret_cast<uint32_t *>(qbuf + q8_off(t * NR + r, 4 * lane)) = w[t];
      if (lane == 0) {
        sm.qscale[wg][r] = pow2i(ex);
        sm.slope[wg][r] = live && a.slopes ? latest(a.slopes + hq) * kLog2e : 0.f;
        sm.qpos[wg][r] = !live ? 0 : a.qpos ? latest(a.qpos + (long long)b * a.n_q + i) : len - m + i;
        sm.lse[wg][r] = live ? a.lse[((long long)b * a.heads_q + hq) * a.n_q + i] * kLog2e : 0.f;
      }
    }
    fence_proxy_async_shared();
    tc_fence_before_sync();
    bar_wg(wg);
    if (w4 == 0) {
      tc_fence_after_sync();
#pragma unroll
      for (int s = 0; s < kD / 32; ++s)
        if (issue)
          tc_mma_f8(u_s, tc_sdesc_kmajor(u_k + 256 * s, 128, 1024), tc_sdesc_kmajor(u_q + 256 * s, 128, 1024),
                    tc_idesc_f8(128, kN, 0, 1, 0, 0), s > 0);
      if (issue) tc_commit(smem_u32(&sm.bar_s[wg]));
      __syncwarp();
    }
    wait(&sm.bar_s[wg], phase & 1);
    __syncwarp();
    ++phase;
    tc_fence_after_sync();
    float t[NR];
    tmem_term_sums<NR, T>(t_s + lanes, t);
    tc_fence_before_sync();
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int2 see = sm.range[wg][r];
      if (slot < see.x || slot >= see.y || ks < 0.f) continue;
      float x = q8_score_log2(t[r] * (sm.qscale[wg][r] * ks), sc);
      if (a.slopes) x = fmaf(-sm.slope[wg][r], (float)__sad(sm.qpos[wg][r], kp, 0u), x);
      sum += ex2_approx(x - sm.lse[wg][r]);
    }
    bar_wg(wg);  // the rows' arrays and terms are free again
  }
  sm.sum[wg][wt] = sum;
  if (*(volatile int *)&sm.bad) settle();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (tid < kTile && slot < a.c.capacity) {
    const float w = (sm.sum[0][wt] + sm.sum[1][wt]) + (sm.sum[2][wt] + sm.sum[3][wt]);
    a.weights[at + wt] = (a.weights_in ? a.weights_in[at + wt] : 0.f) + (wt < n ? w : 0.f);
  }
  if (warp == 0) tmem_dealloc(sm.tmem, kWg * kN);
}

// ---- many rows with results of 16 bits
constexpr int kTokens = 256;                    // tokens of a CTA: two accumulator tiles
constexpr int kSoft = 512, kManyThreads = kSoft + 64;  // then a warp that issues the MMAs and one that copies
constexpr int kTileRows = 128, kTerm = kTileRows * kD;
constexpr int kInfo = 3 * kTileRows * 8;        // a row tile's {scale, log-sum}, key ranges, {slope, position}
constexpr int tile_bytes(int terms) { return terms * kTerm + kInfo; }
constexpr int many_stages(int terms) { return terms == 2 ? 5 : 3; }

struct Many {
  uint8_t *tiles;  // [batch][heads_kv][row tiles] records of tile_bytes(TERMS): the terms as operand rows, then the rows' numbers
  int4 *see;       // [batch][heads_kv][row tiles]: rows see nothing outside [x, y), and all of [z, w)
  float *parts;    // [splits][batch][heads_kv][slots], or NULL: one CTA sums all rows of its tokens
  int rts, splits, slots;
};

// The query rows' terms and numbers, one CTA per 128 rows: made once here, read by every CTA of tokens that the rows see.
template <int TERMS>
__global__ void __launch_bounds__(256) q8_row_tiles_kernel(const __grid_constant__ Q8AttnArgs a, Many w) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ int see[4][4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rt = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int G = a.group, R = G * a.n_q;
  int len, m;
  pdl_wait();
  seq_sizes(a, b, &len, &m, false);
  float2 *cl = reinterpret_cast<float2 *>(dyn + TERMS * kTerm), *extra = cl + 2 * kTileRows;
  int2 *range = reinterpret_cast<int2 *>(cl + kTileRows);
#pragma unroll 1
  for (int k0 = 0; k0 < 16; k0 += 8) {
    uint2 raw[8];
    const int r0 = warp * 16 + k0;
    load_rows(a, b, h, m, rt * kTileRows + r0, lane, raw);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int row = rt * kTileRows + r0 + k;
      float x[4];
      row_floats(a, raw[k], row < R && row / G < m, x);
      uint32_t t[3];
      const int ex = row_terms(x, t);
#pragma unroll
      for (int j = 0; j < TERMS; ++j) *reinterpret_cast<uint32_t *>(dyn + j * kTerm + q8_off(r0 + k, 4 * lane)) = t[j];
      if (lane == 0) cl[r0 + k].x = pow2i(ex) * score_cap(a.scale, a.softcap).in;
    }
  }
  if (tid < kTileRows) {
    const int row = rt * kTileRows + tid, i = row / G, hq = h * G + row % G;
    const bool live = row < R && i < m;
    const int2 rg = live ? row_range(a, b, i, len, m) : make_int2(0, 0);
    const bool sees = rg.y > rg.x;
    range[tid] = rg;
    // a row that is not there weighs nothing wherever it looks
    cl[tid].y = live ? a.lse[((long long)b * a.heads_q + hq) * a.n_q + i] * kLog2e : INFINITY;
    extra[tid] = make_float2(live && a.slopes ? latest(a.slopes + hq) * kLog2e : 0.f,
                             __int_as_float(!live ? 0 : a.qpos ? latest(a.qpos + (long long)b * a.n_q + i) : len - m + i));
    const int lo = __reduce_min_sync(kFull, sees ? rg.x : 0x7fffffff), hi = __reduce_max_sync(kFull, sees ? rg.y : 0);
    const int maxbeg = __reduce_max_sync(kFull, live ? rg.x : 0), minend = __reduce_min_sync(kFull, live ? rg.y : 0x7fffffff);
    if (lane == 0) see[warp][0] = lo, see[warp][1] = hi, see[warp][2] = maxbeg, see[warp][3] = minend;
  }
  __syncthreads();
  const long long at = ((long long)b * a.heads_kv + h) * w.rts + rt;
  if (tid == 0)
    w.see[at] = make_int4(min(min(see[0][0], see[1][0]), min(see[2][0], see[3][0])), max(max(see[0][1], see[1][1]), max(see[2][1], see[3][1])),
                          max(max(see[0][2], see[1][2]), max(see[2][2], see[3][2])), min(min(see[0][3], see[1][3]), min(see[2][3], see[3][3])));
  uint4 *out = reinterpret_cast<uint4 *>(w.tiles + at * tile_bytes(TERMS));
  for (int i = tid; i < tile_bytes(TERMS) / 16; i += 256) out[i] = reinterpret_cast<const uint4 *>(dyn)[i];
}

struct ManyShared {
  uint64_t keys, full[5], empty[5], bar_s[2], freed[2];
  int4 see[5];  // a stage's rows (x < 0: no more)
  float sum[2][kTokens];
  uint32_t tmem;
  int bad;
};

template <int TERMS, int EXTRA>
__global__ void __launch_bounds__(kManyThreads, 1)
q8_weights_many_kernel(const __grid_constant__ Q8AttnArgs a, const __grid_constant__ Many w) {
  constexpr int kS = many_stages(TERMS), kBytes = tile_bytes(TERMS);
  extern __shared__ __align__(1024) uint8_t dyn[];  // the keys, then the ring of row tiles
  __shared__ ManyShared sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tok0 = blockIdx.x / w.splits * kTokens, split = blockIdx.x % w.splits, h = blockIdx.y, b = blockIdx.z;
  uint8_t *ring = dyn + kTokens * kD;
  int len, m;
  pdl_wait();
  seq_sizes(a, b, &len, &m, false);
  const int n = min(kTokens, max(0, len - tok0));
  const long long bh = (long long)b * a.heads_kv + h, at = bh * a.c.capacity + tok0;
  if (n == 0) {  // no token here: the weights as they were
    if (!w.parts && a.weights != a.weights_in && tid < kTokens && tok0 + tid < a.c.capacity)
      a.weights[at + tid] = a.weights_in ? a.weights_in[at + tid] : 0.f;
    return;
  }
  if (tid == 0) {
    mbar_init(&sm.keys, 1);
    for (int s = 0; s < kS; ++s) mbar_init(&sm.full[s], 1), mbar_init(&sm.empty[s], kSoft / 32);
    for (int k = 0; k < 2; ++k) mbar_init(&sm.bar_s[k], 1), mbar_init(&sm.freed[k], kSoft / 32);
    mbar_fence_init();
    sm.bad = 0;
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&sm.tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sm.tmem;
  auto wait = [&](uint64_t *bar, uint32_t parity) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i)
      if (mbar_try_wait(bar, parity)) return;
    if (*(volatile int *)&sm.bad) return;
    if (!mbar_wait_bounded(bar, parity, a.error)) *(volatile int *)&sm.bad = 1;
  };
  const int rt0 = (int)((long long)w.rts * split / w.splits), rt1 = (int)((long long)w.rts * (split + 1) / w.splits);

  if (warp == kSoft / 32 + 1) {
    // ================================ copies: the keys, then every row tile that sees a token of them
    long long src = -1;
    if (lane < kTokens / kQ8Block && lane * kQ8Block < n)
      src = q8_block(a.c.btab, a.c.pool_blocks, bh * a.c.nblk + tok0 / kQ8Block + lane, nullptr);
    const int planes = __popc(__ballot_sync(kFull, src >= 0));
    if (lane == 0) mbar_arrive_expect_tx(&sm.keys, planes * kQ8Plane);
    __syncwarp();
    if (src >= 0) tma_load_1d(dyn + lane * kQ8Plane, a.c.records + src * kQ8BlockBytes, kQ8Plane, &sm.keys);
    __syncwarp();
    int it = 0;
    for (int r0 = rt0; r0 < rt1; r0 += 32) {
      int4 see = make_int4(0, 0, 0, 0);
      if (r0 + lane < rt1) see = latest(w.see + bh * w.rts + r0 + lane);
      uint32_t some = __ballot_sync(kFull, see.x < tok0 + n && see.y > tok0);
      for (; some; some &= some - 1, ++it) {
        const int k = __ffs(some) - 1, s = it % kS;
        const int z = __shfl_sync(kFull, see.z, k), e = __shfl_sync(kFull, see.w, k);
        if (lane == 0) {
          wait(&sm.empty[s], ((it / kS) & 1) ^ 1);
          if (!*(volatile int *)&sm.bad) {
            sm.see[s] = make_int4(0, 0, z, e);
            mbar_arrive_expect_tx(&sm.full[s], kBytes);
            tma_load_1d(ring + s * kBytes, w.tiles + (bh * w.rts + r0 + k) * kBytes, kBytes, &sm.full[s]);
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0) {
      const int s = it % kS;
      wait(&sm.empty[s], ((it / kS) & 1) ^ 1);
      sm.see[s] = make_int4(-1, 0, 0, 0);
      mbar_arrive(&sm.full[s]);
      // every copy lands before the CTA's shared memory goes (the one in this stage has been used)
      mbar_wait_bounded(&sm.keys, 0, nullptr, kWaitBudgetNs / 8);
      for (int k = max(0, it - kS + 1); k < it; ++k) mbar_wait_bounded(&sm.full[k % kS], (k / kS) & 1, nullptr, kWaitBudgetNs / 8);
    }
    __syncwarp();
  } else if (warp == kSoft / 32) {
    // ================================ MMAs: both token tiles' products with a row tile
    const bool issue = elect_lane();
    const uint32_t u_d = warp_uniform(tmem), u_k = warp_uniform(smem_u32(dyn));
    wait(&sm.keys, 0);
    for (int it = 0;; ++it) {
      const int s = it % kS, buf = it & 1;
      wait(&sm.full[s], (it / kS) & 1);
      if (*(volatile int *)&sm.see[s].x < 0 || *(volatile int *)&sm.bad) break;
      wait(&sm.freed[buf], ((it >> 1) & 1) ^ 1);
      tc_fence_after_sync();
      const uint32_t q = warp_uniform(smem_u32(ring + s * kBytes));
      for (int tt = 0; tt * kTile < n; ++tt) {
#pragma unroll
        for (int t = 0; t < TERMS; ++t)
#pragma unroll
          for (int k = 0; k < kD / 32; ++k)
            if (issue)
              tc_mma_f8(u_d + (2 * buf + tt) * kTileRows, tc_sdesc_kmajor(u_k + tt * kTile * kD + 256 * k, 128, 1024),
                        tc_sdesc_kmajor(q + t * kTerm + 256 * k, 128, 1024), tc_idesc_f8(128, kTileRows, 0, t == 2, 0, 0), t > 0 || k > 0);
      }
      if (issue) tc_commit(smem_u32(&sm.bar_s[buf]));
      __syncwarp();
    }
    __syncwarp();
  } else {
    // ================================ probabilities: a token a thread, half of a row tile's rows a warpgroup
    const int tt = warp >> 3, half = (warp >> 2) & 1, tok = tt * kTile + (tid & 127), slot = tok0 + tok;
    float ks = -1.f;
    if (tok < n) {
      const long long blk = q8_block(a.c.btab, a.c.pool_blocks, bh * a.c.nblk + slot / kQ8Block, nullptr);
      if (blk >= 0) ks = latest(a.c.ks + blk);
    }
    const int kp = EXTRA && a.kpos && tok < n ? latest(a.kpos + at + tok) : slot;
    const float cap = score_cap(a.scale, a.softcap).cap;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const float k1 = fmaxf(ks, 0.f);
    float sum0 = 0.f, sum1 = 0.f;
    for (int it = 0;; ++it) {
      const int s = it % kS, buf = it & 1;
      wait(&sm.full[s], (it / kS) & 1);
      const int4 see = sm.see[s];
      if (see.x < 0 || *(volatile int *)&sm.bad) break;
      wait(&sm.bar_s[buf], (it >> 1) & 1);
      __syncwarp();
      tc_fence_after_sync();
      if (tt * kTile < n) {
        const uint32_t t_s = tmem + lanes + (2 * buf + tt) * kTileRows + 64 * half;
        const float2 *cl = reinterpret_cast<const float2 *>(ring + s * kBytes + TERMS * kTerm) + 64 * half;
        const int2 *range = reinterpret_cast<const int2 *>(cl + kTileRows);
        const float2 *extra = cl + 2 * kTileRows;
        auto add = [&](auto mask) {
          uint32_t v[2][16];
          tmem_ld_start(t_s, v[0]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            tmem_ld_done(v[q & 1]);
            if (q < 3) tmem_ld_start(t_s + 16 * (q + 1), v[(q + 1) & 1]);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const int r = 16 * q + i;
              const float4 c = *reinterpret_cast<const float4 *>(cl + r);
              float x0 = __uint_as_float(v[q & 1][i]), x1 = __uint_as_float(v[q & 1][i + 1]);
              if constexpr (EXTRA) {
                x0 = capped_log2<EXTRA == kLongCaps>(x0, c.x * k1, cap), x1 = capped_log2<EXTRA == kLongCaps>(x1, c.z * k1, cap);
                if (a.slopes) {
                  const float4 e = *reinterpret_cast<const float4 *>(extra + r);
                  x0 = fmaf(-e.x, (float)__sad(__float_as_int(e.y), kp, 0u), x0);
                  x1 = fmaf(-e.z, (float)__sad(__float_as_int(e.w), kp, 0u), x1);
                }
                x0 -= c.y, x1 -= c.w;
              } else {
                x0 = fmaf(x0, c.x * k1, -c.y), x1 = fmaf(x1, c.z * k1, -c.w);
              }
              if constexpr (decltype(mask)::value) {
                const int4 rg = *reinterpret_cast<const int4 *>(range + r);
                if (slot < rg.x || slot >= rg.y) x0 = -INFINITY;
                if (slot < rg.z || slot >= rg.w) x1 = -INFINITY;
              }
              sum0 += ex2_approx(x0), sum1 += ex2_approx(x1);
            }
          }
        };
        const int t0 = tok0 + tt * kTile;
        if (see.z <= t0 && see.w >= min(t0 + kTile, tok0 + n)) add(std::false_type{});
        else add(std::true_type{});
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.freed[buf]);
        mbar_arrive(&sm.empty[s]);
      }
    }
    sm.sum[half][tok] = ks < 0.f ? 0.f : sum0 + sum1;
  }
  if (*(volatile int *)&sm.bad) settle();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (tid < kTokens) {
    const float x = sm.sum[0][tid] + sm.sum[1][tid];
    if (w.parts) w.parts[((long long)split * gridDim.z * gridDim.y + bh) * w.slots + tok0 + tid] = x;
    else if (tok0 + tid < a.c.capacity) a.weights[at + tid] = (a.weights_in ? a.weights_in[at + tid] : 0.f) + (tid < n ? x : 0.f);
  }
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// The sums of the splits, in their order.
__global__ void __launch_bounds__(256) q8_weights_sum_kernel(const __grid_constant__ Q8AttnArgs a, const __grid_constant__ Many w) {
  const int slot = blockIdx.x * 256 + threadIdx.x, h = blockIdx.y, b = blockIdx.z;
  int len, m;
  pdl_wait();
  seq_sizes(a, b, &len, &m, false);
  const long long bh = (long long)b * a.heads_kv + h, at = bh * a.c.capacity + slot;
  if (slot >= a.c.capacity || (slot >= len && a.weights == a.weights_in)) return;
  float x = 0.f;
  if (slot < len)
    for (int k = 0; k < w.splits; ++k) x += w.parts[((long long)k * gridDim.z * gridDim.y + bh) * w.slots + slot];
  a.weights[at] = (a.weights_in ? a.weights_in[at] : 0.f) + x;
}

// Row tiles, splits and workspace for tokens up to max_len. Two CTAs an SM where at least four row tiles each remain. The sums of splits
// are fewer than 4 num_sms CTAs' (splits x CTAs < 2 num_sms + CTAs, and there are fewer than 2 num_sms CTAs to split): room for
// so many is counted whatever max_len is, so that a longer call's workspace serves a shorter one.
Many many_of(int num_sms, int batch, int heads_kv, int group, int n_q, int max_len, size_t *bytes) {
  Many w{};
  const long long rts = ((long long)group * n_q + kTileRows - 1) / kTileRows, bh = (long long)batch * heads_kv;
  const long long ctas = bh * ((max_len + kTokens - 1) / kTokens);
  long long splits = (2LL * num_sms + ctas - 1) / ctas;
  if (splits > (rts + 3) / 4) splits = (rts + 3) / 4;
  w.rts = (int)rts, w.splits = (int)splits, w.slots = (max_len + kTokens - 1) / kTokens * kTokens;
  *bytes = (size_t)bh * rts * (tile_bytes(3) + sizeof(int4)) + (rts > 4 ? 4 * (size_t)num_sms * kTokens * sizeof(float) : 0);
  return w;
}

template <int TERMS, int EXTRA>
int launch_many(const Q8AttnArgs &a, Many w, int slots, void *workspace, cudaStream_t st) {
  const size_t tiles = (size_t)a.batch * a.heads_kv * w.rts;
  char *p = (char *)workspace;
  w.tiles = (uint8_t *)p, p += tiles * tile_bytes(3);
  w.see = (int4 *)p, p += tiles * sizeof(int4);
  w.parts = w.splits > 1 ? (float *)p : nullptr;
  constexpr int smem = kTokens * kD + many_stages(TERMS) * tile_bytes(TERMS);
  if (cudaFuncSetAttribute(q8_row_tiles_kernel<TERMS>, cudaFuncAttributeMaxDynamicSharedMemorySize, tile_bytes(TERMS)) != cudaSuccess ||
      cudaFuncSetAttribute(q8_weights_many_kernel<TERMS, EXTRA>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return TQ_ERR_CUDA;
  const dim3 rows((unsigned)w.rts, (unsigned)a.heads_kv, (unsigned)a.batch);
  const int last = w.parts ? a.max_len : slots;
  const dim3 grid((unsigned)((long long)((last + kTokens - 1) / kTokens) * w.splits), (unsigned)a.heads_kv, (unsigned)a.batch);
  const dim3 sum((unsigned)((slots + 255) / 256), (unsigned)a.heads_kv, (unsigned)a.batch);
  cudaError_t e = launch_overlapped(true, q8_row_tiles_kernel<TERMS>, rows, dim3(256), tile_bytes(TERMS), st, a, w);
  if (e == cudaSuccess) e = launch_overlapped(true, q8_weights_many_kernel<TERMS, EXTRA>, grid, dim3(kManyThreads), smem, st, a, w);
  if (e == cudaSuccess && w.parts) e = launch_overlapped(true, q8_weights_sum_kernel, sum, dim3(256), 0, st, a, w);
  return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

constexpr int kKept = 128;  // threads of 4 tokens each

__global__ void __launch_bounds__(kKept) q8_kept_kernel(const __grid_constant__ Q8AttnArgs a) {
  __shared__ float lse[64];
  __shared__ int2 range[64];
  const int slot = (blockIdx.x * kKept + threadIdx.x) * 4, h = blockIdx.y, b = blockIdx.z, R = a.group * a.n_q;
  int len, m;
  pdl_wait();
  seq_sizes(a, b, &len, &m, false);
  const long long bh = (long long)b * a.heads_kv + h;
  if ((int)threadIdx.x < R) {  // R is at most 64
    const int i = threadIdx.x / a.group, hq = h * a.group + threadIdx.x % a.group;
    range[threadIdx.x] = row_range(a, b, i, len, m);
    lse[threadIdx.x] = i < m ? a.lse[((long long)b * a.heads_q + hq) * a.n_q + i] * kLog2e : 0.f;
  }
  __syncthreads();
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  if (slot < len) {
    const float *t = a.scores + bh * R * a.scores_ld + slot;
#pragma unroll 4
    for (int r = 0; r < R; ++r) {
      const int2 see = range[r];
      if (slot + 4 <= see.x || slot >= see.y) continue;
      const float4 x = *reinterpret_cast<const float4 *>(t + r * a.scores_ld);
      const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (slot + k >= see.x && slot + k < see.y && v[k] != -INFINITY) sum[k] += ex2_approx(v[k] - lse[r]);
    }
  }
  const long long at = bh * a.c.capacity + slot;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (slot + k < a.c.capacity && (slot + k < len || a.weights != a.weights_in))
      a.weights[at + k] = (a.weights_in ? a.weights_in[at + k] : 0.f) + sum[k];
}

int launch_wide(const Q8AttnArgs &a, int slots, cudaStream_t st) {
  constexpr int smem = kTile * kD + kWg * kOp;
  if (cudaFuncSetAttribute(q8_weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return TQ_ERR_CUDA;
  const dim3 grid((unsigned)((slots + kTile - 1) / kTile), (unsigned)a.heads_kv, (unsigned)a.batch);
  return launch_overlapped(true, q8_weights_kernel, grid, dim3(kThreads), smem, st, a) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // namespace

size_t q8_weights_workspace(int num_sms, int batch, int heads_kv, int group, int n_q, int max_len) {
  size_t bytes;
  many_of(num_sms, batch, heads_kv, group, n_q, max_len, &bytes);
  return bytes;
}

int launch_q8_weights(const Q8AttnArgs &a, int terms, void *workspace, int num_sms, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  // in place only the tokens in use are touched
  const int slots = a.weights == a.weights_in ? a.max_len : a.c.capacity;
  if (a.scores) {
    const dim3 grid((unsigned)((slots + 4LL * kKept - 1) / (4 * kKept)), (unsigned)a.heads_kv, (unsigned)a.batch);
    return launch_overlapped(true, q8_kept_kernel, grid, dim3(kKept), 0, st, a) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
  }
  if (a.out_dtype == TQ_F32) return launch_wide(a, slots, st);
  size_t bytes;
  const Many m = many_of(num_sms, a.batch, a.heads_kv, a.group, a.n_q, a.max_len, &bytes);
  const bool extra = a.softcap != 0.f || a.slopes != nullptr, far = a.softcap > kShortCap;
  if (terms == 2)
    return far     ? launch_many<2, kLongCaps>(a, m, slots, workspace, st)
           : extra ? launch_many<2, kCapOrBias>(a, m, slots, workspace, st)
                   : launch_many<2, kPlain>(a, m, slots, workspace, st);
  return far     ? launch_many<3, kLongCaps>(a, m, slots, workspace, st)
         : extra ? launch_many<3, kCapOrBias>(a, m, slots, workspace, st)
                 : launch_many<3, kPlain>(a, m, slots, workspace, st);
}

}  // namespace tq
