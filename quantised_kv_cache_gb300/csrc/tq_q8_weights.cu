// Accumulated attention weight of the 8-bit cache (tq_q8_attention with d_weights): per slot the sum,
// over the group's heads and the sequence's query tokens, of p = 2^(t - lse), t and lse in log2. No atomics, one fixed
// order of the sum.
//
// q8_kept_kernel, few rows: the attention has kept its scores (4 bytes a row and token, beside the 256 of the cache that it reads);
// a thread adds up 4 tokens' probabilities over the rows. Bound by those scores' bytes.
// q8_weights_kernel, many rows: after the attention has left each row's lse, the scores are formed again from the keys alone: one CTA per 128
// tokens of a (sequence, KV head), its key tile read once. Four warpgroups take every fourth tile of query
// rows: queries as e5m2 terms, one score MMA chain, and because token = lane = thread, a
// thread adds its own token's probabilities over all rows in one register.
// Row tiles that see none of the tokens are skipped.

#include "tq_q8_rows.cuh"

namespace tq {
namespace {

constexpr int kTile = 128;
constexpr int kWg = 4;
constexpr int kThreads = kWg * 128;

constexpr int kRows = 16;                                 // rows at most
constexpr int rows_of(int T) { return T == 8 ? 8 : 16; }  // rows of a tile: 64 operand rows of terms
constexpr int kN = 64, kOp = kN * 128;

struct Shared {
  uint64_t full, bar_s[kWg];
  float qscale[kWg][kRows], slope[kWg][kRows], lse[kWg][kRows];
  int2 range[kWg][kRows];
  int qpos[kWg][kRows];
  float sum[kWg][kTile];
  uint32_t tmem;
  int bad;
};

template <int T>
__global__ void __launch_bounds__(kThreads) q8_weights_kernel(const __grid_constant__ Q8AttnArgs a) {
  constexpr int NR = rows_of(T);
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
    const long long blk = q8_block(a.c.btab, a.c.pool_blocks, bh * a.c.nblk + (tok0 + wt) / kQ8Block, a.error);
    if (blk >= 0) ks = __ldg(a.c.ks + blk);
  }
  if (tid == 0) {
    int bytes = 0;
    long long src[2] = {-1, -1};
    for (int k = 0; k < 2 && k * kQ8Block < n; ++k) {
      src[k] = q8_block(a.c.btab, a.c.pool_blocks, bh * a.c.nblk + tok0 / kQ8Block + k, a.error);
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
  const int kp = a.kpos && wt < n ? __ldg(a.kpos + at + wt) : slot;
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
        sm.slope[wg][r] = live && a.slopes ? __ldg(a.slopes + hq) * kLog2e : 0.f;
        sm.qpos[wg][r] = !live ? 0 : a.qpos ? __ldg(a.qpos + (long long)b * a.n_q + i) : len - m + i;
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

template <int T>
int launch(const Q8AttnArgs &a, int slots, cudaStream_t st) {
  constexpr int smem = kTile * kD + kWg * kOp;
  if (cudaFuncSetAttribute(q8_weights_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return TQ_ERR_CUDA;
  const dim3 grid((unsigned)((slots + kTile - 1) / kTile), (unsigned)a.heads_kv, (unsigned)a.batch);
  return launch_overlapped(true, q8_weights_kernel<T>, grid, dim3(kThreads), smem, st, a) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // namespace

int launch_q8_weights(const Q8AttnArgs &a, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  // in place only the tokens in use are touched
  const int slots = a.weights == a.weights_in ? a.max_len : a.c.capacity;
  if (a.heads_kv > 65535 || a.batch > 65535) return TQ_ERR_UNSUPPORTED;
  if (a.scores) {
    const dim3 grid((unsigned)((slots + 4LL * kKept - 1) / (4 * kKept)), (unsigned)a.heads_kv, (unsigned)a.batch);
    return launch_overlapped(true, q8_kept_kernel, grid, dim3(kKept), 0, st, a) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
  }
  return a.out_dtype == TQ_F32 ? launch<8>(a, slots, st) : launch<4>(a, slots, st);
}

}  // namespace tq
