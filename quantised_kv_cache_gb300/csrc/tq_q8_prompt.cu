// Attention over the 8-bit cache for many query rows per KV head (tq_q8_attention): prompts. Results of 16 bits.
//
// Here a row (query token, head of the group) is an accumulator lane: S = Q K^T for 128 rows x 128 tokens, keys as
// the K-major B operand and values as the MN-major B operand as they lie in the cache; the queries' 8-bit terms
// sit in shared memory for the whole unit, the probabilities' terms take the place of the scores they came from in tensor memory
// (A operand). Two row tiles of 128 share a CTA and its key / value ring; each has two
// threads a row, one for each 64-token block of a tile, and runs its own chain (scores, softmax, value
// sums), so that one tile's tensor work hides behind the other's exponentials. O stays in registers (64
// coordinates a thread), where the running maximum's corrections and the blocks' value scales multiply it.
//
// Bound by issue and the tensor cores: per 128 x 128 tile two products of TERMS passes (540 clocks a
// product and two passes) and about 7 instructions an element. TERMS = 2 for bf16 (8 significant bits of
// q and p, what a bf16 operand would hold), 3 for fp16 (11). A term costs half an instruction to make: the probabilities go
// through fp16 pairs, in which the differences to the terms are exact.
//
// Two blocks of a tile share one value sum, the smaller scale folded into its probabilities; where the scales are more than
// 2^4 apart that would cost precision, and the blocks' sums are formed one after the other.
// Work split: as in the kernel for few rows, equal slices of the (sequence, 256 rows, head, tile) space, cut units
// joined afterwards; a small kernel finds each unit's tiles first.

#include "tq_q8_rows.cuh"

namespace tq {
namespace {

constexpr int kTile = 128;
constexpr int kUnit = 256;             // rows of a unit: two row tiles
constexpr int kThreads = 512;
constexpr int kStage = 2 * kTile * kD;
constexpr int kQTerm = 128 * kD;       // one term of a row tile's queries
constexpr int kAhead = 64;             // tiles whose sources are looked up at once
constexpr int kPartRow = kD + 4;       // O, m, l, 2 pad
constexpr float kFold = 0.0625f;       // blocks' value scales within 2^4 share a sum

constexpr int stages_of(int terms) { return terms == 2 ? 4 : 3; }

struct Entry {
  int lo, hi;          // first tile, one past the last visible slot
  int maxbeg, minend;  // slots in [maxbeg, minend) are seen by every row that is written
};

struct Cut {
  int b, pair, h, parts;
};

struct Plan {
  int *pre;       // [entries + 1] tiles (of one head) before each entry
  Entry *entry;   // [entries]
  Cut *cuts;      // [CTAs]
  float *parts;   // [CTAs][2][kUnit][kPartRow]
  int entries, pairs;
};

// One warp per entry (sequence, 256 rows).
__global__ void __launch_bounds__(256) q8_entries_kernel(const __grid_constant__ Q8AttnArgs a, Plan p) {
  const int e = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (e >= p.entries) return;
  const int b = e / p.pairs, r0 = (e % p.pairs) * kUnit, G = a.group, R = G * a.n_q;
  int len, m;
  seq_sizes(a, b, &len, &m, lane == 0);
  const int i0 = r0 / G, i1 = min(m - 1, (min(R, r0 + kUnit) - 1) / G);
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
    p.entry[e] = Entry{lo / kTile, hi, maxbeg, minend};
    // rows that see nothing keep one tile, so that their zeros are written
    p.pre[e + 1] = i0 < m ? max(1, (hi + kTile - 1) / kTile - lo / kTile) : 0;
  }
}

// Prefix sum of the entries' tiles, one CTA.
__global__ void __launch_bounds__(1024) q8_prefix_kernel(Plan p) {
  __shared__ int warp_sum_[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int base = 0;
  if (tid == 0) p.pre[0] = 0;
  for (int e0 = 0; e0 < p.entries; e0 += 1024) {
    const int e = e0 + tid;
    int x = e < p.entries ? p.pre[e + 1] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum_[warp] = x;
    __syncthreads();
    int before = base, all = base;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += warp_sum_[w];
      all += warp_sum_[w];
    }
    if (e < p.entries) p.pre[e + 1] = before + x;
    base = all;
    __syncthreads();
  }
}

struct Shared {
  uint64_t full[4], empty[4], bar_s[2], bar_o[2];
  float4 info[kAhead];        // key scales of a tile's two blocks, value scales (negative: not there)
  long long src[kAhead][2];   // its blocks
  float top[2][2][128];       // [row tile][half]: row maxima, then sums
  uint32_t tmem;
  int bad;
};

__device__ __forceinline__ void bar_rt(int rt) { asm volatile("bar.sync %0, 256;" ::"r"(1 + rt) : "memory"); }

// D (TMEM) (+)= A (TMEM, four 8-bit K-elements per column) x B (shared); issued by one thread.
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

// cap tanh(x / cap) in log2 units with tanh = 1 - 2 / (1 + e^2x): off by a few 2^-24 of the cap
__device__ __forceinline__ float capped_log2(float x, const Q8Score &s) {
  if (s.softcap == 0.f) return x * kLog2e;
  const float y = fminf(fmaxf(x * s.inv_cap, -10.f), 10.f);
  const float e = ex2_approx(y * (2.f * kLog2e));
  return s.softcap * kLog2e * (1.f - __fdividef(2.f, 1.f + e));
}

template <int TERMS, bool EXTRA>
__global__ void __launch_bounds__(kThreads, 1)
q8_prompt_kernel(const __grid_constant__ Q8AttnArgs a, const __grid_constant__ Plan p) {
  constexpr int kStages = stages_of(TERMS);
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ Shared sm;
  uint8_t *ring = dyn, *qbuf = dyn + kStages * kStage;  // [row tile][term][128 x 128]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rt = tid >> 8, half = (tid >> 7) & 1, lrow = tid & 127, w4 = warp & 3;
  const int G = a.group, R = G * a.n_q;
  const bool leader = (tid & 255) == 0;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&sm.full[s], 1), mbar_init(&sm.empty[s], 2);
    for (int r = 0; r < 2; ++r) mbar_init(&sm.bar_s[r], 1), mbar_init(&sm.bar_o[r], 1);
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
  const uint32_t tmem = sm.tmem, t_s = tmem + rt * 256, t_o = t_s + 128;
  const uint32_t mine = ((uint32_t)(32 * w4) << 16);

  const long long total = (long long)p.pre[p.entries] * a.heads_kv;
  const long long slices = min((long long)gridDim.x, total);
  const bool idle = blockIdx.x >= slices;
  const long long g0 = idle ? 0 : total * blockIdx.x / slices, g1 = idle ? 0 : total * (blockIdx.x + 1) / slices;
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (*(volatile int *)&sm.bad) return;
    if (!mbar_wait_bounded(bar, parity, a.error)) *(volatile int *)&sm.bad = 1;
  };
  const uint32_t idesc_s[2] = {tc_idesc_f8(128, 128, 0, 0, 0, 0), tc_idesc_f8(128, 128, 1, 0, 0, 0)};
  const uint32_t idesc_o[2] = {tc_idesc_f8(128, 128, 0, 0, 0, 1), tc_idesc_f8(128, 128, 1, 0, 0, 1)};
  const Q8Score sc{a.scale, a.softcap, a.softcap != 0.f ? 1.f / a.softcap : 0.f};
  int it = 0;              // tiles done before the current chunk: stages and phases count on
  int filled = 0;          // tiles whose copies were issued (thread 0)
  uint32_t phase_s = 0, phase_o = 0;

  long long g = g0;
  while (g < g1) {
    // ---- the unit at g
    int e;
    {
      int lo = 0, hi = p.entries - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((long long)p.pre[mid] * a.heads_kv <= g) lo = mid;
        else hi = mid - 1;
      }
      e = lo;
    }
    const int cnt = p.pre[e + 1] - p.pre[e];
    const long long in = g - (long long)p.pre[e] * a.heads_kv;
    const int h = (int)(in / cnt), t0 = (int)(in - (long long)h * cnt);
    const int b = e / p.pairs, pair = e % p.pairs;
    const long long end = min(g1, g - t0 + cnt);
    const Entry en = p.entry[e];
    int len, m;
    seq_sizes(a, b, &len, &m, false);
    const long long bh = (long long)b * a.heads_kv + h;

    // ---- queries: a warp prepares 16 rows, their terms to shared memory, their powers of two kept for a moment there
    __syncthreads();
#pragma unroll 4
    for (int k = 0; k < 16; ++k) {
      const int r = warp * 16 + k, row = pair * kUnit + r, i = row / G;
      uint32_t w[1][3];
      const int ex = row_terms<1>(a, b, h * G + row % G, i, row < R && i < m, lane, w);
#pragma unroll
      for (int t = 0; t < TERMS; ++t)
        *reinterpret_cast<uint32_t *>(qbuf + ((r >> 7) * TERMS + t) * kQTerm + q8_off(r & 127, 4 * lane)) = w[0][t];
      if (lane == 0) sm.top[r >> 7][0][r & 127] = pow2i(ex);
    }
    fence_proxy_async_shared();
    __syncthreads();
    const float qs = sm.top[rt][0][lrow];
    const int row = pair * kUnit + rt * 128 + lrow, qi = row / G, hq = h * G + row % G;
    const bool live = row < R && qi < m;
    const int2 rg = live ? row_range(a, b, qi, len, m) : make_int2(0, 0);
    const float slope = EXTRA && live && a.slopes ? __ldg(a.slopes + hq) * kLog2e : 0.f;
    const int qp = !EXTRA || !live ? 0 : a.qpos ? __ldg(a.qpos + (long long)b * a.n_q + qi) : len - m + qi;

    float2 o[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = make_float2(0.f, 0.f);
    float mx = -INFINITY, l = 0.f;

    for (long long c0 = g; c0 < end; c0 += kAhead) {
      const int todo = (int)min((long long)kAhead, end - c0);
      const int tile0 = en.lo + t0 + (int)(c0 - g);
      __syncthreads();
      if (tid < todo) {  // the chunk's sources
        const int tok = (tile0 + tid) * kTile, n = min(kTile, max(0, en.hi - tok));
        float4 f = make_float4(-1.f, -1.f, -1.f, -1.f);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          long long blk = -1;
          if (n > k * kQ8Block) blk = q8_block(a.c.btab, a.c.pool_blocks, bh * a.c.nblk + tok / kQ8Block + k, a.error);
          if (blk >= 0) {
            (k ? f.y : f.x) = __ldg(a.c.ks + blk);
            (k ? f.w : f.z) = __ldg(a.c.vs + blk);
          }
          sm.src[tid][k] = blk;
        }
        sm.info[tid] = f;
      }
      __syncthreads();
      const int last = it + todo;
      auto fill = [&](int upto, bool block) {  // thread 0: issue the copies of tiles < upto (and beyond, while stages are free)
        while (filled < last) {
          const int s = filled % kStages;
          if (filled >= kStages) {
            const uint32_t par = ((filled / kStages) & 1) ^ 1;
            if (filled < upto && block) wait(&sm.empty[s], par);
            else if (!mbar_test_wait(&sm.empty[s], par)) return;
          }
          if (*(volatile int *)&sm.bad) return;
          const int k = filled - it, tok = (tile0 + k) * kTile, n = min(kTile, max(0, en.hi - tok));
          uint8_t *dst = ring + s * kStage;
          const long long b0 = sm.src[k][0], b1 = sm.src[k][1];
          const int n0 = b0 >= 0 ? (min(kQ8Block, n) + 31) / 32 * 32 * kD : 0;
          const int n1 = b1 >= 0 ? (n - kQ8Block + 31) / 32 * 32 * kD : 0;
          mbar_arrive_expect_tx(&sm.full[s], 2 * (n0 + n1));
          if (n0) {
            const uint8_t *q = a.c.records + b0 * kQ8BlockBytes;
            tma_load_1d(dst, q, n0, &sm.full[s]);
            tma_load_1d(dst + kTile * kD, q + kQ8Plane, n0, &sm.full[s]);
          }
          if (n1) {
            const uint8_t *q = a.c.records + b1 * kQ8BlockBytes;
            tma_load_1d(dst + kQ8Plane, q, n1, &sm.full[s]);
            tma_load_1d(dst + kTile * kD + kQ8Plane, q + kQ8Plane, n1, &sm.full[s]);
          }
          ++filled;
        }
      };
      auto scores = [&](int j) {  // a leader: S of tile j
        if (tid == 0) fill(j + 1, true);
        const int s = j % kStages;
        wait(&sm.full[s], (j / kStages) & 1);
        tc_fence_after_sync();
        const uint32_t kt = smem_u32(ring + s * kStage);
#pragma unroll
        for (int t = 0; t < TERMS; ++t) {
          const uint32_t q = smem_u32(qbuf + (rt * TERMS + t) * kQTerm);
#pragma unroll
          for (int k = 0; k < kD / 32; ++k)
            tc_mma_f8(t_s, tc_sdesc_kmajor(q + 256 * k, 128, 1024), tc_sdesc_kmajor(kt + 256 * k, 128, 1024),
                      idesc_s[t == 2], t > 0 || k > 0);
        }
        tc_commit(smem_u32(&sm.bar_s[rt]));
      };
      if (leader) scores(it);

      for (int j = it; j < last; ++j) {
        const int s = j % kStages, tok0 = (tile0 + j - it) * kTile, n = min(kTile, max(0, en.hi - tok0));
        const float4 f = sm.info[j - it];
        const float ks = half ? f.y : f.x;
        uint8_t *const vt = ring + s * kStage + kTile * kD;
        const bool masked = !(en.maxbeg <= tok0 && en.minend >= tok0 + kTile) || f.x < 0.f || f.y < 0.f;
        // bits of the 64 tokens of this half that the row sees
        int from = 0, to = 64;
        if (masked) {
          from = min(max(rg.x - tok0 - 64 * half, 0), 64), to = min(max(rg.y - tok0 - 64 * half, 0), 64);
          if (ks < 0.f) to = 0;
        }
        wait(&sm.bar_s[rt], phase_s & 1);
        ++phase_s;
        __syncwarp();
        tc_fence_after_sync();
        // never 0, so that an unseen score of -inf stays -inf (products so small make no difference)
        const float c = fmaxf(qs * fmaxf(ks, 0.f) * (EXTRA ? 1.f : a.scale * kLog2e), 1e-30f);
        // a score in log2 (EXTRA), or the raw product (the scaling is in c); MASK: unseen ones are -inf
        auto score = [&](float x, int i, auto mask) {
          if constexpr (EXTRA) {
            x = capped_log2(x * c * sc.scale, sc);
            if (a.slopes) {
              const int slot = tok0 + 64 * half + i;
              const int kp = a.kpos ? (slot < en.hi ? __ldg(a.kpos + bh * a.c.capacity + slot) : 0) : slot;
              x = fmaf(-slope, (float)__sad(qp, kp, 0u), x);
            }
          }
          if constexpr (decltype(mask)::value) x = i >= from && i < to ? x : -INFINITY;
          return x;
        };
        // ---- the row's maximum over this half
        float top = -INFINITY;
        auto maximum = [&](auto mask) {
          float top1 = -INFINITY;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float x[16];
            tmem_ld_cols<16>(t_s + mine + 64 * half + 16 * q, x);
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              top = fmaxf(top, fmaxf(score(x[i], 16 * q + i, mask), score(x[i + 1], 16 * q + i + 1, mask)));
              top1 = fmaxf(top1, fmaxf(score(x[i + 2], 16 * q + i + 2, mask), score(x[i + 3], 16 * q + i + 3, mask)));
            }
          }
          top = fmaxf(top, top1);
        };
        if (masked) maximum(std::true_type{});
        else maximum(std::false_type{});
        if constexpr (!EXTRA) top = top == -INFINITY ? top : top * c;
        sm.top[rt][half][lrow] = top;
        bar_rt(rt);
        top = fmaxf(fmaxf(top, sm.top[rt][half ^ 1][lrow]), mx);
        const float use = top == -INFINITY ? 0.f : top;
        const float corr = ex2_approx(mx - use);
        mx = top;
        // ---- the two blocks' value scales: folded into the probabilities, or two sums
        const float vs0 = f.z, vs1 = f.w, vmax = fmaxf(fmaxf(vs0, vs1), 0.f);
        const bool both = vs0 >= 0.f && vs1 >= 0.f, apart = both && fminf(vs0, vs1) < vmax * kFold;
        float fold = 1.f;
        if (both && !apart) fold = __int_as_float((127 << 23) + __float_as_int(half ? vs1 : vs0) - __float_as_int(vmax));
        const float shift = 8.f - use + (float)log2i(fold);
        // ---- probabilities times 2^8, their terms over the scores they come from, their sum
        float2 sum = make_float2(0.f, 0.f);
        auto probabilities = [&](auto mask) {
          const float2 c2 = make_float2(c, c), shift2 = make_float2(shift, shift);
          uint32_t held[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float x[16];
            tmem_ld_cols<16>(t_s + mine + 64 * half + 16 * q, x);
            uint32_t w[TERMS][4];
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              uint32_t t[TERMS][2];
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const int k = i + 2 * u;
                float2 y = make_float2(score(x[k], 16 * q + k, mask), score(x[k + 1], 16 * q + k + 1, mask));
                y = EXTRA ? __fadd2_rn(y, shift2) : __ffma2_rn(y, c2, shift2);
                y = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                sum = __fadd2_rn(sum, y);
                const __half2 hp = __floats2half2_rn(y.x, y.y);
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
            const uint32_t to = t_s + mine + 64 * half + 32 * (q >> 1) + 4 * (q & 1);
            tmem_st_x4(to, w[0]);
            tmem_st_x4(to + 8, w[1]);
            if constexpr (TERMS == 3) {
              if (q & 1) {
                tmem_st_x4(to + 12, held);
                tmem_st_x4(to + 16, w[2]);
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) held[i] = w[2][i];
              }
            }
          }
        };
        if (masked) probabilities(std::true_type{});
        else probabilities(std::false_type{});
        l = fmaf(l, corr, (sum.x + sum.y) / fold);
        // value rows past the copied tokens, up to a whole K-step, hold what the cache holds there
        if (n < kTile && (n & 31)) {
          const int t = n + (tid & 255);
          if (t < ((n + 31) & ~31)) {
#pragma unroll
            for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4 *>(vt + q8_off(t, 16 * k)) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_shared();
        }
        tmem_st_wait();
        auto values = [&](int from_step, int to_step) {  // a leader: D = P V over the K-steps
          bool first = true;
#pragma unroll
          for (int t = 0; t < TERMS; ++t)
            for (int k = from_step; k < to_step; ++k) {
              if (k * 32 >= n || (k < 2 ? vs0 : vs1) < 0.f) continue;
              tc_mma_f8_ts(t_o, t_s + 32 * k + 8 * t, tc_sdesc_kmajor(smem_u32(vt) + 4096 * k, 1024, 128), idesc_o[t == 2],
                           !first);
              first = false;
            }
        };
        auto add = [&](float vs, float by) {  // O = O by + vs D
          const bool same = __all_sync(kFull, by == 1.f);
          const float2 v2 = make_float2(vs, vs), b2 = make_float2(by, by);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float d[16];
            tmem_ld_cols<16>(t_o + mine + 64 * half + 16 * q, d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float2 &y = o[8 * q + i];
              if (!same) y = __fmul2_rn(y, b2);
              y = __ffma2_rn(make_float2(d[2 * i], d[2 * i + 1]), v2, y);
            }
          }
        };
        tc_fence_before_sync();
        bar_rt(rt);
        const bool some = vs0 >= 0.f || vs1 >= 0.f;
        if (!apart) {
          if (leader) {
            tc_fence_after_sync();
            values(0, 4);
            tc_commit(smem_u32(&sm.empty[s]));
            tc_commit(smem_u32(&sm.bar_o[rt]));
            if (tid == 0) fill(0, false);
          }
          wait(&sm.bar_o[rt], phase_o & 1);
          ++phase_o;
          tc_fence_after_sync();
          if (leader && j + 1 < last) scores(j + 1);
          __syncwarp();
          if (some) add(vmax, corr);
          else
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __fmul2_rn(o[i], make_float2(corr, corr));
        } else {
          for (int k = 0; k < 2; ++k) {
            if (leader) {
              tc_fence_after_sync();
              values(2 * k, 2 * k + 2);
              if (k) tc_commit(smem_u32(&sm.empty[s]));
              tc_commit(smem_u32(&sm.bar_o[rt]));
            }
            wait(&sm.bar_o[rt], phase_o & 1);
            ++phase_o;
            __syncwarp();
            tc_fence_after_sync();
            add(k ? vs1 : vs0, k ? 1.f : corr);
            tc_fence_before_sync();
            bar_rt(rt);
          }
          if (leader && j + 1 < last) scores(j + 1);
          __syncwarp();
        }
        tc_fence_before_sync();
      }
      it = last;
    }

    // ---- the unit's rows
    sm.top[rt][half][lrow] = l;
    bar_rt(rt);
    l += sm.top[rt][half ^ 1][lrow];
    const bool whole = t0 == 0 && end == g + cnt;
    if (live) {
      if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const long long off = b * a.os.b + hq * a.os.h + qi * a.os.t + 64 * half;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          float y[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) y[2 * i] = o[4 * q + i].x * inv, y[2 * i + 1] = o[4 * q + i].y * inv;
          if (a.out_dtype == TQ_BF16) store_vec<__nv_bfloat16, 8>(static_cast<__nv_bfloat16 *>(a.out) + off + 8 * q, y);
          else store_vec<__half, 8>(static_cast<__half *>(a.out) + off + 8 * q, y);
        }
        if (a.lse && !half) a.lse[((long long)b * a.heads_q + hq) * a.n_q + qi] = (mx + log2f(l) - 8.f) * kLn2;
      } else {
        float *part = p.parts + (((long long)blockIdx.x * 2 + (t0 == 0 ? 1 : 0)) * kUnit + rt * 128 + lrow) * kPartRow;
#pragma unroll
        for (int q = 0; q < 16; ++q)
          reinterpret_cast<float4 *>(part + 64 * half)[q] = make_float4(o[2 * q].x, o[2 * q].y, o[2 * q + 1].x, o[2 * q + 1].y);
        if (!half) part[kD] = mx, part[kD + 1] = l;
      }
    }
    if (tid == 0 && end == g1) {
      const long long stop = g - t0 + cnt;
      int parts = 0;
      if (t0 == 0 && stop > g1) {
        parts = 1;
        for (long long k = blockIdx.x + 1; k < slices && total * k / slices < stop; ++k) ++parts;
      }
      p.cuts[blockIdx.x] = Cut{b, pair, h, parts};
    }
    g = end;
  }
  if (tid == 0 && idle) p.cuts[blockIdx.x] = Cut{0, 0, 0, 0};
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// The rows of a unit that was cut: one warp per row, lane = 4 coordinates.
__global__ void __launch_bounds__(256) q8_prompt_join_kernel(const __grid_constant__ Q8AttnArgs a, const __grid_constant__ Plan p) {
  const Cut cut = p.cuts[blockIdx.x];
  if (cut.parts < 2) return;
  const int lane = threadIdx.x & 31, r = blockIdx.y * 8 + (threadIdx.x >> 5), row = cut.pair * kUnit + r, G = a.group;
  int len, m;
  seq_sizes(a, cut.b, &len, &m, false);
  const int i = row / G;
  if (row >= G * a.n_q || i >= m) return;
  auto rec = [&](int k) {
    return p.parts + (((long long)blockIdx.x + k) * 2 + (k == 0 ? 1 : 0)) * kUnit * kPartRow + (long long)r * kPartRow;
  };
  float top = -INFINITY;
  for (int k = lane; k < cut.parts; k += 32) top = fmaxf(top, rec(k)[kD]);
  top = warp_max(top);
  float o[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
#pragma unroll 4
  for (int k = 0; k < cut.parts; ++k) {
    const float *x = rec(k);
    const float f = x[kD] == -INFINITY ? 1.f : ex2_approx(x[kD] - top);  // without a maximum: zeros (or NaN)
    const float4 y = reinterpret_cast<const float4 *>(x)[lane];
    o[0] = fmaf(y.x, f, o[0]), o[1] = fmaf(y.y, f, o[1]), o[2] = fmaf(y.z, f, o[2]), o[3] = fmaf(y.w, f, o[3]);
    l = fmaf(x[kD + 1], f, l);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] *= inv;
  const int hq = cut.h * G + row % G;
  const long long off = cut.b * a.os.b + hq * a.os.h + i * a.os.t + 4 * lane;
  if (a.out_dtype == TQ_BF16) store_vec<__nv_bfloat16, 4>(static_cast<__nv_bfloat16 *>(a.out) + off, o);
  else store_vec<__half, 4>(static_cast<__half *>(a.out) + off, o);
  if (a.lse && lane == 0) a.lse[((long long)cut.b * a.heads_q + hq) * a.n_q + i] = (top + log2f(l) - 8.f) * kLn2;
}

template <int TERMS, bool EXTRA>
int launch(const Q8AttnArgs &a, const Plan &p, int num_sms, cudaStream_t st) {
  constexpr int smem = stages_of(TERMS) * kStage + 2 * TERMS * kQTerm;
  if (cudaFuncSetAttribute(q8_prompt_kernel<TERMS, EXTRA>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return TQ_ERR_CUDA;
  q8_entries_kernel<<<(p.entries + 7) / 8, 256, 0, st>>>(a, p);
  q8_prefix_kernel<<<1, 1024, 0, st>>>(p);
  q8_prompt_kernel<TERMS, EXTRA><<<num_sms, kThreads, smem, st>>>(a, p);
  q8_prompt_join_kernel<<<dim3(num_sms, kUnit / 8), 256, 0, st>>>(a, p);
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

}  // namespace

size_t q8_prompt_workspace(int num_sms, int batch, int group, int n_q) {
  const size_t pairs = ((size_t)group * n_q + kUnit - 1) / kUnit, entries = pairs * batch;
  return round16((entries + 1) * sizeof(int)) + entries * sizeof(Entry) + (size_t)num_sms * sizeof(Cut) +
         (size_t)num_sms * 2 * kUnit * kPartRow * sizeof(float);
}

int launch_q8_prompt(const Q8AttnArgs &a, void *workspace, int num_sms, void *stream) {
  const long long pairs = ((long long)a.group * a.n_q + kUnit - 1) / kUnit, entries = pairs * a.batch;
  if (entries > 1 << 24) return TQ_ERR_UNSUPPORTED;
  Plan p;
  p.entries = (int)entries, p.pairs = (int)pairs;
  char *w = (char *)workspace;
  p.pre = (int *)w, w += round16((size_t)(entries + 1) * sizeof(int));
  p.entry = (Entry *)w, w += (size_t)entries * sizeof(Entry);
  p.cuts = (Cut *)w, w += (size_t)num_sms * sizeof(Cut);
  p.parts = (float *)w;
  cudaStream_t st = (cudaStream_t)stream;
  const bool extra = a.softcap != 0.f || a.slopes != nullptr || !(a.scale > 0.f);
  if (a.q_dtype == TQ_BF16)
    return extra ? launch<2, true>(a, p, num_sms, st) : launch<2, false>(a, p, num_sms, st);
  return extra ? launch<3, true>(a, p, num_sms, st) : launch<3, false>(a, p, num_sms, st);
}

}  // namespace tq
