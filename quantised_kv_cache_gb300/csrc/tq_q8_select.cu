// The choice of blocks that query tokens are to look at (tq_q8_select): per (sequence, KV head, `span` query tokens) the first
// and last blocks that the tokens see and those of the largest scores, in order.
//
// Mathematics. The list's rows become whole numbers within +-127 on one power of two, w = round(q 2^-x). With w+ and w- their
// positive and negative parts, a row's score of a block is S = sum w+ hi + w- lo: two chains of byte products with 32-bit whole sums, |S| < 2^21.
// The block's score max S 2^e has 21 significant bits whatever e: the products, sums and comparisons are exact and the choice does
// not depend on any order. Scores map to unsigned numbers of the same order; the last one that is taken is found bit by bit from the first in
// which any two differ, counting how many are not below a guess; ties go to the lowest blocks.
//
// Split: a list has a cluster of 1 to 8 CTAs, each with a run of blocks, that write their scores into the first one's shared memory; that one
// chooses. 16 lanes share a block (8 coordinates each: whole 128-byte lines), up to 16 rows' words stay in registers, and the rows' sums are
// added over the lanes in halves that change places. Bound by latency for few lists (the queries, then bounds, a cluster barrier, the search).

#include <cooperative_groups.h>

#include <algorithm>

#include "tq_q8_rows.cuh"
#include "tq_q8_select.cuh"

namespace cg = cooperative_groups;

namespace tq {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kHeld = 32768;               // scores kept in shared memory (128 KB): 2 M tokens
constexpr int kOwn = 8;                    // scores a thread of the choosing CTA keeps in registers
// Rows up to which a list's scores are formed here, by products of bytes; more go to the tensor cores.
constexpr long long kFewRows = 16;
constexpr int kNone = -0x7fffffff - 1;

struct Shared {
  uint32_t plus[16][kD / 4], minus[16][kD / 4];  // of 16 rows: w+ and w-, four coordinates a word
  uint32_t amax[kWarps];
  int lo[kWarps], hi[kWarps], count[2][kWarps];
  uint32_t rows;  // which of the 16 count
};

// exclusive prefix sum over the CTA
__device__ __forceinline__ int block_scan(int v, int *warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the sums of the scan before have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += warp_sums[w];
  return before + x - v;
}

// `keep` of the n > keep scores, in order, as block numbers from `first` on. A thread has `per` neighbouring ones.
template <bool REGS>
__device__ __forceinline__ void choose(const uint32_t *keys, int n, int keep, int first, int32_t *out, Shared &sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + kThreads - 1) / kThreads, i0 = min(n, tid * per), i1 = min(n, i0 + per);
  uint32_t k[REGS ? kOwn : 1];
  if constexpr (REGS) {
#pragma unroll
    for (int u = 0; u < kOwn; ++u) k[u] = i0 + u < i1 ? keys[i0 + u] : 0u;
  }
  auto each = [&](auto f) {
    if constexpr (REGS) {
#pragma unroll
      for (int u = 0; u < kOwn; ++u) f(k[u], i0 + u < i1);
    } else {
      for (int i = i0; i < i1; ++i) f(keys[i], true);
    }
  };
  // the bits in which all scores agree
  uint32_t all = kAlways, any = 0u;
  each([&](uint32_t x, bool there) { all &= there ? x : kAlways, any |= there ? x : 0u; });
  all = __reduce_and_sync(kFull, all), any = __reduce_or_sync(kFull, any);
  if (lane == 0) sm.count[0][warp] = (int)all, sm.count[1][warp] = (int)any;
  __syncthreads();
  all = kAlways, any = 0u;
  for (int w = 0; w < kWarps; ++w) all &= (uint32_t)sm.count[0][w], any |= (uint32_t)sm.count[1][w];
  __syncthreads();
  const uint32_t differ = all ^ any;
  uint32_t least = differ ? all & ~((2u << (31 - __clz((int)differ))) - 1u) : all;  // (a shift by 32 leaves 0, less 1: all bits)
  int taken = n;  // scores >= least
  for (int bit = differ ? 31 - __clz((int)differ) : -1, turn = 0; bit >= 0 && taken > keep; --bit, turn ^= 1) {
    const uint32_t guess = least | (1u << bit);
    int c = 0;
    each([&](uint32_t x, bool there) { c += there && x >= guess ? 1 : 0; });
    c = __reduce_add_sync(kFull, c);
    if (lane == 0) sm.count[turn][warp] = c;
    __syncthreads();
    c = __reduce_add_sync(kFull, lane < kWarps ? sm.count[turn][lane] : 0);
    if (c >= keep) least = guess, taken = c;
  }
  int more = 0, ties = 0;
  each([&](uint32_t x, bool there) { more += there && x > least ? 1 : 0, ties += there && x == least ? 1 : 0; });
  // of `taken` scores all above `least` stay, and the lowest blocks of those equal to it
  __syncthreads();
  const int ties_before = block_scan(ties, sm.count[0]);
  int c = __reduce_add_sync(kFull, more);
  if (lane == 0) sm.count[1][warp] = c;
  __syncthreads();
  c = __reduce_add_sync(kFull, lane < kWarps ? sm.count[1][lane] : 0);
  int left = min(max(keep - c - ties_before, 0), ties);
  int at = block_scan(more + left, sm.count[0]);
  int i = i0;
  each([&](uint32_t x, bool there) {
    if (there && (x > least || (x == least && left > 0))) {
      if (x == least) --left;
      out[at++] = first + i;
    }
    ++i;
  });
}

// Sums of s[0 .. N) over the 16 lanes that differ in 2 O - 1: while there is more than one, a half of them stays here and the other goes to the
// lane O away. s[0] is the sum of number `at` then.
template <int N, int O>
__device__ __forceinline__ void lane_sums(int *s, int lane, int &at) {
  if constexpr (O > 0) {
    const bool up = lane & O;
    if constexpr (N > 1) {
#pragma unroll
      for (int r = 0; r < N / 2; ++r) {
        const int give = up ? s[r] : s[r + N / 2];
        s[r] = (up ? s[r + N / 2] : s[r]) + __shfl_xor_sync(kFull, give, O);
      }
      at += up ? N / 2 : 0;
      lane_sums<N / 2, O / 2>(s, lane, at);
    } else {
      s[0] += __shfl_xor_sync(kFull, s[0], O);
      lane_sums<1, O / 2>(s, lane, at);
    }
  }
}

// NR: 1, 4 or 16 rows at a time; 0: the scores are there (q8_scores_kernel)
template <int NR>
__global__ void __launch_bounds__(kThreads) q8_choose_kernel(const __grid_constant__ Q8SelectArgs a) {
  extern __shared__ __align__(16) uint32_t held[];
  __shared__ Shared sm;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ranks = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const long long list = blockIdx.x / ranks;  // [batch][heads_kv][lists]
  const long long bh = list / a.lists;
  const int l = (int)(list - bh * a.lists), b = (int)(bh / a.q.heads_kv), h = (int)(bh - (long long)b * a.q.heads_kv), G = a.q.group;
  if (ranks > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");  // the first CTA has begun: its shared memory may be written
  pdl_wait();
  int len, m;
  seq_sizes(a.q, b, &len, &m, h == 0 && l == 0 && rank == 0 && tid == 0);
  const int tok0 = l * a.span, tok1 = min(m, (int)min((long long)a.q.n_q, (long long)tok0 + a.span));
  int lo = 0x7fffffff, hi = 0;
  for (int i = tok0 + tid; i < tok1; i += kThreads) {
    const int2 r = row_range(a.q, b, i, len, m);
    if (r.y > r.x) lo = min(lo, r.x), hi = max(hi, r.y);
  }
  lo = __reduce_min_sync(kFull, lo), hi = __reduce_max_sync(kFull, hi);
  if constexpr (NR == 0) {
    if (lane == 0) sm.lo[warp] = lo, sm.hi[warp] = hi;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) lo = min(lo, sm.lo[w]), hi = max(hi, sm.hi[w]);
    const int first = hi > 0 ? lo / kQ8Block : 0, n = (hi + kQ8Block - 1) / kQ8Block - first;
    int32_t *out = a.blocks + list * a.keep;
    const uint32_t *keys = a.keys + list * a.keys_ld + first;
    if (n <= a.keep) {
      for (int i = tid; i < a.keep; i += kThreads) out[i] = i < n ? first + i : -1;
    } else if (n <= kThreads * kOwn) {
      choose<true>(keys, n, a.keep, first, out, sm);
    } else {
      choose<false>(keys, n, a.keep, first, out, sm);
    }
    return;
  } else {
  // ---- the rows' largest coordinate
  const int rows = max(0, tok1 - tok0) * G;
  auto row = [&](int r, float (&x)[4]) {  // a whole warp; whether it counts
    const int i = tok0 + r / G;
    bool live = r < rows;
    if (live) {
      const int2 rg = row_range(a.q, b, i, len, m);
      live = rg.y > rg.x;
    }
    row_coords(a.q, b, h * G + r % G, i, live, lane, x);
    const uint32_t top = row_top(x);
    return live && top < 0x7f800000u ? top : kAlways;
  };
  uint32_t amax = 0;
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  uint32_t mine = kAlways;  // of this warp's only row, where there are 16 at most
  for (int r = warp; r < rows; r += kWarps) {
    mine = row(r, x);
    if (mine != kAlways) amax = max(amax, mine);
  }
  if (lane == 0) sm.amax[warp] = amax, sm.lo[warp] = lo, sm.hi[warp] = hi;
  if (tid == 0) sm.rows = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) amax = max(amax, sm.amax[w]), lo = min(lo, sm.lo[w]), hi = max(hi, sm.hi[w]);
  const int first = hi > 0 ? lo / kQ8Block : 0, n = (hi + kQ8Block - 1) / kQ8Block - first;  // the blocks that are seen
  int32_t *out = a.blocks + list * a.keep;
  if (n <= a.keep) {
    if (rank == 0)
      for (int i = tid; i < a.keep; i += kThreads) out[i] = i < n ? first + i : -1;
    if (ranks > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    return;
  }
  // from tiny rows' (also below the normal numbers) 2^100-fold on, so that their power of two is a number itself
  const float lift = amax < 0x0d800000u ? pow2i(100) : 1.f;
  const float by = pow2i(-row_exponent(__float_as_uint(__uint_as_float(amax) * lift), 6));
  const bool big = n > kHeld;
  uint32_t *const far = a.keys + list * a.keys_ld;
  const int run = (n + ranks - 1) / ranks, s0 = min(n, rank * run), s1 = min(n, s0 + run);
  uint32_t *const own = big ? far + s0 : held;  // this CTA's scores before the last of several passes
  const long long blocks = bh * a.q.c.nblk + first;
  bool joined = false;
  for (int r0 = 0; r0 < rows; r0 += NR) {
    const bool last = r0 + NR >= rows;
    if (r0 || rows > kWarps) mine = warp < NR ? row(r0 + warp, x) : kAlways;
    if (warp < NR) {
      uint32_t p = 0, q = 0;
      const bool live = mine != kAlways;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int w = live ? min(max(__float2int_rn(x[k] * lift * by), -127), 127) : 0;
        p |= (uint32_t)max(w, 0) << (8 * k);
        q |= ((uint32_t)min(w, 0) & 0xffu) << (8 * k);
      }
      sm.plus[warp][lane] = p, sm.minus[warp][lane] = q;
      if (lane == 0 && live) atomicOr(&sm.rows, 1u << warp);
    }
    __syncthreads();
    const uint32_t which = sm.rows;
    const int part = lane & 15;
    uint2 wp[NR], wm[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      wp[r] = *reinterpret_cast<const uint2 *>(&sm.plus[r][2 * part]);
      wm[r] = *reinterpret_cast<const uint2 *>(&sm.minus[r][2 * part]);
    }
    if (last && ranks > 1) {
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
      joined = true;
    }
    uint32_t *const dest = big ? far + s0 : ranks > 1 ? cl.map_shared_rank(held, 0) + s0 : held;
    constexpr int U = 4;  // blocks of 16 lanes in flight
    for (int i0 = s0 + 2 * warp + (lane >> 4); i0 - (lane >> 4) < s1; i0 += 2 * kWarps * U) {
      uint2 low[U], high[U];
      float ks[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + 2 * kWarps * u;
        ks[u] = -1.f;
        low[u] = high[u] = make_uint2(0u, 0u);
        if (i < s1) {
          const long long at = q8_block(a.q.c.btab, a.q.c.pool_blocks, blocks + i, a.q.error);
          if (at >= 0) {
            const uint2 *src = reinterpret_cast<const uint2 *>(a.bounds + at * (2 * kD)) + part;
            low[u] = __ldg(src), high[u] = __ldg(src + kD / 8);
            ks[u] = __ldg(a.q.c.ks + at);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + 2 * kWarps * u;
        int s[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          int t = __dp4a((int)wp[r].x, (int)high[u].x, 0);
          t = __dp4a((int)wp[r].y, (int)high[u].y, t);
          t = __dp4a((int)wm[r].x, (int)low[u].x, t);
          s[r] = __dp4a((int)wm[r].y, (int)low[u].y, t);
        }
        int at = 0;
        lane_sums<NR, 8>(s, lane, at);
        int best = (which >> at) & 1u ? s[0] : kNone;
#pragma unroll
        for (int o = 8; o > (NR == 1 ? 8 : NR == 4 ? 2 : 0); o >>= 1) best = max(best, __shfl_xor_sync(kFull, best, o));
        if (part == 0 && i < s1) {
          if (r0) best = max(best, (int)own[i - s0]);
          if (!last) {
            own[i - s0] = (uint32_t)best;
          } else {
            const bool sure = i < a.sink || i >= n - a.recent;
            const float score = (best == kNone ? 0.f : (float)best) * (ks[u] * 1.9073486e-6f);  // 2^-19: within float32 whatever the scale
            dest[i - s0] = sure ? kAlways : ks[u] < 0.f ? 0u : score_key(score);
          }
        }
      }
    }
    __syncthreads();  // the rows' words are used, and in a later pass the scores read by others
    if (tid == 0) sm.rows = 0;
    if (!last) __syncthreads();
  }
  if (ranks > 1) {
    if (!joined) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    cl.sync();
  } else {
    __syncthreads();
  }
  if (rank) return;
  const uint32_t *keys = big ? far : held;
  if (n <= kThreads * kOwn) choose<true>(keys, n, a.keep, first, out, sm);
  else choose<false>(keys, n, a.keep, first, out, sm);
  }
}

template <int NR>
int launch(const Q8SelectArgs &a, int ranks, size_t smem, cudaStream_t st) {
  if (cudaFuncSetAttribute(q8_choose_kernel<NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeld * 4) != cudaSuccess) return TQ_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((long long)a.q.batch * a.q.heads_kv * a.lists * ranks));
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
  return cudaLaunchKernelEx(&cfg, q8_choose_kernel<NR>, a) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

long long lists_of(int n_q, int span) { return ((long long)n_q + span - 1) / span; }

}  // namespace

size_t q8_select_workspace(int batch, int heads_kv, int group, int n_q, int span, int max_len) {
  const size_t blocks = q8_blocks_of(max_len);
  return blocks <= kHeld && (long long)group * std::min(span, n_q) <= kFewRows ? 0 : (size_t)batch * heads_kv * lists_of(n_q, span) * blocks * sizeof(uint32_t);
}

bool q8_select_fits(const Q8SelectArgs &a) {
  return (long long)a.q.group * a.q.n_q <= 0x7fffffff - 1023 && (long long)a.q.batch * a.q.heads_kv <= 0x7fffffff / 8 / a.lists;
}

int launch_q8_select(const Q8SelectArgs &args, void *workspace, int num_sms, void *stream) {
  Q8SelectArgs a = args;
  const int blocks = q8_blocks_of(a.q.max_len);
  const long long lists = (long long)a.q.batch * a.q.heads_kv * a.lists, rows = (long long)a.q.group * std::min(a.span, a.q.n_q);
  if (blocks > kHeld || rows > kFewRows) a.keys = (uint32_t *)workspace, a.keys_ld = blocks;
  if (rows > kFewRows) {
    const int s = launch_q8_scores(a, num_sms, stream);
    return s != TQ_OK ? s : launch<0>(a, 1, 0, (cudaStream_t)stream);
  }
  int ranks = 1;
  while (ranks < 8 && lists * ranks * 2 <= num_sms && blocks >= 128 * ranks) ranks *= 2;
  const size_t smem = (size_t)std::min(blocks, kHeld) * sizeof(uint32_t);
  cudaStream_t st = (cudaStream_t)stream;
  return rows == 1 ? launch<1>(a, ranks, smem, st) : rows <= 4 ? launch<4>(a, ranks, smem, st) : launch<16>(a, ranks, smem, st);
}

}  // namespace tq
