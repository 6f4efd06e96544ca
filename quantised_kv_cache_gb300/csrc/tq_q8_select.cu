// The choice of blocks that query tokens are to look at (tq_q8_select): per (sequence, KV head, `span` query tokens) the first
// and last blocks that the tokens see and those of the largest scores, in order.
//
// Mathematics. The list's rows become whole numbers within +-127 on one power of two, w = round(q 2^-x). With w+ and w- their
// positive and negative parts, a row's score of a block is S = sum w+ hi + w- lo, a product over 256 whole numbers: exact in fp16, their
// products and sums (|S| < 2^21) in fp32. The block's score max S 2^e has 21 significant bits whatever e: the products, sums and comparisons
// are exact and the choice does not depend on any order. Scores map to unsigned numbers of the same order; the last one that is taken is found
// eight bits at a time from the first in which any two differ; ties go to the lowest blocks.
//
// Split: a list has a cluster of 1 to 8 CTAs, each with a run of blocks, that write their scores into the first one's shared memory; that one
// chooses. A warp forms the scores of 16 blocks and 8 or 16 rows with m16n8k16 products: so few rows would leave a tcgen05 tile empty, and bounds
// go from memory to the operand's registers as they lie (chains of four byte products in one instruction, dp4a, took 17 clocks each on
// a quarter of an SM: 6 of the 13 us). Lists of more rows: q8_scores_kernel. Bound by latency for few lists (lengths, bounds, a cluster barrier,
// the passes of the choice): 8 KV heads of 4 rows among 2048 blocks 9.0 us, 2.5 of them the launch; 384 lists among up to 512 blocks (7 MB of
// bounds) 11.8 us.

#include <cooperative_groups.h>

#include <algorithm>

#include "tq_q8_rows.cuh"
#include "tq_q8_select.cuh"

namespace cg = cooperative_groups;

namespace tq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kHeld = 32768;  // scores kept in shared memory (128 KB): 2 M tokens
// Rows up to which a list's scores are formed here, by m16n8k16 products; more go to q8_scores_kernel's of 128 x 256.
constexpr long long kFewRows = 16;
constexpr int kBins = 256;

struct Shared {
  // Rows 8 n .. 8 n + 7 as a product's second operand, a lane's part of each of its 16 steps: steps 0 .. 7 have w+, the others w-.
  alignas(16) uint2 rows8[2][16][32];
  uint32_t amax[kWarps];
  int lo[kWarps], hi[kWarps], more[kWarps], ties[kWarps];
  uint32_t all[kWarps], any[kWarps];
  uint32_t rows;       // which of the 16 count
  alignas(16) int hist[4][kBins];  // of every pass (read four at a time)
};

// All threads: the first and one past the last slot that a list's rows see. `span` of one token needs no exchange.
__device__ __forceinline__ void list_range(const Q8SelectArgs &a, int b, int len, int m, int tok0, int tok1, int *lo, int *hi, Shared &sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int first = 0x7fffffff, last = 0;
  if (a.span == 1) {
    const int2 r = row_range(a.q, b, tok0, len, m);  // (0, 0) for a token that is not there
    if (r.y > r.x) first = r.x, last = r.y;
  } else {
    for (int i = tok0 + (int)threadIdx.x; i < tok1; i += kThreads) {
      const int2 r = row_range(a.q, b, i, len, m);
      if (r.y > r.x) first = min(first, r.x), last = max(last, r.y);
    }
    first = __reduce_min_sync(kFull, first), last = __reduce_max_sync(kFull, last);
    if (lane == 0) sm.lo[warp] = first, sm.hi[warp] = last;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) first = min(first, sm.lo[w]), last = max(last, sm.hi[w]);
  }
  *lo = first, *hi = last;
}

// Of n > keep scores the first `sink`, the last `recent` and the largest others, `keep` in all, in order, as block numbers from `first` on.
// The digits of the last one taken are found from the highest bit in which scores differ, eight at a time, by counting (sm.hist is
// zeroed); every warp adds the counts up for itself.
__device__ __forceinline__ void choose(const uint32_t *keys, int n, int keep, int sink, int recent, int first, int32_t *out, Shared &sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int end = n - recent;
  int need = keep - sink - recent;  // of the scores from the sink to the recent ones
  uint32_t all = kAlways, any = 0u;
#pragma unroll 8
  for (int i = sink + tid; i < end; i += kThreads) all &= keys[i], any |= keys[i];
  all = __reduce_and_sync(kFull, all), any = __reduce_or_sync(kFull, any);
  if (lane == 0) sm.all[warp] = all, sm.any[warp] = any;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) all &= sm.all[w], any |= sm.any[w];
  // scores >= least are candidates; the bits of `known` are those of all candidates' fate so far
  const uint32_t differ = all ^ any;
  int top = differ ? 32 - __clz((int)differ) : 0;               // bits below are unknown
  uint32_t least = top < 32 ? all >> top << top : 0u;
  bool whole = need == 0 || top == 0;                            // nothing left to find
  for (int pass = 0; !whole; ++pass) {
    const int shift = max(0, top - 8);
    const uint32_t digits = (1u << (top - shift)) - 1u;
#pragma unroll 8
    for (int i = sink + tid; i < end; i += kThreads) {
      const uint32_t k = keys[i] ^ least;
      if (top == 32 || k >> top == 0u) atomicAdd(&sm.hist[pass][(k >> shift) & digits], 1);  // (bits of `least` below top are 0)
    }
    __syncthreads();
    // lane l: bins 255 - 8 l down to 248 - 8 l
    const int4 lo4 = *reinterpret_cast<const int4 *>(&sm.hist[pass][kBins - 8 - 8 * lane]);
    const int4 hi4 = *reinterpret_cast<const int4 *>(&sm.hist[pass][kBins - 4 - 8 * lane]);
    const int c[8] = {hi4.w, hi4.z, hi4.y, hi4.x, lo4.w, lo4.z, lo4.y, lo4.x};
    int mine = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) mine += c[u];
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, upto, o);
      if (lane >= o) upto += y;
    }
    const int who = __ffs(__ballot_sync(kFull, upto >= need)) - 1;  // the lane whose bins hold the last one taken
    int before = upto - mine, bin = 0, in = 0;
    bool found = false;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (!found && before + c[u] >= need) bin = kBins - 1 - 8 * lane - u, in = c[u], found = true;
      if (!found) before += c[u];
    }
    bin = __shfl_sync(kFull, bin, who), before = __shfl_sync(kFull, before, who), in = __shfl_sync(kFull, in, who);
    need -= before;                                              // of the `in` scores with these digits
    least |= (uint32_t)bin << shift;
    top = shift;
    whole = in == need || top == 0;
  }
  // Of the scores that agree with `least` above bit `top`: all of them if need is their number, else (top is 0) the lowest blocks.
  // A warp has a run of the blocks.
  const int run = (n + 32 * kWarps - 1) / (32 * kWarps) * 32, i0 = min(n, warp * run), i1 = min(n, i0 + run);
  auto above = [&](int i, uint32_t k) { return i < sink || i >= end || (top < 32 && (k >> top) > (least >> top)); };
  auto equal = [&](int i, uint32_t k) { return i >= sink && i < end && (top >= 32 || (k >> top) == (least >> top)); };
  int more = 0, ties = 0;
  for (int i = i0 + lane; i < i1; i += 32) {
    const uint32_t k = keys[i];
    more += above(i, k) ? 1 : 0, ties += equal(i, k) ? 1 : 0;
  }
  more = __reduce_add_sync(kFull, more), ties = __reduce_add_sync(kFull, ties);
  if (lane == 0) sm.more[warp] = more, sm.ties[warp] = ties;
  __syncthreads();
  int at = 0, left = need;
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < warp) {
      at += sm.more[w] + min(left, sm.ties[w]);
      left -= min(left, sm.ties[w]);
    }
  const uint32_t below = (1u << lane) - 1u;
  for (int base = i0; base < i1; base += 32) {
    const int i = base + lane;
    const uint32_t k = i < i1 ? keys[i] : 0u;
    const bool tie = i < i1 && equal(i, k);
    const uint32_t tied = __ballot_sync(kFull, tie);
    const bool stay = i < i1 && (above(i, k) || (tie && __popc(tied & below) < left));
    const uint32_t stays = __ballot_sync(kFull, stay);
    if (stay) out[at + __popc(stays & below)] = first + i;
    at += __popc(stays);
    left -= min(left, __popc(tied));
  }
}

// The lists whose scores are there (q8_scores_kernel).
__global__ void __launch_bounds__(kThreads) q8_choose_scored_kernel(const __grid_constant__ Q8SelectArgs a) {
  __shared__ Shared sm;
  const int tid = threadIdx.x;
  const long long list = blockIdx.x, bh = list / a.lists;
  const int l = (int)(list - bh * a.lists), b = (int)(bh / a.q.heads_kv);
  for (int i = tid; i < 4 * kBins; i += kThreads) sm.hist[0][i] = 0;
  pdl_trigger();
  pdl_wait();
  int len, m, lo, hi;
  seq_sizes(a.q, b, &len, &m, false);
  const int tok0 = l * a.span, tok1 = min(m, (int)min((long long)a.q.n_q, (long long)tok0 + a.span));
  list_range(a, b, len, m, tok0, tok1, &lo, &hi, sm);
  const int first = hi > 0 ? lo / kQ8Block : 0, n = (hi + kQ8Block - 1) / kQ8Block - first;
  int32_t *out = a.blocks + list * a.keep;
  if (n <= a.keep) {
    for (int i = tid; i < a.keep; i += kThreads) out[i] = i < n ? first + i : -1;
    return;
  }
  choose(a.keys + list * a.keys_ld + first, n, a.keep, a.sink, a.recent, first, out, sm);
}

// NT: 8 rows or 16 at a time
template <int NT>
__global__ void __launch_bounds__(kThreads, 2) q8_choose_kernel(const __grid_constant__ Q8SelectArgs a) {
  extern __shared__ __align__(16) uint32_t held[];
  __shared__ Shared sm;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ranks = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const long long list = blockIdx.x / ranks;  // [batch][heads_kv][lists]
  const long long bh = list / a.lists;
  const int l = (int)(list - bh * a.lists), b = (int)(bh / a.q.heads_kv), h = (int)(bh - (long long)b * a.q.heads_kv), G = a.q.group;
  // (to an aligned barrier a warp's lanes come together)
  if (ranks > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");  // the first CTA has begun: its shared memory may be written
  auto cluster_wait = [&] {
    __syncwarp();
    if (ranks > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  };
  for (int i = tid; i < 4 * kBins; i += kThreads) sm.hist[0][i] = 0;
  if (tid == 0) sm.rows = 0;
  pdl_trigger();
  pdl_wait();
  // ---- the rows and the lengths on their way at once: a warp has rows `warp` and, of 16, `warp` + 8
  const int tok0 = l * a.span;
  float x[NT][4];
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const int r = warp + 8 * u, i = tok0 + r / G;
    row_coords(a.q, b, h * G + r % G, i, i < min((long long)a.q.n_q, (long long)tok0 + a.span), lane, x[u]);
  }
  int len, m, lo, hi;
  seq_sizes(a.q, b, &len, &m, h == 0 && l == 0 && rank == 0 && tid == 0);
  const int tok1 = min(m, (int)min((long long)a.q.n_q, (long long)tok0 + a.span));
  list_range(a, b, len, m, tok0, tok1, &lo, &hi, sm);
  const int first = hi > 0 ? lo / kQ8Block : 0, n = (hi + kQ8Block - 1) / kQ8Block - first;  // the blocks that are seen
  int32_t *out = a.blocks + list * a.keep;
  if (n <= a.keep) {
    cluster_wait();  // before the loop, which the lanes of a warp leave at different turns
    if (rank == 0)
      for (int i = tid; i < a.keep; i += kThreads) out[i] = i < n ? first + i : -1;
    return;
  }
  // ---- a warp's next 16 blocks' bounds on their way: four lanes share a block, and the one 8 after it
  const int run = (n + ranks - 1) / ranks, s0 = min(n, rank * run), s1 = min(n, s0 + run), g = lane >> 2, part = lane & 3;
  const long long blocks = bh * a.q.c.nblk + first;
  uint4 v[2][2][2];  // of either block: hi, lo; columns `part` and `part` + 4 of 16 coordinates
  float ks[2];
  auto fetch = [&](int i0) {
    long long at[2];
    const int i = i0 + g;
    q8_two_blocks(a.q.c, {blocks + i, blocks + i + 8}, {i < s1, i + 8 < s1}, a.q.error, at);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint4 *src = reinterpret_cast<const uint4 *>(a.bounds + max(at[u], 0ll) * (2 * kD)) + part;
      ks[u] = -1.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[u][k >> 1][k & 1] = make_uint4(0, 0, 0, 0);
      if (at[u] < 0) continue;
      v[u][0][0] = latest(src + 8), v[u][0][1] = latest(src + 12), v[u][1][0] = latest(src), v[u][1][1] = latest(src + 4);
      ks[u] = latest(a.q.c.ks + at[u]);
    }
  };
  const int begin = s0 + 16 * warp;
  fetch(begin);
  // ---- the rows' largest coordinate, over those that count
  const int rows = max(0, tok1 - tok0) * G;
  bool live[NT];
  uint32_t amax = 0;
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const int r = warp + 8 * u;
    const uint32_t top = row_top(x[u]);
    live[u] = r < rows && top < 0x7f800000u;
    if (live[u]) {
      const int2 rg = row_range(a.q, b, tok0 + r / G, len, m);
      live[u] = rg.y > rg.x;
    }
    if (live[u]) amax = max(amax, top);
  }
  if (lane == 0) sm.amax[warp] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) amax = max(amax, sm.amax[w]);
  // from tiny rows' (also below the normal numbers) 2^100-fold on, so that their power of two is a number itself
  const float lift = amax < 0x0d800000u ? pow2i(100) : 1.f;
  const float by = pow2i(-row_exponent(__float_as_uint(__uint_as_float(amax) * lift), 6));
  const bool big = n > kHeld;
  uint32_t *const far = a.keys + list * a.keys_ld;
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const int r = warp + 8 * u;
    int w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = live[u] ? min(max(__float2int_rn(x[u][k] * lift * by), -127), 127) : 0;
    auto pair = [](int p, int q) {
      const __half2 y = __halves2half2(__int2half_rn(p), __int2half_rn(q));
      return *reinterpret_cast<const uint32_t *>(&y);
    };
    // coordinates 4 lane ..: of column lane / 4, step lane % 4 of that column's four
    const int step = (lane >> 4) * 4 + (lane & 3), at = 4 * warp + ((lane >> 2) & 3);
    sm.rows8[u][step][at] = make_uint2(pair(max(w[0], 0), max(w[1], 0)), pair(max(w[2], 0), max(w[3], 0)));
    sm.rows8[u][step + 8][at] = make_uint2(pair(min(w[0], 0), min(w[1], 0)), pair(min(w[2], 0), min(w[3], 0)));
    if (lane == 0 && live[u]) atomicOr(&sm.rows, 1u << r);
  }
  __syncthreads();
  const uint32_t which = sm.rows;
  cluster_wait();
  uint32_t *const dest = big ? far + s0 : ranks > 1 ? cl.map_shared_rank(held, 0) + s0 : held;
  for (int i0 = begin; i0 < s1; i0 += 16 * kWarps) {
    if (i0 != begin) fetch(i0);
    __syncwarp();  // the products are a warp's
    float d[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) d[t][0] = d[t][1] = d[t][2] = d[t][3] = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // hi, lo; either column
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 p0 = v[0][k >> 1][k & 1], p1 = v[1][k >> 1][k & 1];
        const uint2 a0 = bytes_h4(q == 0 ? p0.x : q == 1 ? p0.y : q == 2 ? p0.z : p0.w);
        const uint2 a1 = bytes_h4(q == 0 ? p1.x : q == 1 ? p1.y : q == 2 ? p1.z : p1.w);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint2 w = sm.rows8[t][4 * k + q][lane];
          mma_16816(d[t], a0.x, a1.x, a0.y, a1.y, w.x, w.y);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = i0 + g + 8 * u;
      float best = -INFINITY;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if ((which >> (8 * t + 2 * part + e)) & 1u) best = fmaxf(best, d[t][2 * u + e]);
      best = fmaxf(best, __shfl_xor_sync(kFull, best, 1));
      best = fmaxf(best, __shfl_xor_sync(kFull, best, 2));
      if (part == 0 && i < s1) {
        const float score = (best == -INFINITY ? 0.f : best) * (ks[u] * 1.9073486e-6f);  // 2^-19: within float32 whatever the scale
        dest[i - s0] = ks[u] < 0.f ? 0u : score_key(score);
      }
    }
  }
  __syncwarp();
  if (ranks > 1) cl.sync();
  else __syncthreads();
  if (rank) return;
  choose(big ? far : held, n, a.keep, a.sink, a.recent, first, out, sm);
}

template <int NT>
int launch(const Q8SelectArgs &a, int ranks, size_t smem, cudaStream_t st) {
  if (!allow_shared<q8_choose_kernel<NT>>(kHeld * 4)) return TQ_ERR_CUDA;
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
  return cudaLaunchKernelEx(&cfg, q8_choose_kernel<NT>, a) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
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
    if (s != TQ_OK) return s;
    return launch_overlapped(true, q8_choose_scored_kernel, dim3((unsigned)lists), dim3(kThreads), 0, (cudaStream_t)stream, a) == cudaSuccess
               ? TQ_OK : TQ_ERR_CUDA;
  }
  // Clusters of 2 and 4 up to two CTAs an SM, of 8 up to one. 64 lists among 1024 blocks 11.8 us in twos, 9.9 in fours; 128 among 512 10.9 alone,
  // 9.1 in twos; 32 among 1024 9.1 in fours, 10.2 in eights.
  int ranks = 1;
  while (ranks < 8 && lists * ranks * 2 <= (ranks < 4 ? 2 : 1) * num_sms && blocks >= 128 * ranks) ranks *= 2;
  const size_t smem = (size_t)std::min(blocks, kHeld) * sizeof(uint32_t);
  cudaStream_t st = (cudaStream_t)stream;
  return rows <= 8 ? launch<1>(a, ranks, smem, st) : launch<2>(a, ranks, smem, st);
}

}  // namespace tq
