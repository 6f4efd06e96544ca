// Scores of blocks for lists of many rows (tq_q8_select), on the tensor cores.
//
// A row's score of a block is sum w+ hi + w- lo (tq_q8_select.cu): with the bounds of 128 blocks as the rows of one operand, [hi | lo],
// and up to 256 query rows as those of the other, [w+ | w-], it is one product over 256 numbers. Whole numbers up to 127
// are exact in fp16, their products in fp32, and every partial sum is a whole number below 2^21, so that the accumulators hold the scores
// exactly whatever the order. Blocks are accumulator lanes: a block's largest score over the rows is a maximum along its lane.
// Rows that do not count, and those that fill the operand up, are copies of one that does.
//
// Split: the (list, 128 blocks) space in slices, one CTA per SM, equal ones or of whole lists; a list's rows are converted once a slice and
// 256 rows, the next list's load behind this one's tiles, the next tile's bounds behind this one's product.
// 2048 tokens x 32 heads over 256 blocks, one list for 64 tokens: 21 us, and 6 for the choice. A CTA has one list or two, and each a chain of
// its rows' loads (3 us in the first), their largest, the conversions (1.6 us) and two tiles of 2 us, 1.1 of them the product; the products
// alone would take 5 us at the tensor cores' rate, with operands that were made beside them.

#include <algorithm>

#include "tq_q8_rows.cuh"
#include "tq_q8_select.cuh"

namespace tq {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kTileBlocks = 128, kTileRows = 256, kK = 2 * kD;
constexpr int kGroupBytes = kK / 8 * 128;                  // 8 rows of an operand: 32 columns of 8 numbers, 16 bytes each, a row after the other
constexpr int kABytes = kTileBlocks / 8 * kGroupBytes;     // 64 KB
constexpr int kBBytes = kTileRows / 8 * kGroupBytes;       // 128 KB

struct Shared {
  uint64_t bar;
  uint32_t amax[kWarps];
  int lo[kWarps], hi[kWarps], good[kWarps];
  float part[3][kTileBlocks];  // the maxima of all quarters of the columns but the first
  uint32_t tmem;
};

// D (TMEM) (+)= A (shared) x B (shared) of fp16 operands, 16 K-elements; executed by one lane.
__device__ __forceinline__ void tc_mma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// Eight numbers of a row as they lie.
template <typename T>
struct Eight {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) w[k] = latest(reinterpret_cast<const uint4 *>(p) + k);
  }
  // the largest magnitude's bits, as of a float32 (16-bit magnitudes have the order of their bits)
  __device__ __forceinline__ uint32_t top() const {
    if constexpr (sizeof(T) == 4) {
      uint32_t t = 0;
#pragma unroll
      for (int k = 0; k < 2; ++k) t = max(t, max(max(w[k].x & 0x7fffffffu, w[k].y & 0x7fffffffu), max(w[k].z & 0x7fffffffu, w[k].w & 0x7fffffffu)));
      return t;
    } else {
      const uint32_t t = __vmaxu2(__vmaxu2(w[0].x & 0x7fff7fffu, w[0].y & 0x7fff7fffu), __vmaxu2(w[0].z & 0x7fff7fffu, w[0].w & 0x7fff7fffu));
      const uint32_t h = max(t >> 16, t & 0xffffu);
      if constexpr (std::is_same<T, __nv_bfloat16>::value) return h << 16;
      else return h >= 0x7c00u ? 0x7f800000u : __float_as_uint(__half2float(__ushort_as_half((unsigned short)h)));
    }
  }
  // numbers 2 k and 2 k + 1
  __device__ __forceinline__ float2 pair(int k) const {
    if constexpr (sizeof(T) == 4) {
      const uint4 v = w[k >> 1];
      return (k & 1) ? make_float2(__uint_as_float(v.z), __uint_as_float(v.w)) : make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    } else {
      const uint32_t v = k == 0 ? w[0].x : k == 1 ? w[0].y : k == 2 ? w[0].z : w[0].w;
      if constexpr (std::is_same<T, __nv_bfloat16>::value) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
      else return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) q8_scores_kernel(const __grid_constant__ Q8SelectArgs a, int tiles, long long total, int step) {
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ Shared sm;
  uint8_t *const abuf = dyn, *const bbuf = dyn + kABytes;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = a.q.group;
  if (tid == 0) {
    mbar_init(&sm.bar, 1);
    mbar_fence_init();
  }
  if (warp == 1) {  // (one whose lanes are together: the first's have just parted)
    tmem_alloc(smem_u32(&sm.tmem), kTileRows);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sm.tmem, u_d = warp_uniform(tmem);
  pdl_wait();
  // slices begin at multiples of `step` tiles
  const long long g0 = total / step * blockIdx.x / gridDim.x * step, g1 = total / step * (blockIdx.x + 1) / gridDim.x * step;
  const bool issue = elect_lane();
  const uint32_t u_a = warp_uniform(smem_u32(abuf)), u_b = warp_uniform(smem_u32(bbuf));
  const int r8 = lane & 7, c8 = lane >> 3;  // a warp's part of an operand's conversion: 8 rows, four columns of 16 bytes
  uint32_t phase = 0;
  bool bad = false;
  // A list's part of the slice: its blocks first .. first + n - 1 and its rows, of the tiles ta .. tb - 1. Lists that take all of their
  // blocks, or see none of the slice's, are passed over. All threads.
  struct Part {
    long long list, bh;
    int b, h, len, m, tok0, rows, first, n, ta, tb;
  };
  auto next_part = [&](long long &g, Part &p) {
    while (g < g1) {
      p.list = quotient(g, tiles), p.bh = quotient(p.list, a.lists);
      const int t0 = (int)(g - p.list * tiles), t1 = (int)min((long long)tiles, g1 - p.list * tiles);
      g = p.list * tiles + t1;
      const int l = (int)(p.list - p.bh * a.lists);
      p.b = (int)quotient(p.bh, a.q.heads_kv), p.h = (int)(p.bh - (long long)p.b * a.q.heads_kv);
      seq_sizes(a.q, p.b, &p.len, &p.m, p.h == 0 && l == 0 && t0 == 0 && tid == 0);
      p.tok0 = l * a.span;
      const int tok1 = min(p.m, (int)min((long long)a.q.n_q, (long long)p.tok0 + a.span));
      int lo = 0x7fffffff, hi = 0;
      for (int i = p.tok0 + tid; i < tok1; i += kThreads) {
        const int2 r = row_range(a.q, p.b, i, p.len, p.m);
        if (r.y > r.x) lo = min(lo, r.x), hi = max(hi, r.y);
      }
      lo = __reduce_min_sync(kFull, lo), hi = __reduce_max_sync(kFull, hi);
      if (lane == 0) sm.lo[warp] = lo, sm.hi[warp] = hi;
      __syncthreads();
      lo = __reduce_min_sync(kFull, lane < kWarps ? sm.lo[lane] : 0x7fffffff), hi = __reduce_max_sync(kFull, lane < kWarps ? sm.hi[lane] : 0);
      __syncthreads();
      p.first = hi > 0 ? lo / kQ8Block : 0, p.n = (hi + kQ8Block - 1) / kQ8Block - p.first;
      p.rows = max(0, tok1 - p.tok0) * G;
      p.ta = max(t0, p.first / kTileBlocks), p.tb = min(t1, (p.first + p.n + kTileBlocks - 1) / kTileBlocks);
      if (p.n > a.keep && p.ta < p.tb) return true;
    }
    return false;
  };
  // a warp has 8 rows of every 128, four lanes a row: as they lie, on their way
  constexpr int kTurns = kTileRows / (8 * kWarps);
  Eight<T> x[kTurns][4];
  auto load_row = [&](const Part &p, int r, Eight<T> (&y)[4]) {
    const int i = r / G, hq = p.h * G + r - i * G;
    const T *src = static_cast<const T *>(a.q.q) + p.b * a.q.qs.b + hq * a.q.qs.h + (p.tok0 + i) * a.q.qs.t + 8 * c8;
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c].load(src + 32 * c);
  };
  auto load = [&](const Part &p, int r0) {
#pragma unroll
    for (int u = 0; u < kTurns; ++u)
      if (r0 + 128 * u + 8 * warp < p.rows) load_row(p, min(r0 + 128 * u + 8 * warp + r8, p.rows - 1), x[u]);
  };
  // a warp's 8 blocks of a tile: their bounds on their way; and a block's scale, of the thread that writes its score
  uint4 v[4];
  float scale = 0.f;
  auto fetch = [&](const Part &p, int t) {
    auto block = [&](int j) {
      return j >= p.first && j < p.first + p.n ? q8_block(a.q.c.btab, a.q.c.pool_blocks, p.bh * a.q.c.nblk + j, a.q.error) : -1;
    };
    const long long at = block(t * kTileBlocks + 8 * warp + r8);
    const uint4 *src = reinterpret_cast<const uint4 *>(a.bounds + max(at, 0ll) * kK);
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = at >= 0 ? latest(src + c8 + 4 * c) : make_uint4(0, 0, 0, 0);  // 16 bounds, lo's first
    if (tid < kTileBlocks) {
      const long long mine = block(t * kTileBlocks + tid);
      scale = mine >= 0 ? latest(a.q.c.ks + mine) : -1.f;
    }
  };
  long long g = g0;
  Part cur;
  bool more = next_part(g, cur);
  if (more) load(cur, 0), fetch(cur, cur.ta);
  while (more && !bad) {
    // ---- the largest coordinate of the rows that count, and the first of these rows
    bool live[kTurns];
    uint32_t amax = 0;
    int good = 0x7fffffff;
    auto look = [&](int r0) {
#pragma unroll
      for (int u = 0; u < kTurns; ++u) {
        live[u] = false;
        const int r = r0 + 128 * u + 8 * warp + r8;
        if (r0 + 128 * u + 8 * warp >= cur.rows) continue;
        uint32_t top = max(max(x[u][0].top(), x[u][1].top()), max(x[u][2].top(), x[u][3].top()));
        top = max(top, __shfl_xor_sync(kFull, top, 8));
        top = max(top, __shfl_xor_sync(kFull, top, 16));
        const int2 rg = row_range(a.q, cur.b, cur.tok0 + min(r, cur.rows - 1) / G, cur.len, cur.m);
        live[u] = r < cur.rows && top < 0x7f800000u && rg.y > rg.x;
        if (live[u]) amax = max(amax, top), good = min(good, r);
      }
    };
    look(0);
    if (cur.rows > kTileRows) {
#pragma unroll 1
      for (int r0 = kTileRows; r0 < cur.rows; r0 += kTileRows) load(cur, r0), look(r0);
      load(cur, 0), look(0);
    }
    amax = __reduce_max_sync(kFull, amax), good = __reduce_min_sync(kFull, good);
    if (lane == 0) sm.amax[warp] = amax, sm.good[warp] = good;
    __syncthreads();
    amax = __reduce_max_sync(kFull, lane < kWarps ? sm.amax[lane] : 0u), good = __reduce_min_sync(kFull, lane < kWarps ? sm.good[lane] : 0x7fffffff);
    const float lift = amax < 0x0d800000u ? pow2i(100) : 1.f;  // as in q8_choose_kernel
    const float by = pow2i(-row_exponent(__float_as_uint(__uint_as_float(amax) * lift), 6));
    const bool none = good == 0x7fffffff;
    const __half2 zero = __half2half2(__ushort_as_half(0)), most = __half2half2(__ushort_as_half(0x57f0));  // 127
    uint32_t *const keys = a.keys + cur.list * a.keys_ld;
    Part after;
    bool next = false;
#pragma unroll 1
    for (int r0 = 0; r0 < cur.rows && !bad; r0 += kTileRows) {
      // ---- the rows' operand; it is read by no product any more
      if (r0) load(cur, r0), look(r0);
      const int cols = cur.rows - r0 <= 128 ? 128 : 256;
      const bool last = r0 + kTileRows >= cur.rows;
#pragma unroll
      for (int u = 0; u < kTurns; ++u) {
        const int q = 128 * u + 8 * warp;
        if (q >= cols) continue;
        if (!none && !__all_sync(kFull, live[u])) {  // rows that do not count are copies of one that does
          if (!live[u]) load_row(cur, good, x[u]);
        }
        uint8_t *row = bbuf + (q >> 3) * kGroupBytes + r8 * 16;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t p[4], w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // to nearest even: 1.5 2^23 has steps of 1
            float2 f = x[u][c].pair(k);
            f.x = fmaf(f.x * lift, by, 12582912.f) - 12582912.f, f.y = fmaf(f.y * lift, by, 12582912.f) - 12582912.f;
            __half2 y = __floats2half2_rn(f.x, f.y);
            if (none) y = zero;
            const __half2 up = __hmin2(__hmax2(y, zero), most), down = __hmax2(__hmin2(y, zero), __hneg2(most));
            p[k] = *reinterpret_cast<const uint32_t *>(&up), w[k] = *reinterpret_cast<const uint32_t *>(&down);
          }
          *reinterpret_cast<uint4 *>(row + (c8 + 4 * c) * 128) = make_uint4(p[0], p[1], p[2], p[3]);
          *reinterpret_cast<uint4 *>(row + (c8 + 4 * c + 16) * 128) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (last) {  // the next list's rows load behind this one's tiles
        next = next_part(g, after);
        if (next) load(after, 0);
      }
#pragma unroll 1
      for (int t = cur.ta; t < cur.tb; ++t) {
        // ---- the blocks' operand: hi, then lo
        {
          uint8_t *row = abuf + warp * kGroupBytes + r8 * 16;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int col = (2 * (c8 + 4 * c) + 16) & 31;  // of 8 numbers; the second half of the bounds comes first
            const uint2 y0 = bytes_h4(v[c].x), y1 = bytes_h4(v[c].y), y2 = bytes_h4(v[c].z), y3 = bytes_h4(v[c].w);
            *reinterpret_cast<uint4 *>(row + col * 128) = make_uint4(y0.x, y0.y, y1.x, y1.y);
            *reinterpret_cast<uint4 *>(row + (col + 1) * 128) = make_uint4(y2.x, y2.y, y3.x, y3.y);
          }
        }
        const float its = scale;
        fence_proxy_async_shared();
        tc_fence_before_sync();
        __syncthreads();
        if (warp == 0) {
          tc_fence_after_sync();
          const uint32_t idesc = warp_uniform(tc_idesc_f16_f32(kTileBlocks, cols));
#pragma unroll 1  // (descriptors of more than one are as many registers)
          for (int k = 0; k < kK / 16; ++k)
            if (issue) tc_mma_f16(u_d, tc_sdesc_kmajor(u_a + 256 * k, 128, kGroupBytes), tc_sdesc_kmajor(u_b + 256 * k, 128, kGroupBytes), idesc, k > 0);
          if (issue) tc_commit(smem_u32(&sm.bar));
          __syncwarp();
        }
        if (t + 1 < cur.tb) fetch(cur, t + 1);
        else if (!last) fetch(cur, cur.ta);
        else if (next) fetch(after, after.ta);
        bad = !mbar_wait_bounded(&sm.bar, phase & 1, a.q.error);
        ++phase;
        bad = __syncthreads_or(bad);
        if (bad) break;
        tc_fence_after_sync();
        // ---- a lane's maximum: a quarter of its columns a warp
        const int part = warp >> 2, row = 32 * (warp & 3) + lane, each = cols / 4;
        float best = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < each; c += 16) {
          float w[16];
          tmem_ld_cols<16>(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + part * each + c, w);
#pragma unroll
          for (int k = 0; k < 16; k += 2) best = fmaxf(best, fmaxf(w[k], w[k + 1]));
        }
        if (part) sm.part[part - 1][row] = best;
        tc_fence_before_sync();
        __syncthreads();
        tc_fence_after_sync();
        const int j = t * kTileBlocks + row;
        if (!part && j >= cur.first && j < cur.first + cur.n) {  // (row is tid: its scale is this block's)
          best = fmaxf(fmaxf(best, sm.part[0][row]), fmaxf(sm.part[1][row], sm.part[2][row]));
          if (r0) best = fmaxf(best, __uint_as_float(keys[j]));
          keys[j] = !last ? __float_as_uint(best) : its < 0.f ? 0u : score_key(best * (its * 1.9073486e-6f));
        }
      }
    }
    cur = after, more = next;
    __syncthreads();  // sm.amax and the like are written again
  }
  if (bad) settle();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, kTileRows);
}

}  // namespace

int launch_q8_scores(const Q8SelectArgs &a, int num_sms, void *stream) {
  constexpr int smem = kABytes + kBBytes;
  const int tiles = (q8_blocks_of(a.q.max_len) + kTileBlocks - 1) / kTileBlocks;
  const long long lists = (long long)a.q.batch * a.q.heads_kv * a.lists, total = lists * tiles;
  const dim3 grid((unsigned)std::min((long long)num_sms, total));
  // A tile takes 2 us, a list's start 5: whole lists where the CTA with the most tiles and starts has no more than one of equal slices would (which
  // may begin with a list's last tile). 32 heads over 256 blocks, lists of 64 tokens, cut and whole: 1024 tokens 22.6 and 17.2 us, 2048
  // 32.6 and 27.4 (lists of 128: 44.3 and 29.5), 4096 45.9 and 48.0.
  const long long n = (lists + num_sms - 1) / num_sms, most = (total + num_sms - 1) / num_sms;
  const int step = 2 * n * tiles + 5 * n <= 2 * most + 5 * (1 + (most + tiles - 2) / tiles) ? tiles : 1;
  auto run = [&](bool allowed, auto kernel) {
    if (!allowed) return TQ_ERR_CUDA;
    return launch_overlapped(true, kernel, grid, dim3(kThreads), smem, (cudaStream_t)stream, a, tiles, total, step) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
  };
  if (a.q.q_dtype == TQ_F32) return run(allow_shared<q8_scores_kernel<float>>(smem), q8_scores_kernel<float>);
  if (a.q.q_dtype == TQ_BF16) return run(allow_shared<q8_scores_kernel<__nv_bfloat16>>(smem), q8_scores_kernel<__nv_bfloat16>);
  return run(allow_shared<q8_scores_kernel<__half>>(smem), q8_scores_kernel<__half>);
}

}  // namespace tq
