// Scores of blocks for lists of many rows (tq_q8_select), on the tensor cores.
//
// A row's score of a block is sum w+ hi + w- lo (tq_q8_select.cu): with the bounds of 128 blocks as the rows of one operand, [hi | lo],
// and up to 256 query rows as those of the other, [w+ | w-], it is one product over 256 numbers. Whole numbers up to 127
// are exact in fp16, their products in fp32, and every partial sum is a whole number below 2^21, so that the accumulators hold the scores
// exactly whatever the order. Blocks are accumulator lanes: a block's largest score over the rows is a maximum along its lane.
// Rows that do not count, and those that fill the operand up, are copies of one that does.
//
// Split: the (list, 128 blocks) space in equal slices, one CTA per SM; a list's rows are converted once a slice and
// 256 rows. Bound by the conversions and their loads; the products of 2048 tokens x 32 heads over 256 blocks would take 5 us.

#include <algorithm>

#include "tq_q8_rows.cuh"
#include "tq_q8_select.cuh"

namespace tq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kTileBlocks = 128, kTileRows = 256, kK = 2 * kD;
constexpr int kGroupBytes = kK / 8 * 128;                  // 8 rows of an operand: 32 columns of 8 numbers, 16 bytes each, a row after the other
constexpr int kABytes = kTileBlocks / 8 * kGroupBytes;     // 64 KB
constexpr int kBBytes = kTileRows / 8 * kGroupBytes;       // 128 KB

struct Shared {
  uint64_t bar;
  uint32_t amax[kWarps];
  int lo[kWarps], hi[kWarps], good[kWarps];
  float half[kTileBlocks];  // the second half of the columns' maxima
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

// Four signed bytes as fp16 numbers: 1024 + (b + 128) has b + 128 as its lowest bits.
__device__ __forceinline__ uint2 bytes_h4(uint32_t w) {
  w ^= 0x80808080u;
  uint32_t p = __byte_perm(w, 0x64646464u, 0x4140), q = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 base = __half2half2(__ushort_as_half(0x6480));  // 1152
  const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&p), base), y = __hsub2(*reinterpret_cast<__half2 *>(&q), base);
  return make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
}

// Eight coordinates from c on of row r of the list that begins with token tok0.
__device__ __forceinline__ void row_eight(const Q8AttnArgs &a, int b, int h, int tok0, int r, int c, float (&x)[8]) {
  const int i = tok0 + r / a.group, hq = h * a.group + r % a.group;
  const long long off = b * a.qs.b + hq * a.qs.h + i * a.qs.t + c;
  if (a.q_dtype == TQ_F32) load_vec<float, 8>(static_cast<const float *>(a.q) + off, x);
  else if (a.q_dtype == TQ_BF16) load_vec<__nv_bfloat16, 8>(static_cast<const __nv_bfloat16 *>(a.q) + off, x);
  else load_vec<__half, 8>(static_cast<const __half *>(a.q) + off, x);
}

__global__ void __launch_bounds__(kThreads, 1) q8_scores_kernel(const __grid_constant__ Q8SelectArgs a, int tiles, long long total) {
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ Shared sm;
  uint8_t *const abuf = dyn, *const bbuf = dyn + kABytes;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = a.q.group;
  if (tid == 0) {
    mbar_init(&sm.bar, 1);
    mbar_fence_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&sm.tmem), kTileRows);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sm.tmem;
  pdl_wait();
  const long long g0 = total * blockIdx.x / gridDim.x, g1 = total * (blockIdx.x + 1) / gridDim.x;
  const bool issue = elect_lane();
  const uint32_t u_a = smem_u32(abuf), u_b = smem_u32(bbuf);
  const int r8 = lane & 7, c8 = lane >> 3;  // a warp's part of an operand's conversion: 8 rows, four columns of 16 bytes
  uint32_t phase = 0;
  bool bad = false;
  for (long long g = g0; g < g1 && !bad;) {
    const long long list = g / tiles, bh = list / a.lists;
    const int t0 = (int)(g - list * tiles), t1 = (int)min((long long)tiles, g1 - list * tiles);
    g = list * tiles + t1;
    const int l = (int)(list - bh * a.lists), b = (int)(bh / a.q.heads_kv), h = (int)(bh - (long long)b * a.q.heads_kv);
    // ---- the list's blocks
    int len, m;
    seq_sizes(a.q, b, &len, &m, h == 0 && l == 0 && t0 == 0 && tid == 0);
    const int tok0 = l * a.span, tok1 = min(m, (int)min((long long)a.q.n_q, (long long)tok0 + a.span));
    int lo = 0x7fffffff, hi = 0;
    for (int i = tok0 + tid; i < tok1; i += kThreads) {
      const int2 r = row_range(a.q, b, i, len, m);
      if (r.y > r.x) lo = min(lo, r.x), hi = max(hi, r.y);
    }
    lo = __reduce_min_sync(kFull, lo), hi = __reduce_max_sync(kFull, hi);
    if (lane == 0) sm.lo[warp] = lo, sm.hi[warp] = hi;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) lo = min(lo, sm.lo[w]), hi = max(hi, sm.hi[w]);
    __syncthreads();
    const int first = hi > 0 ? lo / kQ8Block : 0, n = (hi + kQ8Block - 1) / kQ8Block - first;
    if (n <= a.keep || t1 * kTileBlocks <= first || t0 * kTileBlocks >= first + n) continue;  // all are taken, or none of these is seen
    // ---- the largest coordinate of the rows that count, and the first of these rows
    const int rows = (tok1 - tok0) * G;
    uint32_t amax = 0;
    int good = 0x7fffffff;
    auto counts = [&](int r, uint32_t top) {  // top: the row's largest
      const int2 rg = row_range(a.q, b, tok0 + r / G, len, m);
      return top < 0x7f800000u && rg.y > rg.x;
    };
    auto row_largest = [&](int r) {  // of a row that is there; four lanes of a warp share it
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float x[8];
        row_eight(a.q, b, h, tok0, r, 8 * (c8 + 4 * c), x);
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(x[k]) & 0x7fffffffu);
      }
      top = max(top, __shfl_xor_sync(kFull, top, 8));
      return max(top, __shfl_xor_sync(kFull, top, 16));
    };
    for (int r0 = 8 * warp; r0 < rows; r0 += 8 * kWarps) {
      const int r = min(r0 + r8, rows - 1);
      const uint32_t top = row_largest(r);
      if (counts(r, top)) amax = max(amax, top), good = min(good, r);
    }
    amax = __reduce_max_sync(kFull, amax), good = __reduce_min_sync(kFull, good);
    if (lane == 0) sm.amax[warp] = amax, sm.good[warp] = good;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) amax = max(amax, sm.amax[w]), good = min(good, sm.good[w]);
    const float lift = amax < 0x0d800000u ? pow2i(100) : 1.f;  // as in q8_choose_kernel
    const float by = pow2i(-row_exponent(__float_as_uint(__uint_as_float(amax) * lift), 6));
    const bool none = good == 0x7fffffff;
    uint32_t *const keys = a.keys + list * a.keys_ld;
    for (int r0 = 0; r0 < rows && !bad; r0 += kTileRows) {
      // ---- the rows' operand; it is read by no product any more
      const int cols = min(kTileRows, (rows - r0 + 63) & ~63);
      for (int q = 8 * warp; q < cols; q += 8 * kWarps) {
        int r = min(r0 + q + r8, rows - 1);
        const uint32_t top = row_largest(r);
        if (!counts(r, top)) r = none ? r : good;
        uint8_t *row = bbuf + (q >> 3) * kGroupBytes + r8 * 16;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float x[8];
          row_eight(a.q, b, h, tok0, r, 8 * (c8 + 4 * c), x);
          uint32_t p[4], w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float x0 = none ? 0.f : fminf(fmaxf(rintf(x[2 * k] * lift * by), -127.f), 127.f);
            const float x1 = none ? 0.f : fminf(fmaxf(rintf(x[2 * k + 1] * lift * by), -127.f), 127.f);
            const __half2 up = __floats2half2_rn(fmaxf(x0, 0.f), fmaxf(x1, 0.f)), down = __floats2half2_rn(fminf(x0, 0.f), fminf(x1, 0.f));
            p[k] = *reinterpret_cast<const uint32_t *>(&up), w[k] = *reinterpret_cast<const uint32_t *>(&down);
          }
          *reinterpret_cast<uint4 *>(row + (c8 + 4 * c) * 128) = make_uint4(p[0], p[1], p[2], p[3]);
          *reinterpret_cast<uint4 *>(row + (c8 + 4 * c + 16) * 128) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      for (int t = max(t0, first / kTileBlocks); t < min(t1, (first + n + kTileBlocks - 1) / kTileBlocks); ++t) {
        // ---- the blocks' operand: hi, then lo
        for (int q = 8 * warp; q < kTileBlocks; q += 8 * kWarps) {
          const int j = t * kTileBlocks + q + r8;
          const long long at = j >= first && j < first + n ? q8_block(a.q.c.btab, a.q.c.pool_blocks, bh * a.q.c.nblk + j, a.q.error) : -1;
          const uint4 *src = reinterpret_cast<const uint4 *>(a.bounds + max(at, 0ll) * kK);
          uint8_t *row = abuf + (q >> 3) * kGroupBytes + r8 * 16;
          uint4 v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = at >= 0 ? __ldg(src + c8 + 4 * c) : make_uint4(0, 0, 0, 0);  // 16 bounds, lo's first
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int col = (2 * (c8 + 4 * c) + 16) & 31;  // of 8 numbers; the second half of the bounds comes first
            const uint2 x = bytes_h4(v[c].x), y = bytes_h4(v[c].y), z = bytes_h4(v[c].z), w = bytes_h4(v[c].w);
            *reinterpret_cast<uint4 *>(row + col * 128) = make_uint4(x.x, x.y, y.x, y.y);
            *reinterpret_cast<uint4 *>(row + (col + 1) * 128) = make_uint4(z.x, z.y, w.x, w.y);
          }
        }
        fence_proxy_async_shared();
        tc_fence_before_sync();
        __syncthreads();
        if (warp == 0) {
          tc_fence_after_sync();
          const uint32_t idesc = tc_idesc_f16_f32(kTileBlocks, cols);
#pragma unroll
          for (int k = 0; k < kK / 16; ++k)
            if (issue) tc_mma_f16(tmem, tc_sdesc_kmajor(u_a + 256 * k, 128, kGroupBytes), tc_sdesc_kmajor(u_b + 256 * k, 128, kGroupBytes), idesc, k > 0);
          if (issue) tc_commit(smem_u32(&sm.bar));
          __syncwarp();
        }
        bad = !mbar_wait_bounded(&sm.bar, phase & 1, a.q.error);
        ++phase;
        bad = __syncthreads_or(bad);
        if (bad) break;
        tc_fence_after_sync();
        // ---- a lane's maximum: half of its columns a warp
        const int half = warp >> 2, row = 32 * (warp & 3) + lane, part = cols / 2;
        float best = -INFINITY;
        for (int c = 0; c < part; c += 32) {
          uint32_t v[32];
          tmem_ld_x32(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + half * part + c, v);
#pragma unroll
          for (int k = 0; k < 32; k += 2) best = fmaxf(best, fmaxf(__uint_as_float(v[k]), __uint_as_float(v[k + 1])));
        }
        if (half) sm.half[row] = best;
        tc_fence_before_sync();
        __syncthreads();
        tc_fence_after_sync();
        const int j = t * kTileBlocks + row;
        if (!half && j >= first && j < first + n) {
          best = fmaxf(best, sm.half[row]);
          const bool last = r0 + kTileRows >= rows;
          if (r0) best = fmaxf(best, __uint_as_float(keys[j]));
          uint32_t key = __float_as_uint(best);
          if (last) {
            const long long at = q8_block(a.q.c.btab, a.q.c.pool_blocks, bh * a.q.c.nblk + j, a.q.error);
            const bool sure = j < first + a.sink || j >= first + n - a.recent;
            key = sure ? kAlways : at < 0 ? 0u : score_key(best * (__ldg(a.q.c.ks + at) * 1.9073486e-6f));
          }
          keys[j] = key;
        }
      }
    }
    __syncthreads();  // sm.amax and the like are written again
  }
  if (bad) settle();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 0) tmem_dealloc(tmem, kTileRows);
}

}  // namespace

int launch_q8_scores(const Q8SelectArgs &a, int num_sms, void *stream) {
  constexpr int smem = kABytes + kBBytes;
  const int tiles = (q8_blocks_of(a.q.max_len) + kTileBlocks - 1) / kTileBlocks;
  const long long total = (long long)a.q.batch * a.q.heads_kv * a.lists * tiles;
  if (cudaFuncSetAttribute(q8_scores_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return TQ_ERR_CUDA;
  return launch_overlapped(true, q8_scores_kernel, dim3((unsigned)std::min((long long)num_sms, total)), dim3(kThreads), smem, (cudaStream_t)stream,
                           a, tiles, total) == cudaSuccess
             ? TQ_OK : TQ_ERR_CUDA;
}

}  // namespace tq
