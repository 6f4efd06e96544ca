// Bounds of the key codes of each 64-token block (tq_q8_bounds): per coordinate the floor of a quarter of the smallest
// code and the ceiling of a quarter of the largest, as int8.
//
// One warp per block. A lane owns a 16-coordinate column of every fourth token (16 loads of 16 bytes, all in flight; four lanes read
// 64 bytes of a line, the next load the other 64), keeps the smallest and largest codes as 16-bit pairs without converting
// them, and the four lanes of a column split its coordinates among them to finish.
// e4m3 bytes are sign and magnitude. As upper bytes of 16-bit numbers (the lower byte only breaks ties): the largest unsigned number is the
// smallest code if any is negative, else the smallest unsigned one is; the largest signed number is the largest code if any
// is not negative, else the smallest unsigned one is. So three running numbers, in instructions that take two new ones at a time.
// Bound by memory, or for one step's blocks by a launch and the chain of lengths, table and codes. 4 x 16384 tokens, 8 KV heads: 13.3 us where
// the keys' 67 MB take 9.9 (2.5 us are the launch; ALU 48 % busy); one new token for each of 16 sequences: 2.5 us.

#include <algorithm>

#include "tq_q8.cuh"

namespace tq {
namespace {

constexpr int kWarps = 8;

__global__ void __launch_bounds__(32 * kWarps) q8_bounds_kernel(const __grid_constant__ Q8BoundsArgs a, int reach) {
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);  // (sequence, head, block of the new tokens)
  const int bh = (int)(unit / reach), b = bh / a.heads;
  pdl_trigger();
  pdl_wait();
  if (b >= a.batch) return;
  const int len = latest(a.seq_lens + b), m = a.new_lens ? latest(a.new_lens + b) : a.n_new;
  if (m < 0 || m > a.n_new) {
    if (lane == 0) set_error(a.error, TQ_ERR_ARG);
    return;
  }
  if (m == 0) return;
  if (len < 0 || len > a.c.capacity - m) {
    if (lane == 0) set_error(a.error, TQ_ERR_CAPACITY);
    return;
  }
  const int blk = len / kQ8Block + (int)(unit - (long long)bh * reach);
  const int count = min(kQ8Block, len + m - blk * kQ8Block);
  if (count <= 0) return;
  const long long at = q8_block(a.c.btab, a.c.pool_blocks, (long long)bh * a.c.nblk + blk, a.error);
  if (at < 0) return;
  const int col = lane >> 2, t0 = lane & 3;
  const uint8_t *src = a.c.records + at * kQ8BlockBytes + 128 * col;
  uint4 x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int t = 4 * i + t0;
    x[i] = *reinterpret_cast<const uint4 *>(src + q8_off(t < count ? t : 0, 0));  // a token that is not there counts as the first again
  }
  uint32_t umax[8], umin[8], smax[8];  // of the column's words, upper bytes of the halves, then lower bytes
#pragma unroll
  for (int k = 0; k < 8; ++k) umax[k] = 0u, umin[k] = 0xffffffffu, smax[k] = 0x80008000u;
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const uint32_t v[2][4] = {{x[i].x, x[i].y, x[i].z, x[i].w}, {x[i + 1].x, x[i + 1].y, x[i + 1].z, x[i + 1].w}};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t p = k < 4 ? v[0][k & 3] : v[0][k & 3] << 8, q = k < 4 ? v[1][k & 3] : v[1][k & 3] << 8;
      umax[k] = __vimax3_u16x2(umax[k], p, q);
      umin[k] = __vimin3_u16x2(umin[k], p, q);
      smax[k] = __vimax3_s16x2(smax[k], p, q);
    }
  }
  // the other lanes' tokens: halves of the words change places, then halves of these, so that a lane ends with one word's
  auto merge = [&](uint32_t &um, uint32_t &un, uint32_t &sm, uint32_t um1, uint32_t un1, uint32_t sm1, int o) {
    um = __vmaxu2(um, __shfl_xor_sync(kFull, um1, o));
    un = __vminu2(un, __shfl_xor_sync(kFull, un1, o));
    sm = __vmaxs2(sm, __shfl_xor_sync(kFull, sm1, o));
  };
  const bool hi2 = lane & 2, hi1 = lane & 1;
#pragma unroll
  for (int part = 0; part < 8; part += 4) {  // upper bytes, lower bytes
#pragma unroll
    for (int k = part; k < part + 2; ++k) {
      uint32_t um = hi2 ? umax[k + 2] : umax[k], un = hi2 ? umin[k + 2] : umin[k], sm = hi2 ? smax[k + 2] : smax[k];
      merge(um, un, sm, hi2 ? umax[k] : umax[k + 2], hi2 ? umin[k] : umin[k + 2], hi2 ? smax[k] : smax[k + 2], 2);
      umax[k] = um, umin[k] = un, smax[k] = sm;
    }
    uint32_t um = hi1 ? umax[part + 1] : umax[part], un = hi1 ? umin[part + 1] : umin[part], sm = hi1 ? smax[part + 1] : smax[part];
    merge(um, un, sm, hi1 ? umax[part] : umax[part + 1], hi1 ? umin[part] : umin[part + 1], hi1 ? smax[part] : smax[part + 1], 1);
    umax[part] = um, umin[part] = un, smax[part] = sm;
  }
  // this lane's word: coordinates 16 col + 4 (lane % 4) ..; bytes 1 and 3 from the upper half of the work, 0 and 2 from the lower
  uint32_t lo = 0, hi = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int k = (c & 1) ? 0 : 4, sh = (c & 2) ? 24 : 8;
    const uint32_t um = (umax[k] >> sh) & 0xffu, un = (umin[k] >> sh) & 0xffu, sm = (smax[k] >> sh) & 0xffu;
    const float low = e4m3x2_f((um & 0x80u) ? um : un).x, high = e4m3x2_f((sm & 0x80u) ? un : sm).x;
    lo |= ((uint32_t)__float2int_rd(low * 0.25f) & 0xffu) << (8 * c);
    hi |= ((uint32_t)__float2int_ru(high * 0.25f) & 0xffu) << (8 * c);
  }
  uint32_t *dst = reinterpret_cast<uint32_t *>(a.bounds + at * (2 * kD));
  dst[lane] = lo;
  dst[kD / 4 + lane] = hi;
}

}  // namespace

int launch_q8_bounds(const Q8BoundsArgs &a, void *stream) {
  const int reach = (std::min(a.n_new, a.c.capacity) - 1 + kQ8Block - 1) / kQ8Block + 1;  // blocks that the tokens of one call lie in, at most
  const long long units = (long long)a.batch * a.heads * reach, grid = (units + kWarps - 1) / kWarps;
  if (grid > 0x7fffffff) return TQ_ERR_UNSUPPORTED;
  return launch_overlapped(true, q8_bounds_kernel, dim3((unsigned)grid), dim3(32 * kWarps), 0, (cudaStream_t)stream, a, reach) == cudaSuccess
             ? TQ_OK : TQ_ERR_CUDA;
}

}  // namespace tq
