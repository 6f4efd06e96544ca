// Eviction from the 8-bit cache by accumulated attention weight (tq_q8_evict): per sequence and KV
// head keep the first `sink`, the last `recent` and the heaviest of the other tokens, in order, in
// another cache.
//
// q8_select_kernel: weights map to unsigned keys of the same order (NaN lowest); the key of the last
// token that stays is found digit by digit (11, 11 and 10 bits, from the top) with a histogram of the
// keys that share the digits found so far; ties at that key go to the lowest slots, and the warps' runs of slots
// are walked in order to give every kept one its place. Keys are read once from memory and stay in shared memory (what does not
// fit is read again). A cluster of up to 8 CTAs shares one long sequence-head: each holds a run of
// slots, histograms and counts are added through distributed shared memory.
// Bound by its chain of passes and cluster barriers (8 heads of 131072 slots: 25 us, where reading the weights takes 1).
// q8_gather_kernel: one CTA per 64-token block of the target (or per few). A thread owns one 16-byte piece (16
// coordinates of one token) of the keys and one of the values; the new block's scale comes from the largest value, and codes are rounded
// only where their block's scale differs from it. Bound by memory: a kept token's pieces lie 16 bytes wide among its neighbours', so
// that at one token in two kept three quarters of the source's sectors are read. 128 sequence-heads of 8192 slots cut to 4000:
// 52 us for both caches' 227 MB, 4.4 TB/s, the ALU 65 % busy with rounding; with its selection 72 us.

#include <cooperative_groups.h>

#include "tq_q8.cuh"

namespace cg = cooperative_groups;

namespace tq {
namespace {

constexpr int kSel = 1024;             // threads of a selecting CTA
constexpr int kBins = 2048;
constexpr int kMaxRanks = 8;           // CTAs of a cluster
constexpr int kSelKeys = 45056;        // keys held in shared memory (176 KB)
constexpr uint32_t kAlways = 0xffffffffu;  // a slot that stays whatever its weight

// order-preserving key: larger weight, larger key; -0 = +0, NaN below everything; never kAlways
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// exclusive prefix sum over the CTA; *total receives the sum (all threads call)
__device__ __forceinline__ int block_scan(int v, int *warp_sums, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  *total = warp_sums[31];
  const int before = warp ? warp_sums[warp - 1] : 0;
  __syncthreads();
  return before + x - v;
}

__global__ void __launch_bounds__(kSel) q8_select_kernel(const __grid_constant__ Q8EvictArgs a) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(8) int hist[kBins];
  __shared__ __align__(8) int added[kBins / 2];
  __shared__ int sums[32], found[2], share[2], warp_more[kSel / 32], warp_ties[kSel / 32];
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, ranks = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int bh = blockIdx.x / ranks, b = bh / a.heads;
  pdl_wait();
  int n = latest(a.seq_lens + b);
  if (n < 0 || n > a.src.capacity) {
    if (tid == 0) set_error(a.error, TQ_ERR_ARG);
    n = n < 0 ? 0 : a.src.capacity;
  }
  const int m = min(n, a.keep);
  const float *w = a.weights + (long long)bh * a.src.capacity;
  int32_t *kept = a.kept + (long long)bh * a.keep;
  float *dw = a.dst_weights ? a.dst_weights + (long long)bh * a.dst.capacity : nullptr;
  int32_t *dp = a.dst_positions ? a.dst_positions + (long long)bh * a.dst.capacity : nullptr;

  // this CTA's run of slots
  const int run = (n + ranks - 1) / ranks;
  const int s0 = min(n, rank * run), cnt = min(n, s0 + run) - s0;
  int pick = n > a.keep ? a.keep - a.sink - a.recent : 0;  // tokens chosen by weight
  // slots from the sink to the recent ones have a key, of their weight; where all stay, none
  const int low = n <= a.keep ? cnt : a.sink - s0, high = n - a.recent - s0, held = min(cnt, kSelKeys);
  auto make = [&](int i) -> uint32_t { return i < low || i >= high ? kAlways : weight_key(latest(w + s0 + i)); };
  auto key = [&](int i) -> uint32_t { return i < kSelKeys ? keys[i] : make(i); };
#pragma unroll 16
  for (int i = tid; i < held; i += kSel) keys[i] = make(i);
  if (tid < (-held & 3)) keys[held + tid] = kAlways;  // whole groups of four
  __syncthreads();  // the runs below cross threads, also where nothing is chosen by weight

  uint32_t prefix = pick > 0 ? 0 : kAlways, mask = 0;  // the digits of the threshold found so far
  int need = pick;                // tokens still to choose among the keys with these digits
  if (pick > 0) {                 // the same for every CTA of the cluster
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t digit = pass == 2 ? 1023u : 2047u;
      hist[tid] = 0, hist[tid + kSel] = 0;
      __syncthreads();
      auto count = [&](uint32_t k) {
        if (k != kAlways && ((k ^ prefix) & mask) == 0) atomicAdd(&hist[(k >> shift) & digit], 1);
      };
#pragma unroll 4
      for (int i = 4 * tid; i < held; i += 4 * kSel) {
        const uint4 k = *reinterpret_cast<const uint4 *>(keys + i);
        count(k.x), count(k.y), count(k.z), count(k.w);
      }
      for (int i = kSelKeys + tid; i < cnt; i += kSel) count(make(i));
      cl.sync();
      // bins in falling order: thread t sums bins 2047 - 2t and 2046 - 2t over the cluster
      int hi = 0, lo = 0;
      if (ranks == 1) {
        hi = hist[kBins - 1 - 2 * tid], lo = hist[kBins - 2 - 2 * tid];
      } else {
        // each rank adds up its share of the bins, then reads the others' sums (loads of all ranks in flight at once)
        const int part = kBins / ranks;
        if (tid < part) {
          int x = 0;
#pragma unroll
          for (int r = 0; r < kMaxRanks; ++r) x += r < ranks ? cl.map_shared_rank(hist, r)[rank * part + tid] : 0;
          added[tid] = x;
        }
        cl.sync();
        const int first = kBins - 2 - 2 * tid;  // both bins are one rank's
        const int2 x = *reinterpret_cast<const int2 *>(cl.map_shared_rank(added, first / part) + first % part);
        hi = x.y, lo = x.x;
      }
      int total;
      const int above = block_scan(hi + lo, sums, &total);
      if (above < need && need <= above + hi) found[0] = kBins - 1 - 2 * tid, found[1] = need - above;
      else if (above + hi < need && need <= above + hi + lo) found[0] = kBins - 2 - 2 * tid, found[1] = need - above - hi;
      cl.sync();  // also: every CTA has read the histograms
      prefix |= (uint32_t)found[0] << shift;
      mask |= digit << shift;
      need = found[1];
      __syncthreads();
    }
  }
  // Every warp's run of the CTA's slots, 32 at a time in their order: how many stay for their weight, how many tie, then the places.
  const int lane = tid & 31, warp = tid >> 5, seg = (cnt + kSel - 1) / kSel * 32;
  const int i0 = min(cnt, warp * seg), i1 = min(cnt, i0 + seg);
  auto above = [&](uint32_t k) { return k == kAlways || k > prefix; };
  auto equal = [&](uint32_t k) { return k == prefix && k != kAlways; };
  int more = 0, ties = 0;
#pragma unroll 4
  for (int i = i0 + lane; i < i1; i += 32) {
    const uint32_t k = key(i);
    more += above(k) ? 1 : 0;
    ties += equal(k) ? 1 : 0;
  }
  more = __reduce_add_sync(kFull, more), ties = __reduce_add_sync(kFull, ties);
  if (lane == 0) warp_more[warp] = more, warp_ties[warp] = ties;
  __syncthreads();
  auto scan = [&](int x) {  // inclusive, over the lanes: lane l holds warp l's number
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  const int its = warp_ties[lane];
  int tie = scan(its);
  if (tid == 31) share[0] = tie;
  cl.sync();
  tie -= its;
#pragma unroll
  for (int r = 0; r < kMaxRanks; ++r) tie += r < rank ? *cl.map_shared_rank(&share[0], r) : 0;
  const int won = max(0, min(its, need - tie));  // of that warp's ties, the lowest slots
  const int stays = warp_more[lane] + won;
  int at = scan(stays);
  if (tid == 31) share[1] = at;
  cl.sync();
  at -= stays;
#pragma unroll
  for (int r = 0; r < kMaxRanks; ++r) at += r < rank ? *cl.map_shared_rank(&share[1], r) : 0;
  at = __shfl_sync(kFull, at, warp);
  int left = __shfl_sync(kFull, won, warp);
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll 4
  for (int base = i0; base < i1; base += 32) {
    const int i = base + lane;
    const uint32_t k = i < i1 ? key(i) : 0u;
    const uint32_t tied = __ballot_sync(kFull, i < i1 && equal(k));
    const bool stay = i < i1 && (above(k) || (equal(k) && __popc(tied & below) < left));
    left = max(0, left - __popc(tied));
    const uint32_t all = __ballot_sync(kFull, stay);
    const int place = at + __popc(all & below);
    if (stay && place < a.keep) kept[place] = s0 + i;
    at += __popc(all);
  }
  const int me = rank * kSel + tid, everyone = ranks * kSel;
  for (int i = m + me; i < a.keep; i += everyone) kept[i] = -1;
  for (int i = a.keep + me; i < a.dst.capacity; i += everyone) {  // (the gathering kernel writes the first `keep`)
    if (dw) dw[i] = 0.f;
    if (dp) dp[i] = 0;
  }
  cl.sync();  // no CTA leaves while another may read its shared memory
}

constexpr int kGather = kQ8Block * 8;

// `per` consecutive blocks of the target; the next block's indices are loaded ahead.
__global__ void __launch_bounds__(kGather) q8_gather_kernel(const __grid_constant__ Q8EvictArgs a, int per) {
  __shared__ uint32_t red[2][2][kGather / 32];
  // a warp: one 16-byte column of 32 tokens, whose pieces lie 8 to a 128-byte line
  const int tid = threadIdx.x, t = tid & 63, c = tid >> 6;
  const long long bh = blockIdx.y;
  const int blocks = (a.keep + kQ8Block - 1) / kQ8Block, j0 = blockIdx.x * per, j1 = min(blocks, j0 + per);
  const int32_t *kept = a.kept + bh * a.keep;
  auto index = [&](int j) { return j * kQ8Block + t < a.keep ? latest(kept + j * kQ8Block + t) : -1; };
  pdl_wait();
  if (blockIdx.x == 0 && bh % a.heads == 0 && tid == 0) {  // here, where no other thread reads the lengths: they may be updated in place
    const int b = (int)(bh / a.heads);
    a.dst_lens[b] = min(min(max(a.seq_lens[b], 0), a.src.capacity), a.keep);
  }
  int next = index(j0);
  for (int j = j0; j < j1; ++j) {
    const int s = next;
    if (j + 1 < j1) next = index(j + 1);
    const long long to = q8_block(a.dst.btab, a.dst.pool_blocks, bh * a.dst.nblk + j, a.error);
    uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    int e0[2] = {kQ8MinExp, kQ8MinExp};
    const bool live = s >= 0 && s < a.src.capacity;
    if (c < 2 && j * kQ8Block + t < a.keep) {  // its weight and position
      const long long at = bh * a.dst.capacity + j * kQ8Block + t, of = bh * a.src.capacity + s;
      if (c == 0 && a.dst_weights) a.dst_weights[at] = live ? latest(a.weights + of) : 0.f;
      if (c == 1 && a.dst_positions) a.dst_positions[at] = !live ? 0 : a.positions ? latest(a.positions + of) : s;
    }
    if (live) {
      const long long from = q8_block(a.src.btab, a.src.pool_blocks, bh * a.src.nblk + s / kQ8Block, a.error);
      if (from >= 0) {
        const uint8_t *p = a.src.records + from * kQ8BlockBytes + q8_off(s % kQ8Block, 16 * c);
        w[0] = latest(reinterpret_cast<const uint4 *>(p));
        w[1] = latest(reinterpret_cast<const uint4 *>(p + kQ8Plane));
        e0[0] = log2i(latest(a.src.ks + from));
        e0[1] = log2i(latest(a.src.vs + from));
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      // the largest magnitude of the piece: e4m3 magnitudes are ordered as their low seven bits
      uint32_t top = __vmaxu4(__vmaxu4(w[k].x & 0x7f7f7f7fu, w[k].y & 0x7f7f7f7fu),
                              __vmaxu4(w[k].z & 0x7f7f7f7fu, w[k].w & 0x7f7f7f7fu));
      top = __vmaxu4(top, top >> 16);
      top = max(top & 0xffu, (top >> 8) & 0xffu);
      const uint32_t amax = __reduce_max_sync(kFull, __float_as_uint(e4m3x2_f(top).x * pow2i(e0[k])));
      if ((tid & 31) == 0) red[j & 1][k][tid >> 5] = amax;
    }
    __syncthreads();
    if (to < 0) continue;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int e = q8_exponent(__reduce_max_sync(kFull, red[j & 1][k][tid & (kGather / 32 - 1)]));
      if (e != e0[k]) {
        const float f = pow2i(min(max(e0[k] - e, -126), 126));
        w[k] = make_uint4(e4m3x4_scaled(w[k].x, f), e4m3x4_scaled(w[k].y, f), e4m3x4_scaled(w[k].z, f), e4m3x4_scaled(w[k].w, f));
      }
      *reinterpret_cast<uint4 *>(a.dst.records + to * kQ8BlockBytes + k * kQ8Plane + q8_off(t, 16 * c)) = w[k];
      if (tid == 0) (k ? a.dst.vs : a.dst.ks)[to] = pow2i(e);
    }
  }
}

}  // namespace

int launch_q8_evict(const Q8EvictArgs &a, int num_sms, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  const long long bh = (long long)a.batch * a.heads;
  if (bh > 65535) return TQ_ERR_UNSUPPORTED;
  // CTAs per sequence-head: as many as keep 2048 slots each while all run at once, and enough to hold the keys in shared memory.
  // Clusters of 8 fill only half of the SMs (a GPC takes whole clusters). 8 heads of 131072 slots: 37 us with 8 CTAs each, 46 with
  // 4, 104 with 2 (keys read again), 219 with 1; 16 heads: 70 with 8, 56 with 4; 64 heads: 202, 150, 177, 293; 128
  // heads of 8192 slots: 76 with 1, 89 with 2; 32 heads: 37 with 1, 33 with 4.
  int ranks = 1;
  while (ranks < kMaxRanks && (a.src.capacity > (long long)kSelKeys * ranks ||
                               (a.src.capacity > 2048LL * ranks && 2 * ranks * bh <= (ranks == 4 ? num_sms / 2 : num_sms))))
    ranks *= 2;
  const int held = ((a.src.capacity + ranks - 1) / ranks + 3) / 4 * 4;
  const size_t smem = sizeof(uint32_t) * (size_t)(held < kSelKeys ? held : kSelKeys);
  if (cudaFuncSetAttribute(q8_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelKeys * 4) != cudaSuccess)
    return TQ_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(bh * ranks));
  cfg.blockDim = dim3(kSel);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the launch overlaps the kernel before it
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, q8_select_kernel, a) != cudaSuccess) return TQ_ERR_CUDA;
  const int blocks = (a.keep + kQ8Block - 1) / kQ8Block;
  // blocks per CTA: 2 or 4 where sixteen CTAs an SM remain (8064 blocks: 75.6 us with 1, 72.9 with 2, 72.8 with 4; 512: 37.6, 37.9, 40.7)
  const long long rounds = (long long)blocks * bh / (16LL * num_sms);
  const int per = rounds >= 4 ? 4 : rounds >= 2 ? 2 : 1;
  const dim3 grid((unsigned)((blocks + per - 1) / per), (unsigned)bh);
  return launch_overlapped(true, q8_gather_kernel, grid, dim3(kGather), 0, st, a, per) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // namespace tq
