// Rotary positions: y = R(pos) x for [batch][heads][n][128] vectors (tq_rotary).
//
// Pair (a, b) -> gain (a cos - b sin, b cos + a sin). Bound by memory: every element is read and
// written once. A thread owns V + V elements of a row (the two halves of V pairs, or 2V
// consecutive elements when the pairs are interleaved; a row's coordinates past `dim` pass
// through), forms their V sines and cosines once and uses them for several heads of its token, the
// loads of four in flight before the first is used (one at a time: 71 us where four take 45). V = 8
// (16-byte accesses for 16-bit types) needs dim a multiple of 16, V = 4 covers the other multiples of 8.
// Measured: 16384 tokens of 32 heads in bf16, 64 of 128 coordinates interleaved: 44 us, 6.1 TB/s, 0.90 of a
// plain copy; what is left is the loads' latency (7 of 10 stalled warps) and the sines (ALU 38 % busy). 16 tokens: 2.6 us, a launch.

#include "tq_q8.cuh"

namespace tq {
namespace {

// V consecutive elements as they lie in memory
template <typename T, int V>
struct Words {
  static constexpr int kWords = V * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (kWords % 4 == 0) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 x = reinterpret_cast<const uint4 *>(p)[i];
        w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
      }
    } else {
      const uint2 x = *reinterpret_cast<const uint2 *>(p);
      w[0] = x.x, w[1] = x.y;
    }
  }
  __device__ __forceinline__ void store(T *p) const {
    if constexpr (kWords % 4 == 0) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i)
        reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
      *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
  }
  __device__ __forceinline__ void floats(float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
      else if constexpr (std::is_same<T, __nv_bfloat16>::value) v[i] = __uint_as_float((i & 1) ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
      else v[i] = __half2float(__ushort_as_half((unsigned short)((i & 1) ? w[i / 2] >> 16 : w[i / 2])));
    }
  }
};

template <typename T, int V, bool IL>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2) rotary_kernel(const __grid_constant__ RotaryArgs a, int hpt, long long items) {
  constexpr int kRow = kD / (2 * V);  // threads of a row
  __shared__ unsigned long long freq[kD / 2];
  if (threadIdx.x < kD / 2) freq[threadIdx.x] = a.rope.freq[threadIdx.x];
  __syncthreads();
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  if (id >= items) return;
  pdl_wait();
  const int j = (int)(id % kRow);
  long long rest = id / kRow;
  // neighbouring threads on rows that lie together: of one token's heads, or of one head's tokens
  const int chunks = (a.heads + hpt - 1) / hpt, inner = a.by_token ? chunks : a.n, outer = a.by_token ? a.n : chunks;
  const int i0 = (int)(rest % inner);
  rest /= inner;
  const int i1 = (int)(rest % outer), b = (int)(rest / outer);
  const int t = a.by_token ? i1 : i0, h0 = (a.by_token ? i0 : i1) * hpt;
  const int h1 = min(a.heads, h0 + hpt);
  const int dim = a.rope.dim;
  // the two vectors of this thread: the halves of V pairs, or 2V consecutive elements
  const bool turn = 2 * V * j < dim;
  const int c0 = IL || !turn ? 2 * V * j : V * j, c1 = IL || !turn ? c0 + V : c0 + dim / 2;
  float cs[V], sn[V];
  if (turn) {
    const int pos = latest(a.positions + (long long)b * a.n + t);
    const float sign = a.transpose ? -a.rope.gain : a.rope.gain;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      rope_sincos(pos, freq[V * j + i], &cs[i], &sn[i]);
      cs[i] *= a.rope.gain;
      sn[i] *= sign;
    }
  }
  const T *x = static_cast<const T *>(a.x) + b * a.xs.b + t * a.xs.t;
  T *y = static_cast<T *>(a.y) + b * a.ys.b + t * a.ys.t;
  constexpr int kU = 4;
  for (int h = h0; h < h1; h += kU) {
    Words<T, V> u[kU], w[kU];  // as they lie in memory: four heads' loads in flight take 32 registers of a 16-bit type
#pragma unroll
    for (int k = 0; k < kU; ++k)
      if (h + k < h1) {
        u[k].load(x + (h + k) * a.xs.h + c0);
        w[k].load(x + (h + k) * a.xs.h + c1);
      }
#pragma unroll
    for (int k = 0; k < kU; ++k)
      if (h + k < h1) {
        T *const p = y + (h + k) * a.ys.h + c0, *const q = y + (h + k) * a.ys.h + c1;
        if (turn) {
          float d[V], e[V];
          u[k].floats(d), w[k].floats(e);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            if constexpr (IL) {  // pairs (2i, 2i + 1) of the 2V elements
              float *const r = i < V / 2 ? &d[2 * i] : &e[2 * i - V];
              const float e0 = r[0], e1 = r[1];
              r[0] = rope_turn(e0, e1, cs[i], -sn[i]);
              r[1] = rope_turn(e1, e0, cs[i], sn[i]);
            } else {
              const float e0 = d[i], e1 = e[i];
              d[i] = rope_turn(e0, e1, cs[i], -sn[i]);
              e[i] = rope_turn(e1, e0, cs[i], sn[i]);
            }
          }
          store_vec<T, V>(p, d);
          store_vec<T, V>(q, e);
        } else {
          u[k].store(p);
          w[k].store(q);
        }
      }
  }
}

template <typename T, int V>
int launch(const RotaryArgs &a, int num_sms, cudaStream_t st) {
  const long long one = (long long)a.batch * a.n * a.heads * (kD / (2 * V));  // threads at one head each
  // Heads per thread (they share the sines): as many as leave 256 threads an SM, up to 4, and 8 where many remain. bf16, 32
  // heads: 512 tokens 5.3 us at one head, 4.2 at 2, 3.9 at 4; 16384 tokens 100, 60, 45.4 and, at 8, 44.6 (fp32 164 .. 94 and 90);
  // 64 tokens 3.2 at one, 3.5 at 4.
  long long hpt = (one + 256LL * num_sms - 1) / (256LL * num_sms);
  hpt = hpt < 1 ? 1 : hpt >= 32 ? 8 : hpt > 4 ? 4 : hpt;
  if (hpt > a.heads) hpt = a.heads;
  const long long items = (long long)a.batch * a.n * ((a.heads + hpt - 1) / hpt) * (kD / (2 * V));
  const long long grid = (items + 255) / 256;
  if (grid > 0x7fffffffLL) return TQ_ERR_UNSUPPORTED;
  auto *kernel = a.rope.interleaved ? rotary_kernel<T, V, true> : rotary_kernel<T, V, false>;
  const cudaError_t e = launch_overlapped(true, kernel, dim3((unsigned)grid), dim3(256), 0, st, a, (int)hpt, items);
  return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

template <typename T>
int launch_t(const RotaryArgs &a, int num_sms, cudaStream_t st) {
  return a.rope.dim % 16 == 0 ? launch<T, 8>(a, num_sms, st) : launch<T, 4>(a, num_sms, st);
}

}  // namespace

int launch_rotary(const RotaryArgs &args, int num_sms, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  RotaryArgs a = args;
  a.by_token = a.xs.h < a.xs.t;
  switch (a.dtype) {
    case TQ_F32: return launch_t<float>(a, num_sms, st);
    case TQ_BF16: return launch_t<__nv_bfloat16>(a, num_sms, st);
    default: return launch_t<__half>(a, num_sms, st);
  }
}

}  // namespace tq
