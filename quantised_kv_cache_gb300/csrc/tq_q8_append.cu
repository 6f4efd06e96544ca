// Append to the 8-bit cache (tq_q8_append, tq_append_quantize of a TQ_SCHEME_Q8 context) and its
// dequantiser.
//
// Per block of 64 token slots and tensor: e = the least whole e >= -100 with max |x| <= 448 * 2^e
// over the call's new tokens in the block (the maximum with the block's own e when it already held
// tokens, whose codes are then rounded to the new scale), code = e4m3(x * 2^-e). A power-of-two
// scale makes x * 2^-e exact, so the codes do not depend on how the division is carried out.
//
// Bound by memory: the inputs are read and the codes written once. One CTA handles one block of
// slots of one tensor for a few heads: thread (t, j) owns 16 coordinates of token slot t, one 16-byte
// piece of a core matrix, or, for a rotation of halves, the two 8-byte pieces that hold 8 pairs, so that it needs nobody
// else's coordinates and 8 sines. Those are formed once for all heads of the CTA; the next head's inputs are
// loaded before the current one's maximum is awaited. (Halves of a rotation that is no multiple of 16
// wide do not split into such pieces: there the partners are loaded a second time.)
// Measured: 4 sequences of 16384 tokens, 8 KV heads, rotated, bf16: 85 us, 4.7 TB/s (0.70 of a plain copy; without rotation 68 us, 0.88):
// the ALU is 58 % busy with conversions and angles, and the CTA's maximum is a barrier per head (a block's maximum is needed
// before its first code; rows staged through shared memory by asynchronous copies took 98 us); fp16 the same, fp32, at one CTA an SM, 129 us, 5.2 TB/s (117 us, 0.84, without rotation). One token of 16 sequences: 3.9 us.

#include "tq_q8.cuh"

namespace tq {
namespace {

constexpr int kThreads = kQ8Block * 8;  // 64 token slots x 8 pieces of 16 coordinates

// How the keys are rotated: not at all; every pair inside its thread; halves with partners loaded again.
enum Rope { kNone = 0, kOwn = 1, kPartner = 2 };

// 16 coordinates of a token as they lie in memory: 8 in w[0 .. H - 1], 8 in w[H ..]. Two of a 16-bit type stay packed in a
// word until they are scaled, so that magnitudes are compared two at a time.
template <typename T>
struct Piece {
  static constexpr int kWords = 4 * (int)sizeof(T), H = kWords / 2;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T *p, const T *q) {
#pragma unroll
    for (int i = 0; i < H / 4; ++i) {
      const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p) + i), y = __ldg(reinterpret_cast<const uint4 *>(q) + i);
      w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
      w[H + 4 * i] = y.x, w[H + 4 * i + 1] = y.y, w[H + 4 * i + 2] = y.z, w[H + 4 * i + 3] = y.w;
    }
  }
  // coordinates 2 i and 2 i + 1
  __device__ __forceinline__ float2 pair(int i) const {
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else if constexpr (std::is_same<T, __nv_bfloat16>::value)
      return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
  }
  __device__ __forceinline__ void set(int i, float2 v) {  // rounded to T
    if constexpr (sizeof(T) == 4) {
      w[2 * i] = __float_as_uint(v.x), w[2 * i + 1] = __float_as_uint(v.y);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    } else {
      const __half2 h = __floats2half2_rn(v.x, v.y);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
  }
  // the largest magnitude's bits in T (ordered as the magnitudes; infinities and NaN on top)
  __device__ __forceinline__ uint32_t top() const {
    if constexpr (sizeof(T) == 4) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kWords; ++i) m = max(m, w[i] & 0x7fffffffu);
      return m;
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kWords; i += 2) m = __vimax3_u16x2(m, w[i] & 0x7fff7fffu, w[i + 1] & 0x7fff7fffu);
      return max(m & 0xffffu, m >> 16);
    }
  }
  static __device__ __forceinline__ uint32_t float_bits(uint32_t t) {
    if constexpr (sizeof(T) == 4) return t;
    else if constexpr (std::is_same<T, __nv_bfloat16>::value) return t << 16;
    else return __float_as_uint(__half2float(__ushort_as_half((unsigned short)t)));
  }
};

__device__ __forceinline__ float tame(float x) { return x != x ? 0.f : fminf(fmaxf(x, -kQ8Largest), kQ8Largest); }

template <typename T, int ROPE>
__global__ void __launch_bounds__(kThreads, ROPE == kPartner || sizeof(T) == 4 ? 1 : 2)
q8_append_kernel(const __grid_constant__ Q8AppendArgs a, int hpc) {
  __shared__ uint32_t red[4][kThreads / 32];
  const int tid = threadIdx.x, j = tid & 7, t = tid >> 3, warp = tid >> 5;
  const int b = blockIdx.y, tensor = blockIdx.z & 1, h0 = (blockIdx.z >> 1) * hpc;
  const int h1 = min(a.heads, h0 + hpc);
  const bool rope = ROPE != kNone && tensor == 0;

  pdl_wait();
  const int len = __ldg(a.seq_lens + b);
  int n = a.n_new;
  if (a.new_lens) {
    n = __ldg(a.new_lens + b);
    if (n < 0 || n > a.n_new) {
      if (tid == 0) set_error(a.error, TQ_ERR_ARG);
      return;
    }
  }
  if (len < 0 || (long long)len + n > a.c.capacity) {
    if (tid == 0) set_error(a.error, TQ_ERR_CAPACITY);
    return;
  }
  if (n == 0) return;
  const int blk0 = len / kQ8Block + blockIdx.x;   // block of the sequence
  if ((long long)blk0 * kQ8Block >= (long long)len + n) return;
  const int tok = blk0 * kQ8Block + t - len;      // the new token of this thread's slot
  const bool fresh = tok >= 0 && tok < n, older = tok < 0;
  const bool joins = blk0 * kQ8Block < len;       // the block already holds tokens

  // this thread's coordinates: 8 from c0 on, 8 from c1 on
  const int dim = a.table.dim, half = dim / 2;
  const bool turn = rope && 16 * j < dim;
  // (without a rotation too two eights 64 apart: a row's loads of a warp are then whole lines)
  const bool split = (ROPE == kOwn && turn && !a.table.interleaved) || !rope;
  const int c0 = split ? 8 * j : 16 * j, c1 = !split ? c0 + 8 : rope ? half + 8 * j : kD / 2 + 8 * j;
  constexpr int kSines = ROPE == kPartner ? 16 : 8;
  float cs[kSines], sn[kSines];
  if (turn && fresh) {
    const int pos = a.positions ? __ldg(a.positions + (long long)b * a.n_new + tok) : len + tok;
#pragma unroll
    for (int i = 0; i < kSines; ++i) {
      cs[i] = 1.f, sn[i] = 0.f;
      // pair of coordinate(s) i: kOwn 8 j + i in both layouts; kPartner the coordinate's own, sign by its half
      const bool second = ROPE == kPartner && c0 + i >= half;
      const int f = ROPE == kPartner ? c0 + i - (second ? half : 0) : 8 * j + i;
      if (ROPE == kPartner ? c0 + i < dim : 2 * f < dim) {
        rope_sincos(pos, a.table.freq[f], &cs[i], &sn[i]);
        cs[i] *= a.table.gain, sn[i] *= ROPE == kPartner && !second ? -a.table.gain : a.table.gain;
      }
    }
  }

  const Q8Strides st = tensor ? a.vs : a.ks;
  const T *x0 = static_cast<const T *>(tensor ? a.v : a.k) + b * st.b + (fresh ? tok : 0) * st.t;
  float *scales = tensor ? a.c.vs : a.c.ks;
  bool odd = false;  // an infinity or a NaN
  Piece<T> next;
  if (fresh) next.load(x0 + h0 * st.h + c0, x0 + h0 * st.h + c1);
  for (int h = h0; h < h1; ++h) {
    Piece<T> in = next;
    if (fresh && h + 1 < h1) next.load(x0 + (h + 1) * st.h + c0, x0 + (h + 1) * st.h + c1);
    if (turn && fresh) {
      if constexpr (ROPE == kOwn) {
        if (split) {  // pair i: coordinates i of the two eights
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 u = in.pair(i), v = in.pair(i + 4);
            in.set(i, make_float2(rope_turn(u.x, v.x, cs[2 * i], -sn[2 * i]), rope_turn(u.y, v.y, cs[2 * i + 1], -sn[2 * i + 1])));
            in.set(i + 4, make_float2(rope_turn(v.x, u.x, cs[2 * i], sn[2 * i]), rope_turn(v.y, u.y, cs[2 * i + 1], sn[2 * i + 1])));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (16 * j + 2 * i >= dim) continue;  // past the rotated coordinates
            const float2 u = in.pair(i);
            in.set(i, make_float2(rope_turn(u.x, u.y, cs[i], -sn[i]), rope_turn(u.y, u.x, cs[i], sn[i])));
          }
        }
      } else if constexpr (ROPE == kPartner) {
        // dim is a multiple of 8, so groups of 4 coordinates do not straddle a half
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int i0 = c0 + 4 * g;
          if (i0 < dim) {
            float o[4];
            load_vec<T, 4>(x0 + h * st.h + (i0 < half ? i0 + half : i0 - half), o);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float2 u = in.pair(2 * g + i);
              const int k = 4 * g + 2 * i;
              in.set(2 * g + i, make_float2(rope_turn(u.x, o[2 * i], cs[k], sn[k]), rope_turn(u.y, o[2 * i + 1], cs[k + 1], sn[k + 1])));
            }
          }
        }
      }
    }
    auto block_max = [&](uint32_t v, uint32_t *slot) {
      v = __reduce_max_sync(kFull, v);
      if ((tid & 31) == 0) slot[warp] = v;
      __syncthreads();
      return __reduce_max_sync(kFull, slot[tid & (kThreads / 32 - 1)]);
    };
    uint32_t amax = Piece<T>::float_bits(block_max(fresh ? in.top() : 0u, red[h & 1]));
    const bool wild = amax > __float_as_uint(kQ8Largest);  // the whole CTA's: not finite, or would round up to 2^128
    if (wild) {
      amax = 0;
      if (fresh) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 v = in.pair(i);
          const uint32_t u0 = __float_as_uint(v.x) & 0x7fffffffu, u1 = __float_as_uint(v.y) & 0x7fffffffu;
          odd |= max(u0, u1) >= 0x7f800000u;
          amax = max(amax, u0 >= 0x7f800000u ? 0u : min(u0, __float_as_uint(kQ8Largest)));
          amax = max(amax, u1 >= 0x7f800000u ? 0u : min(u1, __float_as_uint(kQ8Largest)));
        }
      }
      amax = block_max(amax, red[2 + (h & 1)]);
    }
    const long long blk = q8_block(a.c.btab, a.c.pool_blocks, ((long long)b * a.heads + h) * a.c.nblk + blk0, a.error);
    if (blk < 0) continue;
    int e = q8_exponent(amax);
    uint8_t *plane = a.c.records + blk * kQ8BlockBytes + tensor * kQ8Plane;
    int shift = 0;
    if (joins) {
      const int was = log2i(scales[blk]);
      e = max(e, was);
      shift = was - e;
    }
    if (fresh) {
      const float f = pow2i(-e);  // exact: e lies in [-100, 120]
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 u = in.pair(2 * i), v = in.pair(2 * i + 1);
        if (wild) {  // NaN to 0, infinities and what is too large to the largest number that stays finite
          u = make_float2(tame(u.x), tame(u.y)), v = make_float2(tame(v.x), tame(v.y));
        }
        w[i] = cvt_e4m3x2(u.x * f, u.y * f) | (cvt_e4m3x2(v.x * f, v.y * f) << 16);
      }
      if (split) {
        *reinterpret_cast<uint2 *>(plane + q8_off(t, c0)) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2 *>(plane + q8_off(t, c1)) = make_uint2(w[2], w[3]);
      } else {
        *reinterpret_cast<uint4 *>(plane + q8_off(t, c0)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else if (older && shift < 0) {
      const float f = pow2i(max(shift, -126));
      uint4 *piece = reinterpret_cast<uint4 *>(plane + q8_off(t, 16 * j));
      const uint4 w = *piece;
      *piece = make_uint4(e4m3x4_scaled(w.x, f), e4m3x4_scaled(w.y, f), e4m3x4_scaled(w.z, f), e4m3x4_scaled(w.w, f));
    }
    if (joins) __syncthreads();  // every thread has read the old scale
    if (tid == 0) scales[blk] = pow2i(e);
  }
  if (odd) set_error(a.error, TQ_ERR_NONFINITE);
}

template <typename T>
int launch(const Q8AppendArgs &a, int num_sms, cudaStream_t st) {
  const int touched = (int)(((long long)a.n_new + kQ8Block - 2) / kQ8Block + 1);  // blocks n_new slots can lie in
  // Heads per CTA (they share the sines and the CTA's start): as many as leave two CTAs an SM, up to 8. 4 sequences, 8 heads: 64 new
  // tokens 4.3 us at one head, 6.6 at 4; 1024 tokens 13.1 at one, 10.1 at 4; 16384 tokens 174 at one, 96 at 4, 86 at 8.
  const long long ctas = 2LL * touched * a.batch * a.heads;
  long long hpc = (ctas + 2LL * num_sms - 1) / (2LL * num_sms);
  hpc = hpc < 1 ? 1 : hpc > 8 ? 8 : hpc;
  if (hpc > a.heads) hpc = a.heads;
  const long long gz = 2 * ((a.heads + hpc - 1) / hpc);
  if (a.batch > 65535 || gz > 65535) return TQ_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)touched, (unsigned)a.batch, (unsigned)gz);
  auto *kernel = !a.rope ? q8_append_kernel<T, kNone>
                 : a.table.interleaved || a.table.dim % 16 == 0 ? q8_append_kernel<T, kOwn> : q8_append_kernel<T, kPartner>;
  return launch_overlapped(true, kernel, grid, dim3(kThreads), 0, st, a, (int)hpc) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

// One thread per 16 coordinates of a token: code * 2^e, exact.
__global__ void __launch_bounds__(256) q8_dequant_kernel(const __grid_constant__ Q8DequantArgs a, long long items) {
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  if (id >= items) return;
  const int c = (int)(id & 7), n = a.t1 - a.t0;
  const long long row = id >> 3, bh = row / n;
  const int s = a.t0 + (int)(row % n);
  const long long blk = q8_block(a.c.btab, a.c.pool_blocks, bh * a.c.nblk + s / kQ8Block, a.error);
#pragma unroll
  for (int tensor = 0; tensor < 2; ++tensor) {
    float *out = tensor ? a.v : a.k;
    if (!out) continue;
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
    if (blk >= 0) {
      const float f = (tensor ? a.c.vs : a.c.ks)[blk];
      const uint4 w = *reinterpret_cast<const uint4 *>(a.c.records + blk * kQ8BlockBytes + tensor * kQ8Plane +
                                                       q8_off(s % kQ8Block, 16 * c));
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 lo = e4m3x2_f(ww[i] & 0xffffu), hi = e4m3x2_f(ww[i] >> 16);
        v[4 * i] = lo.x * f, v[4 * i + 1] = lo.y * f, v[4 * i + 2] = hi.x * f, v[4 * i + 3] = hi.y * f;
      }
    }
    store_vec<float, 16>(out + row * kD + 16 * c, v);
  }
}

}  // namespace

int launch_q8_append(const Q8AppendArgs &a, int num_sms, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  switch (a.dtype) {
    case TQ_F32: return launch<float>(a, num_sms, st);
    case TQ_BF16: return launch<__nv_bfloat16>(a, num_sms, st);
    default: return launch<__half>(a, num_sms, st);
  }
}

int launch_q8_dequant(const Q8DequantArgs &a, void *stream) {
  const long long items = (long long)a.batch * a.heads * (a.t1 - a.t0) * 8;
  const long long grid = (items + 255) / 256;
  if (grid > 0x7fffffffLL) return TQ_ERR_UNSUPPORTED;
  q8_dequant_kernel<<<(unsigned)grid, 256, 0, (cudaStream_t)stream>>>(a, items);
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // namespace tq
