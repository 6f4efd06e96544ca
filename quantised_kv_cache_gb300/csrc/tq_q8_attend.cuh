// Device code shared by the attention kernels of the 8-bit cache: tensor-core issue on e4m3 / e5m2
// operands, the expansion of a number into 8-bit terms, and the score of one (query, key) pair.
//
// The cache's codes go to the tensor cores as they lie (tcgen05.mma kind::f8f6f4: fp8 products are
// exact, sums are fp32). The other operand, queries and probabilities, is a sum of 8-bit terms on one
// scale, each the number nearest to what the ones before have left:
//  - few rows: e5m2 terms (3 significant bits each, down to 2^-16) with a row's largest magnitude near 2^15, so that T
//    terms leave 2^-3T of any number that is not 2^-32 of the largest. The terms of all rows lie side by side
//    in one operand: its N is small whatever T, and an MMA of so few columns takes the time of its other operand.
//  - many rows: e4m3 terms (4 bits each, down to 2^-9), two of them, or a third in e5m2, with the largest in [128, 256):
//    2^-8 (2^-11) of numbers from 2^-2 on, 2^-10 (2^-13) below. Each is one more pass over the same accumulator.
#pragma once

#include "tq_q8.cuh"
#include "tq_tcgen05.cuh"

namespace tq {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Instruction descriptor of kind::f8f6f4, fp32 accumulate: A e4m3, B e4m3 (0) or e5m2 (1); `a_mn`, `b_mn`: the
// operand is MN-major. Fields as in tc_idesc_f16_f32, formats 0 = e4m3, 1 = e5m2.
__host__ __device__ constexpr uint32_t tc_idesc_f8(int M, int N, int a_fmt, int b_fmt, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_fmt << 7) | ((uint32_t)b_fmt << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// MMAs are issued by a whole warp in uniform control flow, one elected lane of which executes them, with descriptors
// from values the compiler knows to be the same in every lane: those stay in uniform registers, where the
// instruction takes them from. Issued in a branch of one thread each MMA cost about 200 clocks to set up (measured for a
// chain of 128 x 128 x 32 products), so 66, their own time.
__device__ __forceinline__ uint32_t warp_uniform(uint32_t x) { return __shfl_sync(kFull, x, 0); }
__device__ __forceinline__ bool elect_lane() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// D (TMEM) (+)= A (shared) x B (shared) of 8-bit operands, 32 K-elements; executed by one lane.
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// After a wait that ran out: time for the tensor-core operations in flight to end (they take microseconds) before tensor
// memory is given back.
__device__ __forceinline__ void settle() {
  const uint64_t t0 = global_ns();
  while (global_ns() - t0 < 2000000ull) __nanosleep(10000);
}

// N consecutive columns of this thread's lane.
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&f)[N]) {
  uint32_t v[N];
  if constexpr (N == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(taddr) : "memory");
  } else if constexpr (N == 8) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
        : "r"(taddr) : "memory");
  } else if constexpr (N == 32) {
    tmem_ld_x32(taddr, v);
  } else {
    static_assert(N == 16, "");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr) : "memory");
  }
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = __uint_as_float(v[i]);
}

// The three terms (e4m3, e4m3, e5m2) of (a, b), each a pair of bytes (a's low).
__device__ __forceinline__ void split_terms(float a, float b, uint32_t (&term)[3]) {
  term[0] = cvt_e4m3x2(a, b);
  float2 f = e4m3x2_f(term[0]);
  a -= f.x, b -= f.y;
  term[1] = cvt_e4m3x2(a, b);
  f = e4m3x2_f(term[1]);
  term[2] = cvt_e5m2x2(a - f.x, b - f.y);
}
// T e5m2 terms; a and b become what is left.
template <int T>
__device__ __forceinline__ void split_e5m2(float &a, float &b, uint32_t (&term)[T]) {
#pragma unroll
  for (int k = 0; k < T; ++k) {
    term[k] = cvt_e5m2x2(a, b);
    const uint32_t h = __byte_perm(term[k], 0, 0x1404);  // an e5m2 number is the upper byte of the fp16 one
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    a -= f.x, b -= f.y;
  }
}

__device__ __forceinline__ float warp_fmax(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// A row's power of two e: |x| 2^-e in [2^top, 2^(top + 1)) for its largest |x|.
__device__ __forceinline__ int row_exponent(uint32_t amax_bits, int top) {
  const int e = (int)(amax_bits >> 23) - 127 - top;
  return max(e, -120);
}

// log2(e) times the scaled and capped product q.k (the bias comes on top).
struct Q8Score {
  float scale, softcap, inv_cap;  // softcap 0: none
};
__device__ __forceinline__ float q8_score_log2(float qk, const Q8Score &s) {
  float x = qk * s.scale;
  if (s.softcap != 0.f) x = s.softcap * tanhf(x * s.inv_cap);
  return x * kLog2e;
}

// scale (times a row's and a block's) x, capped, in log2 units: cap tanh(y) with tanh = 1 - 2 / (1 + e^2y), off by less than 2^-21 of the
// cap; an infinite e^2y gives 1, a zero one -1. `in` and `cap` from score_cap.
struct ScoreCap {
  float in, cap;  // cap 0: none
};
__device__ __forceinline__ ScoreCap score_cap(float scale, float softcap) {
  return softcap == 0.f ? ScoreCap{scale * kLog2e, 0.f} : ScoreCap{scale * (2.f * kLog2e) / softcap, softcap * kLog2e};
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// x times c, which holds in. LONG, for caps above kShortCap, where a few 2^-24 of the cap would show: below |y| = 1/4 the Taylor series of
// tanh (the next term is below 2^-26 of it), so that a score is off by less than 2^-19 of itself.
constexpr float kShortCap = 128.f;
// What kernels for many rows do to scores (a kernel each: where one branched on the cap, caps below took 2 % longer): nothing, a cap or a
// bias, a cap above kShortCap (and perhaps a bias).
enum Extra { kPlain = 0, kCapOrBias = 1, kLongCaps = 2 };
template <bool LONG>
__device__ __forceinline__ float capped_log2(float x, float c, float cap) {
  const float u = x * c;
  if (!LONG && cap == 0.f) return u;
  const float far = fmaf(-2.f * cap, rcp_approx(1.f + ex2_approx(u)), cap);
  if (!LONG) return far;
  const float y = u * (0.5f * kLn2), z = y * y;
  float s = fmaf(z, 2.1869489e-2f, -5.3968254e-2f);
  s = fmaf(z, s, 1.3333333e-1f);
  s = fmaf(z, s, -3.3333333e-1f);
  return fabsf(y) < 0.25f ? cap * fmaf(y * z, s, y) : far;
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 16 columns of this thread's lane on their way to v, and the wait for them (and any others): v may be used after it. A
// loop loads the next 16 after waiting for these, so that they arrive while these are worked on.
__device__ __forceinline__ void tmem_ld_start(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_done(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                 "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}

}  // namespace tq
