// Host side of the 8-bit cache (TQ_SCHEME_Q8) and of rotary positions: argument checks, the
// rotation's frequencies, dispatch to the launchers.

#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "tq_q8.h"
#include "tq_q8_host.h"

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// arrays of 4-byte numbers (NULL among them)
template <typename... P>
bool aligned4(const P *...p) {
  return ((((uintptr_t)p & 3u) == 0) && ...);
}

int size_of(int dtype) { return dtype == TQ_F32 ? 4 : 2; }

bool known(int dtype) { return dtype == TQ_F32 || dtype == TQ_BF16 || dtype == TQ_F16; }

// strides in elements of `dtype`: every row a multiple of 16 bytes away
bool strides_ok(const int64_t *s, int dtype) {
  for (int i = 0; i < 3; ++i)
    if ((s[i] * size_of(dtype)) % 16) return false;
  return true;
}

// distinct rows lie apart in every dimension (a target is never broadcast)
bool spread(const int64_t *s, int batch, int heads, int n) {
  const int64_t size[3] = {batch, heads, n};
  for (int i = 0; i < 3; ++i)
    if (size[i] > 1 && s[i] > -tq::kD && s[i] < tq::kD) return false;
  return true;
}

tq::Q8Strides strides(const int64_t *s) { return tq::Q8Strides{s[0], s[1], s[2]}; }

tq_status on_device(const tq_ctx *ctx) {
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess) return TQ_ERR_CUDA;
  return cur == ctx->device ? TQ_OK : TQ_ERR_ARG;
}

// Caps of scores: from kNoCap on cap tanh(t / cap) is t to its last bit below 2^28; a smaller one than kLeastCap has no reciprocal
// beside a large scale.
constexpr float kNoCap = 1099511627776.f, kLeastCap = 8.6736174e-19f;  // 2^40, 2^-60

typedef __int128 wide;

// Rows of `row` bytes at p + i stride[0] + j stride[1] + k stride[2], i < size[0] and so on.
struct Region {
  const void *p;
  wide stride[3];
  int64_t size[3], row;
};
Region rows(const void *p, const int64_t *s, int dtype, int batch, int heads, int n) {
  const int e = size_of(dtype);
  return Region{p, {(wide)s[0] * e, (wide)s[1] * e, (wide)s[2] * e}, {batch, heads, n}, (int64_t)tq::kD * e};
}
// contiguous bytes (none for NULL)
Region bytes(const void *p, size_t n) { return Region{p, {0, 0, 0}, {1, 1, 1}, p ? (int64_t)n : 0}; }

// The first byte's offset from p and the length of the rows along those dimensions whose stride is no multiple of `period`
// (0: along all of them).
void extent(const Region &r, wide period, wide *first, wide *length) {
  *first = 0, *length = r.row;
  for (int i = 0; i < 3; ++i) {
    if (r.size[i] <= 1 || (period && r.stride[i] % period == 0)) continue;
    const wide d = r.stride[i] * (r.size[i] - 1);
    *length += d < 0 ? -d : d;
    if (d < 0) *first += d;
  }
}

// False when the regions share no byte: their extents lie apart, or the parts of them that repeat at one of their strides do (a
// fused projection's queries and keys, say). True for regions that share one, and for those that neither test can tell.
bool overlap(const Region &a, const Region &b) {
  if (!a.row || !b.row) return false;
  const wide apart = (wide)(uintptr_t)b.p - (wide)(uintptr_t)a.p;
  for (int k = -1; k < 6; ++k) {
    const Region &r = k < 3 ? a : b;
    wide period = 0, a0, b0, na, nb;
    if (k >= 0) {
      period = r.size[k % 3] > 1 ? r.stride[k % 3] : 0;
      if (period == 0) continue;
      if (period < 0) period = -period;
    }
    extent(a, period, &a0, &na);
    extent(b, period, &b0, &nb);
    wide d = apart + b0 - a0;  // from a's first byte to b's
    if (period == 0) {
      if (d >= na || -d >= nb) return false;
      continue;
    }
    d %= period;
    if (d < 0) d += period;
    if (d >= na && period - d >= nb) return false;
  }
  return true;
}

// A buffer that is updated in place, or regions that lie apart.
bool same_or_apart(const Region &a, const Region &b) { return a.p == b.p || !overlap(a, b); }

// Numbers of about 106 bits, as sums of two doubles (Dekker, "A floating-point technique for extending the available precision",
// 1971; Knuth's two-sum): a frequency is needed to 2^-64 turns.
struct Long {
  double hi, lo;
};
Long two_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
Long operator+(Long a, Long b) {
  const Long s = two_sum(a.hi, b.hi);
  return two_sum(s.hi, s.lo + a.lo + b.lo);
}
Long operator-(Long a, Long b) { return a + Long{-b.hi, -b.lo}; }
Long operator*(Long a, Long b) {
  const double p = a.hi * b.hi;
  return two_sum(p, std::fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
Long operator/(Long a, Long b) {
  const double q = a.hi / b.hi;
  const Long r = a - Long{q, 0.0} * b;
  const double q1 = r.hi / b.hi;
  const Long r1 = r - Long{q1, 0.0} * b;
  return two_sum(q, q1) + Long{r1.hi / b.hi, 0.0};
}
Long power(Long x, int n) {
  Long y{1.0, 0.0};
  for (; n; n >>= 1, x = x * x)
    if (n & 1) y = y * x;
  return y;
}

}  // namespace

namespace tq {

tq_status q8_check_cache(const tq_ctx *ctx, const tq_cache *c, int batch, int heads_kv) {
  if (ctx->scheme != TQ_SCHEME_Q8) return TQ_ERR_STATE;
  if (!c || c->batch != batch || c->heads_kv != heads_kv || c->capacity <= 0) return TQ_ERR_ARG;
  if (c->capacity > kQ8MostSlots) return TQ_ERR_UNSUPPORTED;
  if (!c->records || !c->k_stats || !c->v_stats) return TQ_ERR_ARG;
  if (!aligned16(c->records) || !aligned16(c->k_stats) || !aligned16(c->v_stats)) return TQ_ERR_ALIGN;
  if (c->block_table && c->pool_blocks <= 0) return TQ_ERR_ARG;
  if (!aligned4(c->block_table)) return TQ_ERR_ALIGN;
  return TQ_OK;
}

Q8Cache q8_cache(const tq_cache *c) {
  return Q8Cache{c->records, (float *)c->k_stats, (float *)c->v_stats, c->block_table, c->pool_blocks,
                 q8_blocks_of(c->capacity), c->capacity};
}

void q8_cache_sizes(int batch, int heads_kv, int capacity, tq_cache_sizes *out) {
  const size_t blocks = (size_t)batch * heads_kv * q8_blocks_of(capacity);
  out->block_bytes = kQ8BlockBytes;
  out->records = blocks * kQ8BlockBytes;
  out->k_stats = out->v_stats = blocks * sizeof(float);
  out->record_bytes = 2 * kD;
}

}  // namespace tq

extern "C" {

tq_status tq_set_rope(tq_ctx *ctx, const tq_rope *r) {
  if (!ctx || !r) return TQ_ERR_ARG;
  if (r->dim < 8 || r->dim > ctx->d || r->dim % 8) return TQ_ERR_ARG;
  if (!(r->base > 1.0) || !std::isfinite(r->base) || !(r->factor >= 1.0) || !std::isfinite(r->factor) ||
      !(r->gain > 0.0) || !std::isfinite(r->gain) || !std::isfinite(r->low) || !std::isfinite(r->high))
    return TQ_ERR_ARG;
  const bool even = r->low == 0.0 && r->high == 0.0;  // every pair divided by the factor
  if (r->factor > 1.0 && !even && (!(r->original_len > 0.0) || !std::isfinite(r->original_len) || !(r->high > r->low) || !std::isfinite(r->high - r->low)))
    return TQ_ERR_ARG;
  tq::RopeTable t;
  t.dim = r->dim;
  t.interleaved = r->interleaved ? 1 : 0;
  t.gain = (float)r->gain;
  const Long two_pi{6.283185307179586, 2.4492935982947064e-16}, one{1.0, 0.0};
  // f_1 = base^(-2 / dim) by a step of Newton's for f_1^(dim / 2) = 1 / base from its double; the others are its powers
  const int pairs = r->dim / 2;
  const Long guess{std::pow(r->base, -1.0 / pairs), 0.0}, there = power(guess, pairs);
  const Long ratio = guess + guess * (one / Long{r->base, 0.0} - there) / (there * Long{(double)pairs, 0.0});
  Long f{1.0, 0.0};
  for (int i = 0; i < pairs; ++i, f = f * ratio) {
    Long g = f;
    if (r->factor > 1.0) {
      Long keep{0.0, 0.0};
      if (!even) {
        const double about = (r->original_len * f.hi / two_pi.hi - r->low) / (r->high - r->low);  // (may be infinite)
        if (about > -1.0 && about < 2.0) keep = (Long{r->original_len, 0.0} * f / two_pi - Long{r->low, 0.0}) / two_sum(r->high, -r->low);
        else keep.hi = about;
        keep = keep.hi < 0.0 ? Long{0.0, 0.0} : keep.hi >= 1.0 ? one : keep;
      }
      g = (one - keep) * f / Long{r->factor, 0.0} + keep * f;
    }
    const Long turns = g / two_pi;  // at most 1 / (2 pi)
    const double hi = std::ldexp(turns.hi, 64), whole = std::floor(hi);
    t.freq[i] = (unsigned long long)whole + (unsigned long long)std::llrint(hi - whole + std::ldexp(turns.lo, 64));
  }
  ctx->rope = t;
  return TQ_OK;
}

tq_status tq_rotary(const tq_ctx *ctx, const void *d_x, const int64_t *x_strides, void *d_y, const int64_t *y_strides,
                    int dtype, int batch, int heads, int n, const int32_t *d_positions, int transpose, void *stream) {
  if (!ctx || !x_strides || !y_strides) return TQ_ERR_ARG;
  if (!known(dtype) || batch <= 0 || heads <= 0 || n < 0 || (transpose != 0 && transpose != 1)) return TQ_ERR_ARG;
  if (!ctx->rope.dim) return TQ_ERR_STATE;
  if (n == 0) return on_device(ctx);  // no vectors, which then have no addresses
  if (!d_x || !d_y || !d_positions) return TQ_ERR_ARG;
  if (!aligned16(d_x) || !aligned16(d_y) || !aligned4(d_positions) || !strides_ok(x_strides, dtype) || !strides_ok(y_strides, dtype))
    return TQ_ERR_ALIGN;
  if (!spread(y_strides, batch, heads, n)) return TQ_ERR_ARG;
  if (!(d_x == d_y && !std::memcmp(x_strides, y_strides, 3 * sizeof(int64_t))) &&
      overlap(rows(d_x, x_strides, dtype, batch, heads, n), rows(d_y, y_strides, dtype, batch, heads, n)))
    return TQ_ERR_ARG;
  const tq_status s = on_device(ctx);
  if (s != TQ_OK) return s;
  const tq::RotaryArgs a{d_x, d_y, strides(x_strides), strides(y_strides), dtype, batch, heads, n, transpose,
                         d_positions, ctx->rope};
  return (tq_status)tq::launch_rotary(a, ctx->num_sms, stream);
}

tq_status tq_q8_append(const tq_ctx *ctx, const tq_cache *cache, const void *d_k, const int64_t *k_strides,
                       const void *d_v, const int64_t *v_strides, int dtype, int batch, int heads_kv, int n_new,
                       const int32_t *d_seq_lens, const int32_t *d_new_lens, int rope, const int32_t *d_positions,
                       void *stream) {
  if (!ctx || !k_strides || !v_strides || !d_seq_lens) return TQ_ERR_ARG;
  if (!known(dtype) || batch <= 0 || heads_kv <= 0 || n_new < 0 || (rope != 0 && rope != 1)) return TQ_ERR_ARG;
  tq_status s = tq::q8_check_cache(ctx, cache, batch, heads_kv);
  if (s != TQ_OK) return s;
  if (rope && !ctx->rope.dim) return TQ_ERR_STATE;
  if (n_new == 0) return on_device(ctx);
  if (!d_k || !d_v) return TQ_ERR_ARG;
  if (!aligned16(d_k) || !aligned16(d_v) || !aligned4(d_seq_lens, d_new_lens, d_positions) || !strides_ok(k_strides, dtype) ||
      !strides_ok(v_strides, dtype))
    return TQ_ERR_ALIGN;
  if ((s = on_device(ctx)) != TQ_OK) return s;
  const tq::Q8AppendArgs a{tq::q8_cache(cache), d_k, d_v, strides(k_strides), strides(v_strides), dtype, batch, heads_kv,
                           n_new, rope, d_seq_lens, d_new_lens, d_positions, &ctx->dparams->error, ctx->rope};
  return (tq_status)tq::launch_q8_append(a, ctx->num_sms, stream);
}

tq_status tq_q8_attention_workspace(const tq_ctx *ctx, int batch, int heads_q, int heads_kv, int n_q, int max_len,
                                    int weights, size_t *out) {
  if (!ctx || !out || batch <= 0 || heads_q <= 0 || heads_kv <= 0 || heads_q % heads_kv || n_q <= 0 || max_len <= 0 ||
      weights < 0 || weights > 2)
    return TQ_ERR_ARG;
  if (ctx->scheme != TQ_SCHEME_Q8) return TQ_ERR_STATE;
  *out = tq::q8_attention_workspace(ctx->num_sms, batch, heads_q, heads_kv, n_q, max_len, weights, nullptr);
  return TQ_OK;
}

tq_status tq_q8_attention(const tq_ctx *ctx, const tq_cache *cache, const tq_q8_attn *p, void *d_workspace,
                          size_t ws_bytes, void *stream) {
  if (!ctx || !p || !p->d_q || !p->d_out || !p->d_seq_lens || !d_workspace) return TQ_ERR_ARG;
  if (p->batch <= 0 || p->heads_q <= 0 || p->heads_kv <= 0 || p->heads_q % p->heads_kv || p->n_q <= 0 || p->max_len <= 0)
    return TQ_ERR_ARG;
  if (!known(p->q_dtype) || (p->out_dtype != p->q_dtype && p->out_dtype != TQ_F32)) return TQ_ERR_ARG;
  if (!std::isfinite(p->scale) || !std::isfinite(p->softcap)) return TQ_ERR_ARG;
  if (p->softcap != 0.f && !(p->softcap >= kLeastCap)) return TQ_ERR_ARG;  // (negative ones among them)
  if (p->d_k_positions && !p->d_q_positions) return TQ_ERR_ARG;  // a distance needs both on one scale
  if (p->d_weights_in && !p->d_weights) return TQ_ERR_ARG;
  tq_status s = tq::q8_check_cache(ctx, cache, p->batch, p->heads_kv);
  if (s != TQ_OK) return s;
  if (p->max_len > cache->capacity) return TQ_ERR_ARG;
  if (!aligned16(p->d_q) || !aligned16(p->d_out) || !aligned16(d_workspace) || !strides_ok(p->q_strides, p->q_dtype) ||
      !strides_ok(p->out_strides, p->out_dtype) ||
      !aligned4(p->d_seq_lens, p->d_new_lens, p->d_slopes, p->d_q_positions, p->d_k_positions, p->d_key_begin, p->d_key_end, p->d_weights_in,
                p->d_weights, p->d_lse))
    return TQ_ERR_ALIGN;
  size_t least = 0;
  tq::q8_attention_workspace(ctx->num_sms, p->batch, p->heads_q, p->heads_kv, p->n_q, p->max_len, p->d_weights != nullptr, &least);
  if (ws_bytes < least) return TQ_ERR_WORKSPACE;
  if (!spread(p->out_strides, p->batch, p->heads_q, p->n_q)) return TQ_ERR_ARG;
  const Region q = rows(p->d_q, p->q_strides, p->q_dtype, p->batch, p->heads_q, p->n_q);
  const Region out = rows(p->d_out, p->out_strides, p->out_dtype, p->batch, p->heads_q, p->n_q);
  const size_t slots = (size_t)p->batch * p->heads_kv * cache->capacity * sizeof(float);
  const Region weights = bytes(p->d_weights, slots), lse = bytes(p->d_lse, (size_t)p->batch * p->heads_q * p->n_q * sizeof(float));
  // (the queries are read again, for the weights, after the results are written)
  if (overlap(q, out) || overlap(q, weights) || overlap(q, lse) || overlap(out, weights) || overlap(out, lse) || overlap(weights, lse) ||
      !same_or_apart(weights, bytes(p->d_weights_in, slots)))
    return TQ_ERR_ARG;
  tq::Q8AttnArgs a{};
  a.c = tq::q8_cache(cache);
  a.batch = p->batch, a.heads_q = p->heads_q, a.heads_kv = p->heads_kv, a.group = p->heads_q / p->heads_kv;
  a.n_q = p->n_q, a.max_len = p->max_len, a.q_dtype = p->q_dtype, a.out_dtype = p->out_dtype;
  a.q = p->d_q, a.out = p->d_out, a.qs = strides(p->q_strides), a.os = strides(p->out_strides);
  a.seq_lens = p->d_seq_lens, a.new_lens = p->d_new_lens;
  a.scale = p->scale != 0.f ? p->scale : 0.08838834764831845f;  // 1 / sqrt(128)
  a.softcap = p->softcap < kNoCap ? p->softcap : 0.f, a.slopes = p->d_slopes, a.qpos = p->d_q_positions, a.kpos = p->d_k_positions;
  a.kbeg = p->d_key_begin, a.kend = p->d_key_end;
  a.weights_in = p->d_weights_in, a.weights = p->d_weights, a.lse = p->d_lse;
  if (!tq::q8_attention_fits(a, ctx->num_sms)) return TQ_ERR_UNSUPPORTED;
  if ((s = on_device(ctx)) != TQ_OK) return s;
  a.error = &ctx->dparams->error;
  return (tq_status)tq::launch_q8_attention(a, d_workspace, ws_bytes, ctx->num_sms, stream);
}

tq_status tq_q8_evict(const tq_ctx *ctx, const tq_cache *src, const tq_cache *dst, int batch, int heads_kv,
                      const int32_t *d_seq_lens, const float *d_weights, int keep, int sink, int recent,
                      const int32_t *d_positions, int32_t *d_kept, int32_t *d_dst_lens, float *d_dst_weights,
                      int32_t *d_dst_positions, void *stream) {
  if (!ctx || !d_seq_lens || !d_weights || !d_kept || !d_dst_lens || batch <= 0 || heads_kv <= 0) return TQ_ERR_ARG;
  tq_status s = tq::q8_check_cache(ctx, src, batch, heads_kv);
  if (s == TQ_OK) s = tq::q8_check_cache(ctx, dst, batch, heads_kv);
  if (s != TQ_OK) return s;
  if (keep <= 0 || sink < 0 || recent < 0 || (long long)sink + recent > keep || keep > dst->capacity) return TQ_ERR_ARG;
  if (!aligned4(d_seq_lens, d_weights, d_positions, d_kept, d_dst_lens, d_dst_weights, d_dst_positions)) return TQ_ERR_ALIGN;
  const size_t grid = (size_t)batch * heads_kv;
  const size_t sn = src->block_table ? (size_t)src->pool_blocks : grid * tq::q8_blocks_of(src->capacity);
  const size_t dn = dst->block_table ? (size_t)dst->pool_blocks : grid * tq::q8_blocks_of(dst->capacity);
  if (overlap(bytes(src->records, sn * tq::kQ8BlockBytes), bytes(dst->records, dn * tq::kQ8BlockBytes)) ||
      overlap(bytes(src->k_stats, sn * 4), bytes(dst->k_stats, dn * 4)) || overlap(bytes(src->v_stats, sn * 4), bytes(dst->v_stats, dn * 4)))
    return TQ_ERR_ARG;
  const Region lens = bytes(d_seq_lens, batch * sizeof(int32_t));
  const Region in[] = {lens, bytes(d_weights, grid * src->capacity * 4), bytes(d_positions, grid * src->capacity * 4)};
  const Region outs[] = {bytes(d_dst_lens, batch * sizeof(int32_t)), bytes(d_kept, grid * keep * 4),
                         bytes(d_dst_weights, grid * dst->capacity * 4), bytes(d_dst_positions, grid * dst->capacity * 4)};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 3; ++j)
      if (i == 0 && j == 0 ? !same_or_apart(outs[i], in[j]) : overlap(outs[i], in[j])) return TQ_ERR_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return TQ_ERR_ARG;
  }
  if ((s = on_device(ctx)) != TQ_OK) return s;
  const tq::Q8EvictArgs a{tq::q8_cache(src), tq::q8_cache(dst), batch, heads_kv, keep, sink, recent, d_seq_lens,
                          d_weights, d_positions, d_kept, d_dst_lens, d_dst_positions, d_dst_weights,
                          &ctx->dparams->error};
  return (tq_status)tq::launch_q8_evict(a, ctx->num_sms, stream);
}

}  // extern "C"
