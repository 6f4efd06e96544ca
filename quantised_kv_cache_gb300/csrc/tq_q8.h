// Declarations shared by the host code and the kernels of the 8-bit cache (TQ_SCHEME_Q8) and of
// rotary positions. Not part of the ABI.
#pragma once

#include <type_traits>

#include "tq_internal.h"

namespace tq {

constexpr int kQ8Block = 64;                   // token slots of a block
constexpr int kQ8Plane = kQ8Block * kD;        // bytes of its key (or value) plane
constexpr int kQ8BlockBytes = 2 * kQ8Plane;
constexpr int kQ8MinExp = -100;                // smallest exponent of a block's scale
constexpr int kQ8MostSlots = 0x7fffffff - 1023;  // of a sequence: the ends of its last block and tile stay within 32 bits

inline int q8_blocks_of(int capacity) { return (capacity + kQ8Block - 1) / kQ8Block; }

// One cache as the kernels see it.
struct Q8Cache {
  uint8_t *records;
  float *ks, *vs;
  const int32_t *btab;  // paged caches (NULL: contiguous)
  int pool_blocks, nblk, capacity;
};

struct Q8Strides {
  long long b, h, t;  // elements
};

struct RotaryArgs {
  const void *x;
  void *y;
  Q8Strides xs, ys;
  int dtype, batch, heads, n, transpose;
  const int32_t *positions;
  RopeTable rope;
  int by_token = 0;  // a token's heads lie nearer to each other than a head's tokens (set by the launcher)
};
int launch_rotary(const RotaryArgs &a, int num_sms, void *stream);

struct Q8AppendArgs {
  Q8Cache c;
  const void *k, *v;
  Q8Strides ks, vs;
  int dtype, batch, heads, n_new, rope;
  const int32_t *seq_lens, *new_lens, *positions;
  int *error;
  RopeTable table;
};
int launch_q8_append(const Q8AppendArgs &a, int num_sms, void *stream);

struct Q8DequantArgs {
  Q8Cache c;
  int batch, heads, t0, t1;
  float *k, *v;  // [batch][heads][t1 - t0][d], either may be NULL
  int *error;
};
int launch_q8_dequant(const Q8DequantArgs &a, void *stream);

struct Q8EvictArgs {
  Q8Cache src, dst;
  int batch, heads, keep, sink, recent;
  const int32_t *seq_lens;
  const float *weights;
  const int32_t *positions;
  int32_t *kept, *dst_lens, *dst_positions;
  float *dst_weights;
  int *error;
};
int launch_q8_evict(const Q8EvictArgs &a, int num_sms, void *stream);

// Attention: the struct of the ABI with its defaults filled in, and the workspace carved up.
struct Q8AttnArgs {
  Q8Cache c;
  int batch, heads_q, heads_kv, group, n_q, max_len;
  int q_dtype, out_dtype;
  const void *q;
  void *out;
  Q8Strides qs, os;
  const int32_t *seq_lens, *new_lens;
  float scale, softcap;
  const float *slopes;
  const int32_t *qpos, *kpos, *kbeg, *kend;
  const float *weights_in;
  float *weights;
  float *lse;   // [batch][heads_q][n_q], natural log (workspace when the caller gives none but the weights need it)
  float *parts; // partial softmax records
  float *scores = nullptr;  // [batch][heads_kv][group x n_q][scores_ld] in log2, kept for the weights (or NULL)
  long long scores_ld = 0;
  int *error;
};
// The workspace with room for all that is worth keeping; *least (if not NULL): what the call cannot do without, which never falls as
// the batch, the query tokens or max_len grow. `weights`: 0 none, 1 with results of either size, 2 with results of 16 bits
size_t q8_attention_workspace(int num_sms, int batch, int heads_q, int heads_kv, int n_q, int max_len, int weights, size_t *least);
// the units and tiles of this call, and the workspace's, fit into the kernels' 32-bit numbers
bool q8_attention_fits(const Q8AttnArgs &a, int num_sms);
bool q8_prompt_fits(const Q8AttnArgs &a, int num_sms);
size_t q8_prompt_workspace(int num_sms, int batch, int group, int n_q);
int launch_q8_prompt(const Q8AttnArgs &a, void *workspace, int num_sms, void *stream);
// `terms`: of the queries, where 16-bit results' scores were not kept
size_t q8_weights_workspace(int num_sms, int batch, int heads_kv, int group, int n_q, int max_len);
int launch_q8_weights(const Q8AttnArgs &a, int terms, void *workspace, int num_sms, void *stream);
int launch_q8_attention(const Q8AttnArgs &a, void *workspace, size_t ws_bytes, int num_sms, void *stream);

}  // namespace tq
