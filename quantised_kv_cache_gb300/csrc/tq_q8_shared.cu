// Attention of a batch behind a shared prefix in a cache of its own (tq_q8_shared_attention).
//
// out = (X1 + X2) / (l1 + l2): the rows' sums over the prefix, X1 = sum 2^(t - m) v and l1 = sum 2^(t - m), then those over the sequence's own
// tokens, on one reference. Over the prefix the rows of all sequences are the rows of one (its head's, batch x query tokens x
// group of them), so that its keys and values are read once for every 256 of them (32-bit results: 8). Their parts go to the workspace,
// where the kernels of the own tokens fetch them as they finish a row: no pass of its own joins them. 64 sequences of up to 2048 tokens behind
// 32768, 8 KV heads of 4 rows, bf16: 109 us (cold and one after the other: plan 5.5, the prefix's tiles 54.7, their join 12.6, the own tokens
// 33.5, their join 5.7; the prefix's bytes would take 10, the own tokens' 20). Each sequence over a cache of its own with the prefix in it: 64 times
// its bytes, 640 us at the copy's rate. 32-bit results: 490 us, 438 of them the prefix, 32 units of 8 rows that each read it (from L2 for the most part).

#include "tq_q8_solo.cuh"

namespace tq {

static bool takes_few(long long rows, int out_dtype) { return rows <= kFewRows || out_dtype == TQ_F32; }

static size_t prior_bytes(int batch, int heads_q, int n_q) { return (size_t)heads_q * batch * n_q * kPriorRow * sizeof(float); }

size_t q8_shared_workspace(int num_sms, int batch, int heads_q, int heads_kv, int n_q) {
  const int group = heads_q / heads_kv;
  // (the prefix's rows are one sequence's; their units are no more than the sequences')
  const size_t many = (long long)group * n_q * batch <= kFewRows ? 0 : q8_prompt_workspace(num_sms, batch, group, n_q);
  return prior_bytes(batch, heads_q, n_q) + std::max({few_bytes(num_sms), solo_bytes(num_sms), many});
}

// Sequences whose rows fill units of their own (up to a quarter of them empty) take one pass over the prefix and their own tokens: each reads
// the prefix for itself, but nothing passes through memory. 4 sequences of 512 tokens x 4 heads behind 8192 tokens: 341 us, 399 in two passes.
static bool takes_both(long long rows, int out_dtype) {
  const long long padded = rows <= 128 ? 128 : (rows + 255) / 256 * 256;
  return !takes_few(rows, out_dtype) && 4 * padded <= 5 * rows;
}

static Q8AttnArgs of_both(const Q8AttnArgs &own, const Q8Cache &prefix) {
  Q8AttnArgs a = own;
  a.pc = prefix;
  return a;
}

static Q8AttnArgs of_prefix(const Q8AttnArgs &own, const Q8Cache &prefix) {
  Q8AttnArgs a = own;
  a.c = prefix, a.batch = 1, a.n_q = own.batch * own.n_q, a.max_len = own.max_prefix, a.fold = own.n_q, a.own_max = own.max_len;
  return a;
}

bool q8_shared_fits(const Q8AttnArgs &own, int num_sms) {
  if ((long long)own.group * own.n_q * own.batch > 0x7fffffff - 1023) return false;         // rows of the prefix's KV head
  if ((long long)own.max_prefix + own.max_len > kQ8MostSlots) return false;                 // slots of a sequence
  if (takes_both((long long)own.group * own.n_q, own.out_dtype)) return q8_both_many_fits(of_both(own, own.c), num_sms);
  const Q8AttnArgs pre = of_prefix(own, own.c);
  return (takes_few((long long)pre.group * pre.n_q, own.out_dtype) || q8_prefix_many_fits(pre, num_sms)) &&
         (takes_few((long long)own.group * own.n_q, own.out_dtype) || q8_own_many_fits(own, num_sms));
}

template <int KIND>
static int launch_part(const Q8AttnArgs &a, char *w, int num_sms, void *stream, int (*many)(const Q8AttnArgs &, void *, int, void *)) {
  const long long rows = (long long)a.group * a.n_q, unit = rows_of(a.out_dtype == TQ_F32 ? 8 : 4), units = (rows + unit - 1) / unit;
  const long long tiles = (a.max_len + kTile - 1) / kTile;
  if (!takes_few(rows, a.out_dtype) && !team_takes<KIND>(a, rows, 1, tiles, num_sms)) return many(a, w, num_sms, stream);
  if constexpr (KIND == kOwn)
    if (solo_wins(a, 1, num_sms)) return launch_solo<KIND>(a, (int)rows, 1, tiles, w, num_sms, (cudaStream_t)stream);
  return launch_few<KIND>(a, (int)std::min(rows, 1024ll), units, tiles, w, num_sms, (cudaStream_t)stream);
}

int launch_q8_shared(const Q8AttnArgs &args, const Q8Cache &prefix, void *workspace, int num_sms, void *stream) {
  Q8AttnArgs own = args;
  if (takes_both((long long)own.group * own.n_q, own.out_dtype)) return launch_q8_both_many(of_both(own, prefix), workspace, num_sms, stream);
  own.prior = (float *)workspace;
  char *w = (char *)workspace + prior_bytes(own.batch, own.heads_q, own.n_q);
  const int s = launch_part<kPrefix>(of_prefix(own, prefix), w, num_sms, stream, launch_q8_prefix_many);
  return s != TQ_OK ? s : launch_part<kOwn>(own, w, num_sms, stream, launch_q8_own_many);
}

}  // namespace tq
