// Attention over the 8-bit cache (tq_q8_attention): which kernel takes a call, and its workspace.

#include "tq_q8_few.cuh"

namespace tq {
namespace {

// The scores of up to 64 rows that this kernel forms (no more bytes than the cache that they come from) are kept for the weights where they
// fit into a GB and into the workspace; else they are formed again. 16 sequences of 16384 tokens, 8 KV heads, 4 rows: 111 us kept, 706
// formed again.
constexpr long long kKeptRows = 64;
constexpr size_t kScoreBytes = size_t(1) << 30;
size_t score_bytes(int batch, int heads_q, long long rows, int n_q, int max_len, bool half) {
  const size_t n = (size_t)batch * heads_q * n_q * ((max_len + kTile - 1) / kTile * kTile) * sizeof(float);
  return rows <= (half ? kFewRows : kKeptRows) && n <= kScoreBytes ? n : 0;
}
}  // namespace

// Workspace: for the weights the log-sums; then, where they are kept, the scores; then either kernel's records (few rows: cuts and parts),
// in whose place the weights' row tiles come.
size_t lse_bytes(int batch, int heads_q, int n_q) { return round16((size_t)batch * heads_q * n_q * sizeof(float)); }
size_t q8_attention_workspace(int num_sms, int batch, int heads_q, int heads_kv, int n_q, int max_len, int weights, size_t *least) {
  const int group = heads_q / heads_kv;
  const long long R = (long long)group * n_q;
  const size_t lse = weights ? lse_bytes(batch, heads_q, n_q) : 0;
  const size_t many = R <= kFewRows ? 0 : q8_prompt_workspace(num_sms, batch, group, n_q);
  const size_t tiles = weights ? q8_weights_workspace(num_sms, batch, heads_kv, group, n_q, max_len) : 0;
  const size_t scores = weights ? score_bytes(batch, heads_q, R, n_q, max_len, weights == 2) : 0;
  const size_t need = lse + std::max({few_bytes(num_sms), many, tiles});
  if (least) *least = need;
  return scores ? std::max(need, lse + scores + few_bytes(num_sms)) : need;
}

static bool few_rows(const Q8AttnArgs &a) { return (long long)a.group * a.n_q <= kFewRows || a.out_dtype == TQ_F32; }

bool q8_attention_fits(const Q8AttnArgs &a, int num_sms) {
  if ((long long)a.group * a.n_q > 0x7fffffff - 1023) return false;                // a KV head's rows
  if (a.weights && (a.heads_kv > 65535 || a.batch > 65535)) return false;          // grid dimensions of the weights' launches
  return few_rows(a) || q8_prompt_fits(a, num_sms);
}

int launch_q8_attention(const Q8AttnArgs &args, void *workspace, size_t ws_bytes, int num_sms, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  Q8AttnArgs a = args;
  const long long R = (long long)a.group * a.n_q;
  const bool few = few_rows(a);
  char *w = (char *)workspace;
  if (a.weights) {
    if (!a.lse) a.lse = (float *)w;
    const size_t lse = lse_bytes(a.batch, a.heads_q, a.n_q), scores = few ? score_bytes(a.batch, a.heads_q, R, a.n_q, a.max_len, false) : 0;
    w += lse;
    if (scores && ws_bytes >= lse + scores + few_bytes(num_sms)) {
      a.scores = (float *)w, a.scores_ld = (a.max_len + kTile - 1) / kTile * kTile;
      w += scores;
    }
  }
  if (!few) {  // rows as lanes
    const int s = launch_q8_prompt(a, w, num_sms, stream);
    if (s != TQ_OK) return s;
  } else {
    const int unit = rows_of(a.out_dtype == TQ_F32 ? 8 : 4);
    const int s = launch_few<kWhole>(a, (int)std::min(R, 1024ll), (R + unit - 1) / unit, (a.max_len + kTile - 1) / kTile, w, num_sms, st);
    if (s != TQ_OK) return s;
  }
  // the attention's records are read by now: their place serves the weights
  return a.weights ? launch_q8_weights(a, few || a.q_dtype != TQ_BF16 ? 3 : 2, w, num_sms, stream) : TQ_OK;
}

}  // namespace tq
