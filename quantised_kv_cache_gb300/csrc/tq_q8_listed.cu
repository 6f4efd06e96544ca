// Attention over listed blocks of the 8-bit cache (tq_q8_sparse_attention): the kernel for few rows, and which kernel takes a call.
// A tile of 128 tokens is two blocks of a list; everything else is as over a whole cache (tq_q8_few.cuh, tq_q8_many.cuh).

#include "tq_q8_solo.cuh"

namespace tq {

static bool listed_few(int group, int span, int out_dtype) { return (long long)group * span <= kFewRows || out_dtype == TQ_F32; }

size_t q8_listed_workspace(int num_sms, int batch, int group, int n_q, int span) {
  span = std::min(span, n_q);
  const size_t few = std::max(few_bytes(num_sms), solo_bytes(num_sms));
  return listed_few(group, span, TQ_BF16) ? few : std::max(few, q8_listed_many_workspace(num_sms, batch, group, n_q, span));
}

bool q8_listed_fits(const Q8AttnArgs &a) {
  if ((long long)a.group * a.n_q > 0x7fffffff - 1023) return false;  // a KV head's rows
  return listed_few(a.group, a.span, a.out_dtype) || q8_listed_many_fits(a);
}

int launch_q8_listed(const Q8AttnArgs &a, void *workspace, int num_sms, void *stream) {
  const long long rows = (long long)a.group * a.span, unit = rows_of(a.out_dtype == TQ_F32 ? 8 : 4), units = (rows + unit - 1) / unit * a.lists;
  const long long tiles = (std::min(a.n_blocks, a.c.nblk) + 1) / 2;
  if (!listed_few(a.group, a.span, a.out_dtype) && !team_takes<kListed>(a, rows, a.lists, tiles, num_sms))
    return launch_q8_listed_many(a, workspace, num_sms, stream);
  if (solo_wins(a, a.lists, num_sms))
    return launch_solo<kListed>(a, (int)rows, a.lists, tiles, (char *)workspace, num_sms, (cudaStream_t)stream);
  return launch_few<kListed>(a, (int)std::min(rows, 1024ll), units, tiles, (char *)workspace, num_sms, (cudaStream_t)stream);
}

}  // namespace tq
