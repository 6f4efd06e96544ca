// Attention over listed blocks of the 8-bit cache for lists of many rows (tq_q8_sparse_attention). 2048 tokens x 32 query heads, 8 KV heads,
// bf16, 32 blocks for every 64 tokens: 117 us (587 TFLOP/s of the formula's products): 16 tiles a unit of 256 rows and 1.7 units a CTA, so
// that the starts are a tenth and the second unit of most CTAs is waited for.

#include <algorithm>

#include "tq_q8_many.cuh"

namespace tq {
namespace {

// A list's units do not reach into the next list's rows. Those of up to 128 rows are one row tile: units apart.
bool list_apart(long long rows) { return rows <= unit_rows(true); }
long long list_units(long long rows, int lists) {
  const long long unit = unit_rows(list_apart(rows));
  return (rows + unit - 1) / unit * lists;
}

}  // namespace

size_t q8_listed_many_workspace(int num_sms, int batch, int group, int n_q, int span) {
  return many_bytes(num_sms, (size_t)list_units((long long)group * span, (n_q + span - 1) / span) * batch);
}

bool q8_listed_many_fits(const Q8AttnArgs &a) {
  const long long entries = list_units((long long)a.group * a.span, a.lists) * a.batch, tiles = (std::min(a.n_blocks, a.c.nblk) + 1) / 2;
  return entries <= 1 << 24 && entries * tiles <= 0x7fffffff;
}

int launch_q8_listed_many(const Q8AttnArgs &a, void *workspace, int num_sms, void *stream) {
  const long long rows = (long long)a.group * a.span;
  return launch_many<kListed>(a, list_apart(rows), list_units(rows, a.lists), (char *)workspace, num_sms, (cudaStream_t)stream);
}

}  // namespace tq
