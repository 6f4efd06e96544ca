// Attention over the 8-bit cache for many query rows per KV head (tq_q8_attention): units of rows, workspace, launch.

#include "tq_q8_many.cuh"

namespace tq {
namespace {

// Up to 128 rows are one row tile, and the other of a shared unit would have no rows: with units apart every row tile works, but twice as
// many slices are joined and each has half of the ring. So where a CTA has a dozen tiles. 64 rows, 8 KV heads, bf16 (fp16): 8 sequences of
// 16384 tokens (54 tiles a CTA) 121 us apart, 165 us (170, 198) not, capped 178 and 284; 2 of them (13) 59 and 63 (73, 73); one (7) 49 and 45.
bool units_apart(const Q8AttnArgs &a, int num_sms) {
  const long long tiles = (long long)a.batch * a.heads_kv * ((a.max_len + kTile - 1) / kTile);
  return (long long)a.group * a.n_q <= unit_rows(true) && tiles >= 12LL * num_sms;
}

long long units_of(const Q8AttnArgs &a, bool apart) {
  const long long unit = unit_rows(apart);
  return ((long long)a.group * a.n_q + unit - 1) / unit;
}

}  // namespace

size_t q8_prompt_workspace(int num_sms, int batch, int group, int n_q) {
  return many_bytes(num_sms, ((size_t)group * n_q + unit_rows(false) - 1) / unit_rows(false) * batch);
}

// Entries' tiles are counted in 32 bits.
bool q8_prompt_fits(const Q8AttnArgs &a, int num_sms) {
  const long long entries = units_of(a, units_apart(a, num_sms)) * a.batch, tiles = (a.max_len + kTile - 1) / kTile;
  return entries <= 1 << 24 && entries * tiles <= 0x7fffffff;
}

int launch_q8_prompt(const Q8AttnArgs &a, void *workspace, int num_sms, void *stream) {
  const bool apart = units_apart(a, num_sms);
  return launch_many<kWhole>(a, apart, units_of(a, apart), (char *)workspace, num_sms, (cudaStream_t)stream);
}

}  // namespace tq
