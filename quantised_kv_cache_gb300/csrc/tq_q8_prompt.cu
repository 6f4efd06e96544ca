// Attention over the 8-bit cache for many query rows per KV head (tq_q8_attention).

#include "tq_q8_many.cuh"

namespace tq {

size_t q8_prompt_workspace(int num_sms, int batch, int group, int n_q) {
  return many_bytes(num_sms, ((size_t)group * n_q + unit_rows(false) - 1) / unit_rows(false) * batch);
}

bool q8_prompt_fits(const Q8AttnArgs &a, int num_sms) { return many_fits(a, num_sms); }

int launch_q8_prompt(const Q8AttnArgs &a, void *workspace, int num_sms, void *stream) {
  const bool apart = units_apart(a, num_sms);
  return launch_many<kWhole>(a, apart, units_of(a, apart), (char *)workspace, num_sms, (cudaStream_t)stream);
}

}  // namespace tq
