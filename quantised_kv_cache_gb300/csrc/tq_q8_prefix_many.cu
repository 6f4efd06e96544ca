// The shared prefix's part of all sequences' rows, for many rows per KV head (tq_q8_shared_attention).

#include "tq_q8_many.cuh"

namespace tq {

bool q8_prefix_many_fits(const Q8AttnArgs &a, int num_sms) { return many_fits(a, num_sms); }

int launch_q8_prefix_many(const Q8AttnArgs &a, void *workspace, int num_sms, void *stream) {
  const bool apart = units_apart(a, num_sms);
  return launch_many<kPrefix>(a, apart, units_of(a, apart), (char *)workspace, num_sms, (cudaStream_t)stream);
}

}  // namespace tq
