// Attention over a shared prefix and then the sequence's own tokens, for sequences whose rows fill units of their own
// (tq_q8_shared_attention): prompts behind a prefix. One pass over both caches; a unit reads the prefix by itself, from L2 for the most part.

#include "tq_q8_many.cuh"

namespace tq {

bool q8_both_many_fits(const Q8AttnArgs &a, int num_sms) { return many_fits(a, num_sms); }

int launch_q8_both_many(const Q8AttnArgs &a, void *workspace, int num_sms, void *stream) {
  const bool apart = units_apart(a, num_sms);
  return launch_many<kBoth>(a, apart, units_of(a, apart), (char *)workspace, num_sms, (cudaStream_t)stream);
}

}  // namespace tq
