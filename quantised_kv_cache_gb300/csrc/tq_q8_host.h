// Host helpers of the 8-bit cache that the general entry points use.
#pragma once

#include "tq_q8.h"

namespace tq {

tq_status q8_check_cache(const tq_ctx *ctx, const tq_cache *c, int batch, int heads_kv);
Q8Cache q8_cache(const tq_cache *c);
void q8_cache_sizes(int batch, int heads_kv, int capacity, tq_cache_sizes *out);

}  // namespace tq
