// shape_check.h -- what both parts of the C ABI ask of a moe_shape.
#pragma once

#include "moe_dispatch.h"

namespace moe {

// Validates a shape; on success fills L and the receive row count.
inline moe_status check_shape(const moe_shape* s, int* L, int64_t* rows) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->num_tokens < 0 || s->hidden <= 0 || s->num_experts < 1 || s->top_k < 1 ||
      s->num_ranks < 1 || s->rank_capacity < 0)
    return MOE_ERR_INVALID_ARG;
  if (s->payload != MOE_PAYLOAD_BF16 && s->payload != MOE_PAYLOAD_FP8_E4M3_B128)
    return MOE_ERR_INVALID_ARG;
  if (s->top_k > s->num_experts) return MOE_ERR_INVALID_ARG;
  if (s->num_experts % s->num_ranks != 0) return MOE_ERR_INVALID_ARG;
  if (s->num_experts > MOE_MAX_EXPERTS || s->top_k > MOE_MAX_TOP_K) return MOE_ERR_UNSUPPORTED;
  if (s->payload == MOE_PAYLOAD_BF16 && s->hidden % 8 != 0) return MOE_ERR_INVALID_ARG;
  if (s->payload == MOE_PAYLOAD_FP8_E4M3_B128 && s->hidden % 128 != 0) return MOE_ERR_INVALID_ARG;
  const int64_t pairs = (int64_t)s->num_tokens * s->top_k;
  const int64_t r = s->rank_capacity > 0 ? (int64_t)s->num_ranks * s->rank_capacity : pairs;
  if (pairs > INT32_MAX || r > INT32_MAX) return MOE_ERR_UNSUPPORTED;  // rows are int32
  *L = s->num_experts / s->num_ranks;
  *rows = r;
  return MOE_OK;
}

}  // namespace moe
