// capi_check.h -- what the parts of the C ABI around the experts check alike.
#pragma once

#include "experts.h"
#include "moe_experts.h"
#include "shape_check.h"

namespace moe {
namespace capi {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// present and aligned / absent or aligned
inline bool rows_ok(const void* p) { return p && aligned16(p); }
inline bool maybe_rows_ok(const void* p) { return aligned16(p); }

inline moe_status from_hip(hipError_t e) {
  if (e == hipErrorNotSupported) return MOE_ERR_UNSUPPORTED;  // the launchers' own limits
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// A shape's receive rows.
inline moe_status check_shape(const moe_shape* s, int* rows) {
  int L;
  int64_t n;
  const moe_status st = moe::check_shape(s, &L, &n);
  if (st != MOE_OK) return st;
  if (n > MOE_MAX_EXPERT_ROWS) return MOE_ERR_UNSUPPORTED;
  *rows = (int)n;
  return MOE_OK;
}

inline moe_status segments(const moe_shape* s, const moe_layout* lay, int rows, moe::Segments* seg) {
  if (lay) {
    if (!lay->expert_counts || !lay->expert_offsets) return MOE_ERR_INVALID_ARG;
    seg->counts = lay->expert_counts;
    seg->offsets = lay->expert_offsets;
  } else {
    if (s->num_experts != 1 || s->top_k != 1) return MOE_ERR_INVALID_ARG;
    if (s->num_tokens > rows) return MOE_ERR_INVALID_ARG;  // more tokens than rows
    rows = s->num_tokens;
    seg->counts = seg->offsets = nullptr;
  }
  seg->E = s->num_experts;
  seg->L = s->num_experts / s->num_ranks;
  seg->C = s->rank_capacity;
  seg->rows = rows;
  const int64_t pairs = (int64_t)s->num_tokens * s->top_k;
  seg->pairs = (int)(pairs < rows ? pairs : rows);
  if (seg->pairs == 0) seg->rows = 0;  // no segment, whatever the counts say
  return MOE_OK;
}

}  // namespace capi
}  // namespace moe
