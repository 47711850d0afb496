// Attention over packed prompts with a sliding window behind which the first
// tokens stay visible (include/moe_serving.h, moe_attn_prefill_sinks).
//
// Mathematics and matrix form are those of attn_prefill.hip; a row keeps the
// keys j <= p with j > p - window or j < sinks.  A workgroup walks the tiles of
// the first keys and then those of its rows' windows: what lies between is
// neither read nor computed, so its work does not grow with the position.
//
// Bound by the matrix units, as attn_prefill.hip, and by workgroups that start and end: a
// row's keys are few.  8192 tokens, 32 heads of 128 on 8, window of 1024, 16 first tokens 165 us (793 TFLOP/s
// of what the mask leaves; a window's first and last tiles and the one of the first tokens are computed whole);
// five packed prompts 52.7 us.
#include "attn_prefill_kernel.h"

namespace moe {

hipError_t launch_attn_prefill_sinks(const moe_attn_config& c, int sinks, const moe_rows& q,
                                     const moe_rows& k, const moe_rows& v, const int32_t* cu_q,
                                     const int32_t* cu_k, const moe_rows& out, float* lse,
                                     hipStream_t st) {
  return launch_prefill<true>(c, sinks, q, k, v, cu_q, cu_k, out, lse, st);
}

}  // namespace moe
