// Attention over packed prompts (include/moe_attn.h, moe_attn_prefill).
//
// Mathematics: one pass over the keys with the running maximum m and sum l of
// a softmax in base 2: m' = max(m, s2), p = 2^(s2 - m'), o = o 2^(m - m') + p v,
// s2 = scale log2(e) q.k, out = o / l.
//
// Matrix form: S^T = K Q^T and O^T = V^T P^T on 32x32x16 bf16 MFMA.  A wave
// owns 32 rows; lane % 32 is the row in both products, so m, l and the
// rescaling are per lane (and its partner lane + 32), and the P that the first
// product leaves is the second's operand register for register: lane half hh =
// lane / 32 holds keys 16 c + 4 hh + (0..3) and 16 c + 8 + 4 hh + (0..3) of a
// 32-key tile in 8 consecutive registers, and the second product contracts 16 keys in
// whatever order both operands share.  Its V^T operand, 4 keys of one column
// per register pair, comes out of row-major V in LDS by the transposing LDS
// read.
//
// Rows: the heads of one key-value head's group are packed into the row
// index (row = token * group + head in the group), so a workgroup's rows span
// few tokens: short prompts fill their tiles and little is computed above the
// diagonal.
//
// P is rounded to bf16 as v is, its sum taken before: outputs are 2.0e-3 from the
// exact ones in the 2-norm, of which their own rounding is 1.6e-3.  P as the sum of
// two bf16 values would be a second product with V, half as many matrix
// instructions again where they are the bound.
//
// Measured (TFLOP/s count what the mask leaves): 8192 tokens, 32 heads of 128 on 8
// 502 to 519 us (1094 to 1060 TFLOP/s): matrix units busy for 58% of the cycles at a clock that the load
// brings down to 1.6 to 1.8 GHz, no LDS bank conflict; where the exponentials
// and loads stand between the products makes no difference there any more.  Six packed prompts 77 us
// (708), 2048 tokens of 64 heads on one 512-element head that is keys and
// values 304 us (903), 200 tokens of 16 heads of 64 7.6 us, all latencies.
#include "attn_prefill_kernel.h"

namespace moe {

hipError_t launch_attn_prefill(const moe_attn_config& c, const moe_rows& q, const moe_rows& k,
                               const moe_rows& v, const int32_t* cu_q, const int32_t* cu_k,
                               const moe_rows& out, float* lse, hipStream_t st) {
  return launch_prefill<false>(c, 0, q, k, v, cu_q, cu_k, out, lse, st);
}

}  // namespace moe
