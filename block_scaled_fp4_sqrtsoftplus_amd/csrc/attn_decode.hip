// Attention of new tokens over the paged key-value cache (include/moe_attn.h,
// moe_attn_decode).
//
// Mathematics: every wave walks its keys once with the running maximum m and
// sum l of a softmax in base 2 (s2 = scale log2(e) q.k):
//   m' = max(m, s2), p = 2^(s2 - m'), a = 2^(m - m'), l = a l + sum p,
//   o = a o + p v;
// pieces (m_i, l_i, o_i) join as m = max m_i, l = sum 2^(m_i - m) l_i,
// o = sum 2^(m_i - m) o_i / l, first the waves of a workgroup through LDS,
// then the splits of a sequence in a second kernel.
//
// Matrix form: the rows of one key-value head (q_len * group of them, 16 to a
// tile) are the columns of both products, S^T = K Q^T and O^T = V^T P^T on
// 16x16x32 bf16 MFMA, so that m, l and the rescaling are per lane (lane % 16
// is the row), and the P that comes out of the first product is, register
// for register, the operand of the second: with lane group g = lane / 16 the first leaves keys
// 4 g .. 4 g + 3 of two 16-key tiles in a lane, and the second contracts over
// any order of keys that both of its operands share.  K and V go from memory
// to registers without LDS: K's operand is 16 bytes of one key per lane; V's
// needs 8 keys of one column per lane, which a lane gets by loading the same 8
// columns of its 8 keys (a wave then covers whole rows) and transposing 8 x 8
// in registers.  P is rounded to bf16 as v is: kept as the sum of two bf16
// values (16 bits) the output is nearer to the exact one by less than its own
// rounding (1.7e-3 instead of 2.3e-3 in the 2-norm), for 1 to 13% of the time.
//
// Bound by the reads of K and V, each row once.  Measured: 64 sequences of up to
// 4096 keys, 8 heads of 128 in bf16 106 us (6.1 TB/s; the join kernel takes 4.5 of
// them); one sequence of 131071 keys in FP8 49 us (5.5 TB/s); 32 sequences of up to 4096
// keys, 64 query heads on one 512-element head that is keys and values 47 us
// (2.2 TB/s: 35 and a join of 7.6, with 31 MB of partial results between
// them); 300 keys of 8 heads 7.8 us, a chain of latencies.
#include "attn_decode_kernels.h"

namespace moe {

size_t attn_decode_ws_bytes(const moe_attn_config& c) { return decode_ws_bytes(c); }

hipError_t launch_attn_decode(const moe_attn_config& c, const moe_rows& q, const moe_kv_cache& kv,
                              const int32_t* table, int table_width, const int32_t* seq_lens,
                              const moe_rows& out, float* lse, void* ws, hipStream_t st) {
  return launch_decode<false>(c, q, kv, table, table_width, seq_lens, nullptr, 0, out, lse, ws, st);
}

}  // namespace moe
