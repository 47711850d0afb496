// Host side of the C ABI declared in include/moe_attn.h: argument validation
// (pure host code, run before any HIP call) and the launches.
#include "attn_checks.h"

using namespace moe;

extern "C" {

moe_status moe_kv_append(const moe_kv_cache* cache, const moe_rope* rope, int64_t tokens,
                         const int64_t* slots, const int32_t* positions, const moe_rows* k,
                         const moe_rows* v, int32_t heads_q, const moe_rows* q,
                         const moe_rows* q_out, const moe_rows* k_out, void* stream) {
  moe_status s = check_cache(cache);
  if (s != MOE_OK) return s;
  if (tokens < 0 || tokens >= (int64_t(1) << 31)) return MOE_ERR_BAD_SHAPE;
  const bool used = tokens > 0;
  if (rope) {
    if (rope->rot_dim < 16 || rope->rot_dim % 16 || rope->rot_offset < 0 ||
        rope->rot_offset % 8 || (int64_t)rope->rot_offset + rope->rot_dim > cache->head_dim)
      return MOE_ERR_BAD_SHAPE;
    if (rope->positions < 1 || rope->positions > INT32_MAX) return MOE_ERR_BAD_SHAPE;
    if (!rope->cos_sin || (used && !positions)) return MOE_ERR_NULL_ARG;
    if (!aligned16(rope->cos_sin)) return MOE_ERR_MISALIGNED;
  }
  if (used && !slots) return MOE_ERR_NULL_ARG;
  if ((reinterpret_cast<uintptr_t>(slots) & 7u) || (reinterpret_cast<uintptr_t>(positions) & 3u))
    return MOE_ERR_MISALIGNED;
  if ((s = check_rows(k, used)) != MOE_OK) return s;
  // one tensor for keys and values takes no v, two take one
  const bool one = cache->k == cache->v && cache->pages > 0;
  if (cache->pages > 0 && (v == nullptr) != one) return MOE_ERR_NULL_ARG;
  if (v && (s = check_rows(v, used)) != MOE_OK) return s;
  if ((q == nullptr) != (q_out == nullptr)) return MOE_ERR_NULL_ARG;
  if (q) {
    if (heads_q < 1 || heads_q > 1024) return MOE_ERR_BAD_SHAPE;
    if ((s = check_rows(q, used)) != MOE_OK) return s;
    if ((s = check_rows(q_out, used)) != MOE_OK) return s;
  }
  if (k_out && (s = check_rows(k_out, used)) != MOE_OK) return s;
  if (!used) return MOE_OK;
  if ((s = device_ok()) != MOE_OK) return s;
  return hip_status(launch_kv_append(*cache, rope, tokens, slots, positions, *k, v, heads_q, q,
                                     q_out, k_out, static_cast<hipStream_t>(stream)));
}

size_t moe_attn_workspace_size(const moe_attn_config* cfg) {
  return check_decode(cfg, 16) == MOE_OK ? attn_decode_ws_bytes(*cfg) : 0;
}

moe_status moe_attn_decode(const moe_attn_config* cfg, const moe_rows* q,
                           const moe_kv_cache* cache, const int32_t* block_table,
                           int32_t table_width, const int32_t* seq_lens, const moe_rows* out,
                           float* lse, void* ws, size_t ws_bytes, void* stream) {
  return moe_attn_decode_sinks(cfg, 0, q, cache, block_table, table_width, seq_lens, out, lse, ws,
                               ws_bytes, stream);
}

moe_status moe_attn_prefill(const moe_attn_config* cfg, const moe_rows* q, const moe_rows* k,
                            const moe_rows* v, const int32_t* cu_q, const int32_t* cu_k,
                            const moe_rows* out, float* lse, void* stream) {
  return moe_attn_prefill_sinks(cfg, 0, q, k, v, cu_q, cu_k, out, lse, stream);
}

}  // extern "C"
