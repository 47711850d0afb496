// Host side of the C ABI declared in include/moe_attn.h: argument validation
// (pure host code, run before any HIP call) and the launches.
#include <cmath>

#include "attn_internal.h"

namespace {

using namespace moe;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256 || d == 512; }

// Strides stay below 2^40 elements, so that no product with an index of the
// supported ranges passes 63 bits.
bool stride_ok(int64_t s, int64_t multiple) {
  return s >= 0 && s < (int64_t(1) << 40) && s % multiple == 0;
}

// Rows a call reads or writes; `used` is false when there are no tokens.
moe_status check_rows(const moe_rows* r, bool used) {
  if (!r) return MOE_ERR_NULL_ARG;
  if (used && !r->p) return MOE_ERR_NULL_ARG;
  if (!stride_ok(r->stride_token, 1) || !stride_ok(r->stride_head, 1)) return MOE_ERR_BAD_SHAPE;
  if (!aligned16(r->p) || r->stride_token % 8 || r->stride_head % 8) return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

moe_status check_cache(const moe_kv_cache* c) {
  if (!c) return MOE_ERR_NULL_ARG;
  if (!head_dim_ok(c->head_dim) || c->heads < 1 || c->heads > 1024) return MOE_ERR_BAD_SHAPE;
  if (c->page_size < 16 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)))
    return MOE_ERR_BAD_SHAPE;
  if (c->format != MOE_KV_BF16 && c->format != MOE_KV_FP8) return MOE_ERR_BAD_SHAPE;
  if (c->pages < 0 || c->pages > INT32_MAX) return MOE_ERR_BAD_SHAPE;
  if (!stride_ok(c->stride_page, 1) || !stride_ok(c->stride_head, 1) ||
      !stride_ok(c->stride_token, 1))
    return MOE_ERR_BAD_SHAPE;
  const int64_t unit = c->format == MOE_KV_FP8 ? 16 : 8;
  if (c->stride_token > (1 << 23)) return MOE_ERR_BAD_SHAPE;   // rows of a tile: 32-bit offsets
  if (c->stride_page % unit || c->stride_head % unit || c->stride_token % unit)
    return MOE_ERR_MISALIGNED;
  if (c->pages > 0) {
    if (!c->k || !c->v) return MOE_ERR_NULL_ARG;
    if (c->format == MOE_KV_FP8 && (!c->k_scale || !c->v_scale)) return MOE_ERR_NULL_ARG;
  }
  if (!aligned16(c->k) || !aligned16(c->v)) return MOE_ERR_MISALIGNED;
  if (c->format == MOE_KV_FP8 && (!aligned16(c->k_scale) || !aligned16(c->v_scale)))
    return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

moe_status check_attn(const moe_attn_config* c) {
  if (!c) return MOE_ERR_NULL_ARG;
  if (!head_dim_ok(c->head_dim)) return MOE_ERR_BAD_SHAPE;
  if (c->heads_kv < 1 || c->heads_q < c->heads_kv || c->heads_q > 1024 ||
      c->heads_q % c->heads_kv)
    return MOE_ERR_BAD_SHAPE;
  if (c->batch < 0 || c->batch > 65536) return MOE_ERR_BAD_SHAPE;
  if (c->tokens < 0 || c->tokens * c->heads_q >= (int64_t(1) << 31)) return MOE_ERR_BAD_SHAPE;
  if (c->window < 0 || c->window > (1 << 30)) return MOE_ERR_BAD_SHAPE;
  if (!std::isfinite(c->scale) || c->scale == 0.f) return MOE_ERR_BAD_SHAPE;
  return MOE_OK;
}

moe_status check_decode(const moe_attn_config* c) {
  moe_status s = check_attn(c);
  if (s != MOE_OK) return s;
  if (c->q_len < 1 || c->q_len > 16) return MOE_ERR_BAD_SHAPE;
  if (c->tokens != (int64_t)c->batch * c->q_len) return MOE_ERR_BAD_SHAPE;
  return MOE_OK;
}

moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

}  // namespace

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
  return check_decode(cfg) == MOE_OK ? attn_decode_ws_bytes(*cfg) : 0;
}

moe_status moe_attn_decode(const moe_attn_config* cfg, const moe_rows* q,
                           const moe_kv_cache* cache, const int32_t* block_table,
                           int32_t table_width, const int32_t* seq_lens, const moe_rows* out,
                           float* lse, void* ws, size_t ws_bytes, void* stream) {
  moe_status s = check_decode(cfg);
  if (s != MOE_OK) return s;
  if ((s = check_cache(cache)) != MOE_OK) return s;
  if (cache->heads != cfg->heads_kv || cache->head_dim != cfg->head_dim) return MOE_ERR_BAD_SHAPE;
  const int64_t longest = (int64_t)table_width * cache->page_size;
  if (table_width < 0 || longest > (int64_t(1) << 30) ||
      cfg->batch * (longest / 64 + 1) >= (int64_t(1) << 31))   // tiles are counted in 32 bits
    return MOE_ERR_BAD_SHAPE;
  const bool used = cfg->batch > 0;
  if ((s = check_rows(q, used)) != MOE_OK) return s;
  if ((s = check_rows(out, used)) != MOE_OK) return s;
  if (used && (!seq_lens || (table_width > 0 && !block_table))) return MOE_ERR_NULL_ARG;
  if ((reinterpret_cast<uintptr_t>(seq_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return MOE_ERR_MISALIGNED;
  if (ws_bytes < attn_decode_ws_bytes(*cfg)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!ws) return MOE_ERR_NULL_ARG;
  if (!aligned16(ws)) return MOE_ERR_MISALIGNED;
  if (!used) return MOE_OK;
  if ((s = device_ok()) != MOE_OK) return s;
  return hip_status(launch_attn_decode(*cfg, *q, *cache, block_table, table_width, seq_lens, *out,
                                       lse, ws, static_cast<hipStream_t>(stream)));
}

moe_status moe_attn_prefill(const moe_attn_config* cfg, const moe_rows* q, const moe_rows* k,
                            const moe_rows* v, const int32_t* cu_q, const int32_t* cu_k,
                            const moe_rows* out, float* lse, void* stream) {
  moe_status s = check_attn(cfg);
  if (s != MOE_OK) return s;
  if (cfg->causal != 0 && cfg->causal != 1) return MOE_ERR_BAD_SHAPE;
  if (cfg->tokens_kv < 0 || cfg->tokens_kv >= (int64_t(1) << 30)) return MOE_ERR_BAD_SHAPE;
  const bool used = cfg->batch > 0 && cfg->tokens > 0;
  if ((s = check_rows(q, used)) != MOE_OK) return s;
  if ((s = check_rows(k, used && cfg->tokens_kv > 0)) != MOE_OK) return s;
  if ((s = check_rows(v, used && cfg->tokens_kv > 0)) != MOE_OK) return s;
  if ((s = check_rows(out, used)) != MOE_OK) return s;
  // a tile's rows are addressed in 32 bits from its first
  if (k->stride_token > (1 << 23) || v->stride_token > (1 << 23)) return MOE_ERR_BAD_SHAPE;
  if (used && !cu_q) return MOE_ERR_NULL_ARG;
  if ((reinterpret_cast<uintptr_t>(cu_q) & 3u) || (reinterpret_cast<uintptr_t>(cu_k) & 3u) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return MOE_ERR_MISALIGNED;
  if (!used) return MOE_OK;
  if ((s = device_ok()) != MOE_OK) return s;
  return hip_status(launch_attn_prefill(*cfg, *q, *k, *v, cu_q, cu_k ? cu_k : cu_q, *out, lse,
                                        static_cast<hipStream_t>(stream)));
}

}  // extern "C"
