// Argument checks shared by the host sides of include/moe_attn.h and
// include/moe_serving.h: pure host code, run before any HIP call.
#pragma once

#include <cmath>

#include "attn_internal.h"

namespace moe {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256 || d == 512; }

// Strides stay below 2^40 elements, so that no product with an index of the
// supported ranges passes 63 bits.
inline bool stride_ok(int64_t s, int64_t multiple) {
  return s >= 0 && s < (int64_t(1) << 40) && s % multiple == 0;
}

// Rows a call reads or writes; `used` is false when there are no tokens.
inline moe_status check_rows(const moe_rows* r, bool used) {
  if (!r) return MOE_ERR_NULL_ARG;
  if (used && !r->p) return MOE_ERR_NULL_ARG;
  if (!stride_ok(r->stride_token, 1) || !stride_ok(r->stride_head, 1)) return MOE_ERR_BAD_SHAPE;
  if (!aligned16(r->p) || r->stride_token % 8 || r->stride_head % 8) return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

inline moe_status check_cache(const moe_kv_cache* c) {
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

inline moe_status check_attn(const moe_attn_config* c) {
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

// Decode's sizes: up to `most` new tokens per sequence.
inline moe_status check_decode(const moe_attn_config* c, int most) {
  moe_status s = check_attn(c);
  if (s != MOE_OK) return s;
  if (c->q_len < 1 || c->q_len > most) return MOE_ERR_BAD_SHAPE;
  if (c->tokens != (int64_t)c->batch * c->q_len) return MOE_ERR_BAD_SHAPE;
  return MOE_OK;
}

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A decode call's arguments; lens: the sequences' lengths.
inline moe_status check_decode_call(const moe_attn_config* cfg, bool tree, const moe_rows* q,
                                    const moe_kv_cache* cache, const int32_t* block_table,
                                    int32_t table_width, const int32_t* lens, const moe_rows* out,
                                    const float* lse, const void* ws, size_t ws_bytes) {
  moe_status s = check_decode(cfg, tree ? 64 : 16);
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
  if (used && (!lens || (table_width > 0 && !block_table))) return MOE_ERR_NULL_ARG;
  if (!aligned4(lens) || !aligned4(block_table) || !aligned4(lse)) return MOE_ERR_MISALIGNED;
  if (ws_bytes < (tree ? attn_tree_ws_bytes(*cfg) : attn_decode_ws_bytes(*cfg)))
    return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!ws) return MOE_ERR_NULL_ARG;
  if (!aligned16(ws)) return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

// A prompt call's arguments.
inline moe_status check_prefill_call(const moe_attn_config* cfg, const moe_rows* q,
                                     const moe_rows* k, const moe_rows* v, const int32_t* cu_q,
                                     const int32_t* cu_k, const moe_rows* out, const float* lse) {
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
  if (!aligned4(cu_q) || !aligned4(cu_k) || !aligned4(lse)) return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

inline moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

}  // namespace moe
