// Host side of the C ABI declared in include/moe_serving.h: argument
// validation (pure host code, run before any HIP call) and the launches.
#include "attn_checks.h"

using namespace moe;

namespace {

constexpr int32_t kMostTokens = 1 << 30;   // of a window, of first tokens, of a sequence

moe_status check_pool(const moe_page_pool* p) {
  if (!p) return MOE_ERR_NULL_ARG;
  if (p->pages < 0 || p->pages > (int64_t(1) << 28) || p->batch < 0 || p->batch > 65536 ||
      p->width < 1 || p->width > (1 << 26))
    return MOE_ERR_BAD_SHAPE;
  if (p->page_size < 16 || p->page_size > 4096 || (p->page_size & (p->page_size - 1)))
    return MOE_ERR_BAD_SHAPE;
  if ((int64_t)p->width * p->page_size > kMostTokens ||
      (int64_t)p->batch * (p->width + int64_t(1)) >= (int64_t(1) << 31))
    return MOE_ERR_BAD_SHAPE;
  return MOE_OK;
}

// ... and its arrays.
moe_status check_pool_call(const moe_page_pool* p) {
  const moe_status s = check_pool(p);
  if (s != MOE_OK) return s;
  if ((p->pages > 0 && !p->refs) || (p->batch > 0 && (!p->table || !p->lens)))
    return MOE_ERR_NULL_ARG;
  if (!aligned16(p->refs) || !aligned4(p->table) || !aligned4(p->lens)) return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_attn_decode_sinks(const moe_attn_config* cfg, int32_t sinks, const moe_rows* q,
                                 const moe_kv_cache* cache, const int32_t* block_table,
                                 int32_t table_width, const int32_t* seq_lens,
                                 const moe_rows* out, float* lse, void* ws, size_t ws_bytes,
                                 void* stream) {
  moe_status s = check_decode_call(cfg, false, q, cache, block_table, table_width, seq_lens, out, lse,
                                   ws, ws_bytes);
  if (s != MOE_OK) return s;
  if (sinks < 0 || sinks > kMostTokens) return MOE_ERR_BAD_SHAPE;
  if (cfg->batch == 0) return MOE_OK;
  if ((s = device_ok()) != MOE_OK) return s;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (sinks == 0 || cfg->window == 0)
    return hip_status(launch_attn_decode(*cfg, *q, *cache, block_table, table_width, seq_lens,
                                         *out, lse, ws, st));
  return hip_status(launch_attn_tree(*cfg, sinks, *q, *cache, block_table, table_width, seq_lens,
                                     nullptr, *out, lse, ws, st));
}

moe_status moe_attn_prefill_sinks(const moe_attn_config* cfg, int32_t sinks, const moe_rows* q,
                                  const moe_rows* k, const moe_rows* v, const int32_t* cu_q,
                                  const int32_t* cu_k, const moe_rows* out, float* lse,
                                  void* stream) {
  moe_status s = check_prefill_call(cfg, q, k, v, cu_q, cu_k, out, lse);
  if (s != MOE_OK) return s;
  if (sinks < 0 || sinks > kMostTokens) return MOE_ERR_BAD_SHAPE;
  if (cfg->batch == 0 || cfg->tokens == 0) return MOE_OK;
  if ((s = device_ok()) != MOE_OK) return s;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (!cu_k) cu_k = cu_q;
  if (sinks == 0 || cfg->window == 0)
    return hip_status(launch_attn_prefill(*cfg, *q, *k, *v, cu_q, cu_k, *out, lse, st));
  return hip_status(launch_attn_prefill_sinks(*cfg, sinks, *q, *k, *v, cu_q, cu_k, *out, lse, st));
}

moe_status moe_tree_masks(int32_t batch, int32_t nodes, const int32_t* parents, uint64_t* masks,
                          int32_t* depths, void* stream) {
  if (batch < 0 || batch > 65536 || nodes < 1 || nodes > 64) return MOE_ERR_BAD_SHAPE;
  if (batch > 0 && (!parents || !masks)) return MOE_ERR_NULL_ARG;
  if (!aligned4(parents) || !aligned4(depths) || (reinterpret_cast<uintptr_t>(masks) & 7u))
    return MOE_ERR_MISALIGNED;
  if (batch == 0) return MOE_OK;
  const moe_status s = device_ok();
  if (s != MOE_OK) return s;
  return hip_status(launch_tree_masks(batch, nodes, parents, masks, depths,
                                      static_cast<hipStream_t>(stream)));
}

size_t moe_attn_tree_workspace_size(const moe_attn_config* cfg) {
  return check_decode(cfg, 64) == MOE_OK ? attn_tree_ws_bytes(*cfg) : 0;
}

moe_status moe_attn_tree(const moe_attn_config* cfg, int32_t sinks, const moe_rows* q,
                         const moe_kv_cache* cache, const int32_t* block_table,
                         int32_t table_width, const int32_t* context_lens, const uint64_t* masks,
                         const moe_rows* out, float* lse, void* ws, size_t ws_bytes,
                         void* stream) {
  moe_status s = check_decode_call(cfg, true, q, cache, block_table, table_width, context_lens, out,
                                   lse, ws, ws_bytes);
  if (s != MOE_OK) return s;
  if (sinks < 0 || sinks > kMostTokens) return MOE_ERR_BAD_SHAPE;
  if (cfg->batch > 0 && !masks) return MOE_ERR_NULL_ARG;
  if (reinterpret_cast<uintptr_t>(masks) & 7u) return MOE_ERR_MISALIGNED;
  if (cfg->window > 0 && cfg->window < cfg->q_len) return MOE_ERR_UNSUPPORTED;
  if (cfg->batch == 0) return MOE_OK;
  if ((s = device_ok()) != MOE_OK) return s;
  return hip_status(launch_attn_tree(*cfg, sinks, *q, *cache, block_table, table_width,
                                     context_lens, masks, *out, lse, ws,
                                     static_cast<hipStream_t>(stream)));
}

moe_status moe_kv_compact(const moe_kv_cache* cache, int32_t batch, int32_t nodes,
                          const int32_t* block_table, int32_t table_width,
                          const int32_t* context_lens, const int32_t* path,
                          const int32_t* counts, void* stream) {
  moe_status s = check_cache(cache);
  if (s != MOE_OK) return s;
  if (batch < 0 || batch > 65536 || nodes < 1 || nodes > 64) return MOE_ERR_BAD_SHAPE;
  if (table_width < 0 || (int64_t)table_width * cache->page_size > kMostTokens)
    return MOE_ERR_BAD_SHAPE;
  if (batch > 0 && (!context_lens || !path || !counts || (table_width > 0 && !block_table)))
    return MOE_ERR_NULL_ARG;
  if (!aligned4(block_table) || !aligned4(context_lens) || !aligned4(path) || !aligned4(counts))
    return MOE_ERR_MISALIGNED;
  if (batch == 0) return MOE_OK;
  if ((s = device_ok()) != MOE_OK) return s;
  return hip_status(launch_kv_compact(*cache, batch, nodes, block_table, table_width, context_lens,
                                      path, counts, static_cast<hipStream_t>(stream)));
}

moe_status moe_kv_copy_pages(const moe_kv_cache* cache, int64_t n, const int32_t* src,
                             const int32_t* dst, void* stream) {
  moe_status s = check_cache(cache);
  if (s != MOE_OK) return s;
  if (n < 0 || n >= (int64_t(1) << 31)) return MOE_ERR_BAD_SHAPE;
  if (n > 0 && (!src || !dst)) return MOE_ERR_NULL_ARG;
  if (!aligned4(src) || !aligned4(dst)) return MOE_ERR_MISALIGNED;
  if (n == 0) return MOE_OK;
  if ((s = device_ok()) != MOE_OK) return s;
  return hip_status(launch_kv_copy_pages(*cache, n, src, dst, static_cast<hipStream_t>(stream)));
}

size_t moe_pool_workspace_size(const moe_page_pool* pool) {
  return check_pool(pool) == MOE_OK ? pool_ws_bytes(*pool) : 0;
}

moe_status moe_pool_grow(const moe_page_pool* pool, int64_t tokens, const int32_t* cu,
                         int64_t* slots, int32_t* positions, int32_t* src, int32_t* dst,
                         int32_t* missing, void* ws, size_t ws_bytes, void* stream) {
  moe_status s = check_pool_call(pool);
  if (s != MOE_OK) return s;
  if (tokens < 0 || tokens >= (int64_t(1) << 31)) return MOE_ERR_BAD_SHAPE;
  if (!cu || !missing || (tokens > 0 && (!slots || !positions)) ||
      (pool->batch > 0 && (!src || !dst)))
    return MOE_ERR_NULL_ARG;
  if (!aligned4(cu) || (reinterpret_cast<uintptr_t>(slots) & 7u) || !aligned4(positions) ||
      !aligned4(src) || !aligned4(dst) || !aligned4(missing))
    return MOE_ERR_MISALIGNED;
  if (ws_bytes < pool_ws_bytes(*pool)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!ws) return MOE_ERR_NULL_ARG;
  if (!aligned16(ws)) return MOE_ERR_MISALIGNED;
  if ((s = device_ok()) != MOE_OK) return s;
  return hip_status(launch_pool_grow(*pool, tokens, cu, slots, positions, src, dst, missing, ws,
                                     static_cast<hipStream_t>(stream)));
}

moe_status moe_pool_fork(const moe_page_pool* pool, const int32_t* parents, void* stream) {
  moe_status s = check_pool_call(pool);
  if (s != MOE_OK) return s;
  if (pool->batch > 0 && !parents) return MOE_ERR_NULL_ARG;
  if (!aligned4(parents)) return MOE_ERR_MISALIGNED;
  if (pool->batch == 0) return MOE_OK;
  if ((s = device_ok()) != MOE_OK) return s;
  return hip_status(launch_pool_fork(*pool, parents, static_cast<hipStream_t>(stream)));
}

moe_status moe_pool_trim(const moe_page_pool* pool, const int32_t* lens, int32_t window,
                         int32_t sinks, void* stream) {
  moe_status s = check_pool_call(pool);
  if (s != MOE_OK) return s;
  if (window < 0 || window > kMostTokens || sinks < 0 || sinks > kMostTokens)
    return MOE_ERR_BAD_SHAPE;
  if (!aligned4(lens)) return MOE_ERR_MISALIGNED;
  if (pool->batch == 0) return MOE_OK;
  if ((s = device_ok()) != MOE_OK) return s;
  return hip_status(launch_pool_trim(*pool, lens, window, sinks, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
