/*
 * moe_serving.h - C ABI of what a serving loop needs around the paged cache
 * and its attentions (moe_attn.h; same library, libmoe_fp4.so): attention for
 * a tree of drafted tokens, windowed attention whose first tokens stay
 * visible, the rows of an accepted path moved to their places, copies of
 * pages, and a pool from which sequences fork, grow and free pages.
 *
 * Conventions are those of moe_attn.h: scores, softmax sums and outputs are
 * accumulated in fp32, the softmax weights rounded to bf16; offsets are 64
 * bits; values on the device cannot be checked by the host, none of them
 * makes a kernel read or write out of bounds, and each entry point says what
 * it does with one outside its range; no call allocates device memory, clears
 * memory by a memset or synchronises, so all may be captured into a graph.
 */
#ifndef MOE_SERVING_H
#define MOE_SERVING_H

#include "moe_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* moe_attn_decode and moe_attn_prefill for a window behind which the first
 * `sinks` tokens of every sequence stay visible: a row at position p keeps
 *   j <= p (prefill: if `causal`)   and   (j > p - window  or  j < sinks).
 * Arguments, workspace and results are theirs; sinks in [0, 2^30], and with
 * sinks or cfg->window 0 the calls are the same.  Of a sequence's block table
 * only the entries of those keys are read, so the pages between may be freed. */
moe_status moe_attn_decode_sinks(const moe_attn_config* cfg, int32_t sinks, const moe_rows* q,
                                 const moe_kv_cache* cache, const int32_t* block_table,
                                 int32_t table_width, const int32_t* seq_lens,
                                 const moe_rows* out, float* lse, void* ws, size_t ws_bytes,
                                 void* stream);
moe_status moe_attn_prefill_sinks(const moe_attn_config* cfg, int32_t sinks, const moe_rows* q,
                                  const moe_rows* k, const moe_rows* v, const int32_t* cu_q,
                                  const int32_t* cu_k, const moe_rows* out, float* lse,
                                  void* stream);

/* Masks and depths of drafted trees.
 *   parents  [batch, nodes] int32: -1 hangs a node on the sequence's last
 *            token, 0 .. i - 1 on that node; any other value makes node i
 *            an empty place, and so does a parent that is one
 *   masks    [batch, nodes] uint64: bit i and the bits of all nodes above
 *            node i; 0 for an empty place
 *   depths   [batch, nodes] int32 or NULL: how many nodes stand above it, -1
 *            for an empty place; context length + depth is its position
 * batch in [0, 65536], nodes in [1, 64]. */
moe_status moe_tree_masks(int32_t batch, int32_t nodes, const int32_t* parents, uint64_t* masks,
                          int32_t* depths, void* stream);

/* Attention of drafted tokens over the cache, which holds them already: node
 * i of sequence b is row context_lens[b] + i of its cache, whatever its
 * position.  cfg->q_len is the number of nodes, in [1, 64].  Row (b, i) keeps
 *   j < context_lens[b]   and, with a window, (j > p - window  or  j < sinks),
 *   j = context_lens[b] + n   for every bit n of masks[b, i],
 * with p = context_lens[b] + (bits of the mask) - 1, the position of a node
 * that sees itself and the nodes above it.  A mask of 0 keeps nothing: out =
 * 0, lse = -inf, whatever its q.  Masks need not be those of a tree; bits at or past
 * `nodes` are ignored.  A window is at least the number of nodes
 * (MOE_ERR_UNSUPPORTED below it); sinks in [0, 2^30], ignored without a window.
 *   q, out        [batch * nodes, heads_q, head_dim]
 *   block_table   [batch, table_width] int32, as in moe_attn_decode
 *   context_lens  [batch] int32, drafted tokens not included; below 0 is 0,
 *                 above table_width * page_size is that, and drafted tokens
 *                 past the table's end are kept by no row
 *   masks         [batch, nodes] uint64, 8-byte aligned
 *   lse           [batch * nodes, heads_q] fp32 or NULL
 * Drafted rows that no mask names may hold anything.  Equal calls give equal bits. */
size_t moe_attn_tree_workspace_size(const moe_attn_config* cfg);
moe_status moe_attn_tree(const moe_attn_config* cfg, int32_t sinks, const moe_rows* q,
                         const moe_kv_cache* cache, const int32_t* block_table,
                         int32_t table_width, const int32_t* context_lens, const uint64_t* masks,
                         const moe_rows* out, float* lse, void* ws, size_t ws_bytes, void* stream);

/* Moves the rows of accepted drafted tokens to the places behind the context:
 * for every i < counts[b] row context_lens[b] + path[b, i] of sequence b goes
 * to row context_lens[b] + i, in k, v and their scales.  All rows are read
 * before any is written, so a path may be any list of nodes, in any order.
 *   context_lens  [batch] int32, below 0 is 0
 *   path          [batch, nodes] int32; entries past counts[b] are not read,
 *                 and one outside [0, nodes) moves nothing
 *   counts        [batch] int32, clamped to [0, nodes]
 * A row whose place or source is past the table's end or on a page outside
 * [0, pages) is not moved.  Sequences that share the pages of drafted tokens are not
 * allowed.  batch in [0, 65536], nodes in [1, 64]. */
moe_status moe_kv_compact(const moe_kv_cache* cache, int32_t batch, int32_t nodes,
                          const int32_t* block_table, int32_t table_width,
                          const int32_t* context_lens, const int32_t* path,
                          const int32_t* counts, void* stream);

/* Copies page src[i] to page dst[i], k, v and their scales, for i < n; a pair
 * of which one is outside [0, pages), such as (-1, -1), copies nothing.  A page may be the source of
 * many; one that is the destination of two, or of one and a source, is not allowed.
 *   src, dst  [n] int32 */
moe_status moe_kv_copy_pages(const moe_kv_cache* cache, int64_t n, const int32_t* src,
                             const int32_t* dst, void* stream);

/* A pool of pages that the sequences of a block table hold: state on the
 * device that the calls below read and update in place, on one stream at a
 * time.  All layers' caches of one model go by one pool.  At the start refs
 * and lens are 0 and table is -1. */
typedef struct moe_page_pool {
  int32_t* refs;       /* [pages] how many table entries hold the page; 0: free */
  int32_t* table;      /* [batch, width] pages; -1: none                        */
  int32_t* lens;       /* [batch] tokens of each sequence                       */
  int64_t pages;       /* [0, 2^28]                                             */
  int32_t batch;       /* [0, 65536]                                            */
  int32_t width;       /* [1, 2^26]; batch * (width + 1) below 2^31             */
  int32_t page_size;   /* power of two in [16, 4096]; width * page_size at most 2^30 */
  int32_t reserved;    /* set to 0                                              */
} moe_page_pool;

/* Bytes of workspace moe_pool_grow needs (0 if the pool is invalid or NULL).
 * It need not be cleared. */
size_t moe_pool_workspace_size(const moe_page_pool* pool);

/* Adds cu[b + 1] - cu[b] tokens to every sequence b (a sequence ends at width *
 * page_size).  Table entries that new tokens are the first of get the
 * lowest-numbered free pages, sequence by sequence.  A sequence that grows on
 * a partly filled page held by others too gets a fresh page in its place,
 * before its others, and the pair (src, dst) to copy, in every layer's cache, before the new rows are
 * stored; where all holders of such a page grow, the one with the most tokens on it keeps it (of
 * equals the first), so that its new rows are behind every other holder's tokens.
 *   cu         [batch + 1] int32, not decreasing (entries are clamped to [0, tokens])
 *   slots      [tokens] int64 receives the new tokens' slots (moe_kv_append):
 *              -1 for one past the sequence's end, on a page that was not to be had,
 *              or of no sequence
 *   positions  [tokens] int32 receives their positions (0 of no sequence)
 *   src, dst   [batch] int32 receive each sequence's copy, or -1 and -1
 *   missing    [1] int32 receives how many pages were wanted and not free: the last ones
 *              wanted, whose entries stay -1
 * Where pages are missing, a sequence whose copy is among them does not grow: its length and its
 * entries stay, and all its tokens get slot -1.  The others are as long as with their pages; their
 * tokens without one get slot -1, and no attention keeps them.  A drafted node
 * without a slot has to be an empty place (mask 0) and must not be accepted; moe_pool_trim to
 * the lengths from before, after the copies, takes a call back. */
moe_status moe_pool_grow(const moe_page_pool* pool, int64_t tokens, const int32_t* cu,
                         int64_t* slots, int32_t* positions, int32_t* src, int32_t* dst,
                         int32_t* missing, void* ws, size_t ws_bytes, void* stream);

/* Makes every sequence b a fork of sequence parents[b] as it was before the
 * call: the same pages, held once more each, and the same length.  parents[b]
 * = b leaves it; a value outside [0, batch) leaves it empty, its pages
 * released.  What this drops is free afterwards.
 *   parents  [batch] int32 */
moe_status moe_pool_fork(const moe_page_pool* pool, const int32_t* parents, void* stream);

/* Cuts sequences and frees what they no longer need: with `lens` sequence b
 * is at most lens[b] tokens long (below 0 is 0), and table entries past its end are
 * released.  With a window so are the pages of which no token from now on
 * sees a row: those before position lens - window + 1 that hold none of the first `sinks` tokens.
 *   lens  [batch] int32 or NULL
 *   window, sinks  [0, 2^30]; window 0: none */
moe_status moe_pool_trim(const moe_page_pool* pool, const int32_t* lens, int32_t window,
                         int32_t sinks, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_SERVING_H */
