/*
 * moe_attn.h - C ABI of the attention operators that stand before the routed
 * MoE layer in a decoder block (same library, libmoe_fp4.so): a paged
 * key-value cache, the append that rotates and stores new tokens, attention
 * of new tokens over the cache, and attention over packed prompts.
 *
 * Formulas, for one query row q (head h, position p) and the keys k_j, values
 * v_j of its key-value head (h / (heads_q / heads_kv)):
 *   s_j = scale * sum_d q[d] k_j[d]     for the positions j the mask keeps
 *   out = sum_j exp(s_j - lse) v_j,     lse = ln sum_j exp(s_j)
 * A row that keeps no position gives out = 0 and lse = -inf.  The mask keeps
 *   j < length of the row's sequence,
 *   j <= p              (always in decode; in prefill if `causal`),
 *   j > p - window      (if window > 0).
 * Rotation of a pair (a, b) by the angle of position p and pair i:
 *   a' = a cos - b sin,  b' = b cos + a sin, in fp32, rounded to bf16 once.
 *
 * Conventions (those of moe_fp4.h unless said otherwise here):
 *  - Tensors of rows are [tokens, heads, head_dim] bf16 with the last index
 *    contiguous and the strides of the other two given in elements, multiples
 *    of 8; pointers are 16-byte aligned.  So q, k and v may lie side by side
 *    in the output of one fused projection.
 *  - All offsets into caches and rows are computed in 64 bits.
 *  - Values held in integers on the device cannot be checked by the host.  None of
 *    them makes a kernel read or write out of bounds: what each entry point
 *    does with a value outside its range is stated there.
 *  - Scores, softmax sums, outputs and rotations are accumulated in fp32;
 *    the softmax weights are rounded to bf16 for the product with v.
 *  - Keys and values that some row of the sequence keeps must be finite; a
 *    query with a NaN (such as one of a position outside the rotation table) gives
 *    NaN in its own row of out and lse and in no other.  Cache slots past a sequence's
 *    length, keys outside every row's window and rows of other sequences
 *    are not read into any result, whatever they hold.
 *  - No call allocates device memory, clears memory by a memset, or
 *    synchronises; all may be captured into a graph.
 */
#ifndef MOE_ATTN_H
#define MOE_ATTN_H

#include "moe_fp4.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_kv_format {
  MOE_KV_BF16 = 0,
  MOE_KV_FP8 = 1   /* E4M3 bytes and one E8M0 scale byte per 128 elements
                      (per row where head_dim is 64), as moe_quant_act */
} moe_kv_format;

/* bf16 rows [tokens, heads, head_dim], innermost contiguous. */
typedef struct moe_rows {
  uint16_t* p;
  int64_t stride_token;   /* elements, multiple of 8, >= 0 */
  int64_t stride_head;
} moe_rows;

/* A paged cache: page, head, row in the page, element.  Position j of a
 * sequence with block table row `table` is row j % page_size of page
 * table[j / page_size].  v == k is a cache of one tensor that serves as keys and
 * values (a latent cache).  An FP8 one may have two arrays of scales, whose
 * values are then the keys' codes under v_scale; the append gives both a new row's scales. */
typedef struct moe_kv_cache {
  void* k;
  void* v;
  uint8_t* k_scale;      /* MOE_KV_FP8: [pages, heads, page_size, max(1, head_dim / 128)]
                            contiguous; NULL for MOE_KV_BF16 */
  uint8_t* v_scale;
  int64_t pages;         /* >= 0 */
  int64_t stride_page;   /* elements (bf16: 2 bytes, FP8: 1 byte), of k and v alike; */
  int64_t stride_head;   /* multiples of 16 bytes, >= 0 */
  int64_t stride_token;  /* at most 2^23 */
  int32_t page_size;     /* power of two in [16, 4096] */
  int32_t heads;         /* [1, 1024] */
  int32_t head_dim;      /* 64, 128, 256 or 512 */
  int32_t format;        /* moe_kv_format */
} moe_kv_cache;

/* Rotation table.  Row p holds the rot_dim / 2 cosines and then the
 * rot_dim / 2 sines of position p; elements rot_offset .. rot_offset + rot_dim
 * of a head are rotated, the others pass through.  Any frequency scaling is
 * in the table. */
typedef struct moe_rope {
  const float* cos_sin;  /* [positions, rot_dim], 16-byte aligned */
  int64_t positions;     /* >= 1 */
  int32_t rot_dim;       /* multiple of 16 in [16, head_dim] */
  int32_t rot_offset;    /* multiple of 8, rot_offset + rot_dim <= head_dim */
  int32_t interleaved;   /* 0: pairs (i, i + rot_dim / 2); 1: pairs (2i, 2i + 1) */
  int32_t reserved;      /* set to 0 */
} moe_rope;

/* Append: for every token t, rotate q[t] into q_out and k[t] into the cache
 * (and k_out), and copy v[t] into the cache.
 *   slots      [tokens] int64: page * page_size + row of the token's place;
 *              a slot outside [0, pages * page_size), such as the -1 of a
 *              padding token, stores nothing in the cache (q_out and k_out are written)
 *   positions  [tokens] int32, needed with rope: a position outside the table
 *              gives NaN in the rotated elements
 *   rope       NULL: no rotation
 *   k, v       [tokens, heads, head_dim]; v NULL if and only if cache->v == cache->k
 *   q, q_out   [tokens, heads_q, head_dim], both or neither; q_out may be q
 *   k_out      NULL, or receives the rotated k (prompt attention reads it);
 *              may be k
 * Outputs may equal their input as said; any other overlap, and two tokens with one
 * slot, are not allowed.  FP8 caches quantize the bf16-rounded rows. */
moe_status moe_kv_append(const moe_kv_cache* cache, const moe_rope* rope, int64_t tokens,
                         const int64_t* slots, const int32_t* positions, const moe_rows* k,
                         const moe_rows* v, int32_t heads_q, const moe_rows* q,
                         const moe_rows* q_out, const moe_rows* k_out, void* stream);

/* Sizes shared by the two attentions. heads_q is a multiple of heads_kv. */
typedef struct moe_attn_config {
  int64_t tokens;      /* rows of q; decode: batch * q_len                   */
  int64_t tokens_kv;   /* prefill: rows of k and v; decode: unused           */
  int32_t batch;       /* sequences, [0, 65536]                               */
  int32_t q_len;       /* decode: new tokens per sequence, [1, 16]; else unused */
  int32_t heads_q;     /* [1, 1024]                                          */
  int32_t heads_kv;
  int32_t head_dim;    /* 64, 128, 256 or 512                                */
  int32_t causal;      /* prefill: 0 or 1; decode is always causal           */
  int32_t window;      /* 0: none                                            */
  float scale;         /* finite, not 0                                      */
} moe_attn_config;

/* Bytes of device workspace moe_attn_decode needs for `cfg`, whatever the
 * lengths (0 if cfg is invalid or NULL).  Pure host function.  The workspace
 * need not be cleared. */
size_t moe_attn_workspace_size(const moe_attn_config* cfg);

/* Attention of the newest q_len tokens of every sequence over the cache,
 * which holds them already: row i of sequence b stands at position
 * seq_lens[b] - q_len + i.
 *   q, out       [batch * q_len, heads_q, head_dim]
 *   block_table  [batch, table_width] int32 pages; entries that no row's mask
 *                reaches are not read; keys on a page outside [0, pages) are
 *                left out; table_width * page_size at most 2^30, and times
 *                batch below 2^36
 *   seq_lens     [batch] int32, new tokens included; less than 1 keeps
 *                nothing, more than table_width * page_size is that
 *   lse          [batch * q_len, heads_q] fp32 or NULL
 * The work is cut into pieces on the device, which workgroups share; whether,
 * and so the order of every sum, depends on cfg, the cache's sizes, table_width and the lengths
 * alone, so equal calls give equal bits. */
moe_status moe_attn_decode(const moe_attn_config* cfg, const moe_rows* q,
                           const moe_kv_cache* cache, const int32_t* block_table,
                           int32_t table_width, const int32_t* seq_lens, const moe_rows* out,
                           float* lse, void* ws, size_t ws_bytes, void* stream);

/* Attention over packed prompts: sequence b's queries are rows cu_q[b] ..
 * cu_q[b + 1] of q and out, its keys and values rows cu_k[b] .. cu_k[b + 1]
 * of k and v.  The last query stands at the last key's position, so a prompt
 * with a context before it has more keys than queries; with fewer keys the first rows keep nothing.
 *   cu_q, cu_k   [batch + 1] int32, not decreasing (entries are clamped to
 *                [0, tokens] and [0, tokens_kv]); cu_k NULL: cu_q
 *   k, v         [tokens_kv, heads_kv, head_dim], stride_token at most 2^23;
 *                v may be k
 *   lse          [tokens, heads_q] fp32 or NULL
 * Rows of q that belong to no sequence are left as they are in out and lse. */
moe_status moe_attn_prefill(const moe_attn_config* cfg, const moe_rows* q, const moe_rows* k,
                            const moe_rows* v, const int32_t* cu_q, const int32_t* cu_k,
                            const moe_rows* out, float* lse, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ATTN_H */
