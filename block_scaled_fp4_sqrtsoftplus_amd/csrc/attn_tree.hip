// Attention of new tokens over the paged cache whose rows do not see all that
// is before them (include/moe_serving.h): a tree of drafted tokens
// (moe_attn_tree), and a window behind which the first tokens stay visible
// (moe_attn_decode_sinks).
//
// Mathematics and matrix form are those of attn_decode.hip.  Both are one
// mask: a row keeps a part of the context, [row_lo, context) and the first
// tokens, and of the up to 64 new tokens those of a bit mask (64 bits, one
// word a row; for rows that are causal among themselves the kernel makes it).
// A walk over the keys leaves those between the first tokens and the window out: they
// are neither read nor counted, so that a call's work does not grow with the context.
//
// Measured: a tree of 8 nodes behind 300 keys, 32 heads of 128 on 8, with its masks
// 12.2 us, of which the host's two launches are 8; one token of one sequence of 9000 keys,
// window of 512 and 4 first tokens 11.0 us, a chain of latencies (length, pages, keys) and a join; 64
// sequences of up to 500000 keys, window of 4096 and 64 first tokens, FP8 91 us (551 MB, 6.1 TB/s).
#include "attn_decode_kernels.h"

namespace moe {

size_t attn_tree_ws_bytes(const moe_attn_config& c) {
  return tree_rows_apply(c) ? tree_rows_ws_bytes(c) : decode_ws_bytes(c);
}

hipError_t launch_attn_tree(const moe_attn_config& c, int sinks, const moe_rows& q,
                            const moe_kv_cache& kv, const int32_t* table, int table_width,
                            const int32_t* lens, const uint64_t* masks, const moe_rows& out,
                            float* lse, void* ws, hipStream_t st) {
  if (c.batch == 0) return hipSuccess;
  const int64_t tables = (int64_t)table_width * kv.page_size;
  const int64_t longest = c.window > 0 ? std::min(tables, (int64_t)c.window + sinks + c.q_len + 64) : tables;
  const bool f8 = kv.format == MOE_KV_FP8, one = kv.k == kv.v && (!f8 || kv.k_scale == kv.v_scale);
  const bool narrow = narrow_groups(c, longest * c.head_dim * (f8 ? 1 : 2) * (one ? 1 : 2)) > 0;
  if (masks && tree_rows_apply(c) && !narrow)
    return launch_tree_rows(c, sinks, q, kv, table, table_width, lens, masks, out, lse, ws, st);
  return launch_decode<true>(c, q, kv, table, table_width, lens, masks, sinks, out, lse, ws, st);
}

namespace {

// One wave per sequence, a node per lane: in each of six turns a node takes the
// mask of the node it points to and then points where that one does, so that after
// them it holds up to 64 nodes and points past the chain's end.
__global__ __launch_bounds__(256) void tree_masks_kernel(const int32_t* parents, uint64_t* masks,
                                                         int32_t* depths, int batch, int nodes) {
  constexpr int kRoot = -1, kNone = -2;
  const int lane = threadIdx.x & 63;
  const int b = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (b >= batch) return;
  const int64_t at = (int64_t)b * nodes + lane;
  int up = lane < nodes ? parents[at] : kNone;
  if (up >= lane || up < kRoot) up = kNone;      // a parent comes before its children
  uint32_t lo = lane < 32 ? 1u << lane : 0u, hi = lane < 32 ? 0u : 1u << (lane - 32);
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    const int from = up < 0 ? lane : up;
    const uint32_t l = __shfl(lo, from), h = __shfl(hi, from);
    const int next = __shfl(up, from);
    if (up >= 0) {
      lo |= l;
      hi |= h;
      up = next;
    }
  }
  if (up != kRoot) lo = hi = 0;
  if (lane >= nodes) return;
  masks[at] = (uint64_t)hi << 32 | lo;
  if (depths) depths[at] = __popc(lo) + __popc(hi) - 1;
}

}  // namespace

hipError_t launch_tree_masks(int batch, int nodes, const int32_t* parents, uint64_t* masks,
                             int32_t* depths, hipStream_t st) {
  hipLaunchKernelGGL(tree_masks_kernel, dim3((batch + 3) / 4), dim3(256), 0, st, parents, masks,
                     depths, batch, nodes);
  return hipGetLastError();
}

}  // namespace moe
