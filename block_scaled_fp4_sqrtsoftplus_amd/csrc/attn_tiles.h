// Places of K and V in the LDS tiles of the kernels on 32x32x16 MFMA
// (attn_prefill_kernel.h, attn_tree_rows.hip).
#pragma once

#include "attn_internal.h"

namespace moe {

namespace {

// 16-byte chunk c of row r of a K or V tile in LDS sits at chunk c ^ swz(r) of
// the row, so that the reads below touch every bank once.  K: 16 lanes read
// one chunk of 16 rows.  V: the transposing read takes 4 chunks of 4 rows.
// 512-element heads have one permutation for both, so that a tile may be both.
template <int D>
__device__ __forceinline__ int k_swz(int r) {
  return D == 64 ? (r >> 1) & 7 : D == 512 ? ((r & 3) << 2) | ((r >> 2) & 3) : r & 15;
}
template <int D>
__device__ __forceinline__ int v_swz(int r) {
  return D == 64 ? 4 * ((r >> 1) & 1) : D == 512 ? k_swz<D>(r) : 4 * (r & 3);
}
template <int D>
__device__ __forceinline__ int k_at(int r, int c) {
  return (r * (D / 8) + ((c & 15) ^ k_swz<D>(r))) * 16 + (c & ~15) * 16;
}
template <int D>
__device__ __forceinline__ int v_at(int r, int c) {
  return (r * (D / 8) + ((c & 15) ^ v_swz<D>(r))) * 16 + (c & ~15) * 16;
}

}  // namespace

}  // namespace moe
