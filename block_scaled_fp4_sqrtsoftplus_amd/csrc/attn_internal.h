// Internal declarations of the attention sources (include/moe_attn.h): vector
// types, small device helpers and the kernel launchers.
#pragma once

#include "moe_attn.h"
#include "moe_internal.h"

namespace moe {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Stands for "nothing kept yet" in a running maximum: finite, so that the
// difference of two of them is 0 and not NaN, and below any score a finite
// input of use gives.
constexpr float kNoMax = -1.0e38f;

// Two fp32 -> packed bf16 (a in the low half), round to nearest even, NaN kept.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// 2^x by the hardware's exponential (about 1 ulp; 0 far below).
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Device check and cached properties (api.cpp).
moe_status device_ok();

hipError_t launch_kv_append(const moe_kv_cache& c, const moe_rope* rope, int64_t tokens,
                            const int64_t* slots, const int32_t* positions, const moe_rows& k,
                            const moe_rows* v, int heads_q, const moe_rows* q,
                            const moe_rows* q_out, const moe_rows* k_out, hipStream_t st);

size_t attn_decode_ws_bytes(const moe_attn_config& c);
hipError_t launch_attn_decode(const moe_attn_config& c, const moe_rows& q, const moe_kv_cache& kv,
                              const int32_t* table, int table_width, const int32_t* seq_lens,
                              const moe_rows& out, float* lse, void* ws, hipStream_t st);

hipError_t launch_attn_prefill(const moe_attn_config& c, const moe_rows& q, const moe_rows& k,
                               const moe_rows& v, const int32_t* cu_q, const int32_t* cu_k,
                               const moe_rows& out, float* lse, hipStream_t st);

}  // namespace moe
