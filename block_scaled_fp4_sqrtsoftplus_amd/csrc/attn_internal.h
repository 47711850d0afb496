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

// The larger of a lane's and its partner's (lane ^ 32) value, in both.
__device__ __forceinline__ float halves_max(float x) {
  const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// The same over the four lanes that share lane % 16.
__device__ __forceinline__ float quarters_max(float x) {
  const u32x2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return halves_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}

// Sum of x over this lane and the lanes before it.
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);   // row_shr 1, 2, 4, 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);   // lane 15 of a row to the next
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);   // lane 31 to rows 2 and 3
  return x;
}

// Transposing LDS read: the 16 lanes of a quarter wave give the addresses of
// 4 rows of 16 16-bit elements (lane i: row i / 4, elements 4 (i % 4) ..) and
// lane i gets the 4 rows' element i.  Two of them are one bf16x8 operand of an MFMA.
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

__device__ __forceinline__ bf16x8 read_tr(const char* a, const char* b) {
  const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)a);
  const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)b);
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
}

// One asynchronous load of 16 bytes per lane from base + off into LDS at byte
// `to` (wave-uniform) + 16 * lane.  In assembly because the compiler would
// wait for it before the next LDS read, which never reads what it writes: the
// kernels wait at the end of a step.  (m0 is this instruction's
// alone: no other of the kernel's uses it.)
__device__ __forceinline__ void load_lds16(uint32_t to, const char* base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(off), "s"(base)
               : "memory");
}

// Ends a step: all but the last N of this wave's asynchronous loads have
// landed, and every wave is done with the step's tiles.
template <int N>
__device__ __forceinline__ void step_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The waves' LDS writes are seen by all; asynchronous loads stay on their way.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Waits here for a value's load.  Before a loop with asynchronous loads: the
// compiler would otherwise wait at the value's first use inside, each time
// round, and with it for the loads that it does not know of.
template <class T>
__device__ __forceinline__ void arrived(const T& x) {
  asm volatile("" ::"v"(x));
}

// The running maximum follows the scores only when one passes it by more than
// this (base 2): weights then reach 2^kLag, which fp32 sums and bf16's
// exponent hold as well, and the output is seldom rescaled.
constexpr float kLag = 8.f;

// A launch takes less than 2^32 work-items: more workgroups than that go out in
// several, each of which is told the number of its first one.  2^22 of up to
// 512 work-items each, and a multiple of the 8 XCDs that workgroups go to in turn.
template <class Launch>
hipError_t launch_workgroups(int64_t count, Launch launch) {
  constexpr int64_t kMost = int64_t(1) << 22;
  for (int64_t first = 0; first < count; first += kMost) {
    const int64_t n = count - first < kMost ? count - first : kMost;
    launch((uint32_t)first, dim3((unsigned)n));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

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
