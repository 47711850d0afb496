// Append to the paged key-value cache with the position rotation on the way
// (include/moe_attn.h, moe_kv_append).
//
// Mathematics: y_a = a cos - b sin, y_b = b cos + a sin per pair in fp32 (each product and sum
// rounded, no contraction), one rounding to bf16; an FP8 cache then takes the
// bf16 row as quant_act_block does: per 128 elements (or the 64 of a short
// row) the smallest 2^e with max|y| <= 448 * 2^e.
//
// Bound by memory: every row is read once and written once.  A lane owns 8
// elements (16 bytes of bf16) of a head, D / 8 lanes a head, so a wave moves
// whole lines of 64 / (D / 8) heads at once; a pair's other half sits in
// another lane of the same head and comes by a lane shuffle, so q_out may be
// q.  A wave keeps one token's cosines and sines in registers and goes through
// that token's heads (q, then k, then v); few tokens split their heads over
// more waves instead.
//
// Measured: 4099 tokens of 32 + 8 + 8 heads of 128 in bf16 21.4 us (4.8 TB/s read and
// written, a large copy's rate), 16384 of them into an FP8 cache 80.6 us
// (4.7 TB/s), 64 tokens on one 512-element FP8 head 5.9 us and one token
// 5.0 us, of which a launch is 4.
#include <algorithm>

#include "attn_internal.h"

namespace moe {

namespace {

struct AppendArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;       // null: the cache's values are its keys
  uint16_t* q_out;
  uint16_t* k_out;         // may be null
  int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh, qo_st, qo_sh, ko_st, ko_sh;
  char* ck;
  char* cv;
  uint8_t* cks;
  uint8_t* cvs;
  uint8_t* cks2;             // the values' scales where one tensor of codes has two arrays of them, or null
  int64_t c_sp, c_sh, c_st;  // elements
  int64_t slots_end;         // pages * page_size
  int page_shift;
  const int64_t* slots;
  const int32_t* positions;
  const float* cos_sin;      // null: no rotation
  int64_t n_pos;
  int64_t tokens;
  int rot_dim, rot_offset, interleaved;
  int hq, hk, hv;            // heads of q, k and v to go through
  int parts;                 // waves that share one token's heads
  uint32_t first;            // the launch's first workgroup
};

// lane's 8 elements rotated (see the formulas above); partner values by
// shuffle.  c8 / s8: cosines and sines of the lane's 8 (halves) or first 4
// (neighbours) pairs; role: -1 outside the rotated part, 0 first half, 1
// second half, 2 neighbours.
__device__ __forceinline__ u32x4 rotate8(u32x4 x, const float* c8, const float* s8, int role,
                                         int partner) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = (uint32_t)__shfl((int)x[i], partner);
  if (role < 0) return x;
  u32x4 y;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = bf16_to_f32(x[i] & 0xFFFFu), hi = bf16_to_f32(x[i] >> 16);
    if (role == 2) {
      y[i] = pack_bf16(lo * c8[i] - hi * s8[i], hi * c8[i] + lo * s8[i]);
    } else {
      const float plo = bf16_to_f32(o[i] & 0xFFFFu), phi = bf16_to_f32(o[i] >> 16);
      const float a0 = lo * c8[2 * i], b0 = plo * s8[2 * i];
      const float a1 = hi * c8[2 * i + 1], b1 = phi * s8[2 * i + 1];
      y[i] = role == 0 ? pack_bf16(a0 - b0, a1 - b1) : pack_bf16(a0 + b0, a1 + b1);
    }
  }
  return y;
}

// STREAM: rows read past the caches (see the launch).
template <int D, bool FP8, bool STREAM>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendArgs p) {
  constexpr int LPR = D / 8;          // lanes per head
  constexpr int RPW = 64 / LPR;       // heads per wave and step
  constexpr int GROUP = D < 128 ? D / 8 : 16;   // lanes per FP8 scale
  constexpr int NG = D < 128 ? 1 : D / 128;
  const int lane = threadIdx.x & 63;
  const int64_t wave = ((int64_t)p.first + blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int64_t t = wave / p.parts;
  const int part = (int)(wave - t * p.parts);
  if (t >= p.tokens) return;
  const int c = lane % LPR, sub = lane / LPR;
  const int e0 = 8 * c;               // the lane's first element

  // the token's rotation, for this lane's elements
  float c8[8], s8[8];
  int role = -1, partner = lane;
  if (p.cos_sin) {
    const int r = e0 - p.rot_offset, half = p.rot_dim / 2;
    if (r >= 0 && r < p.rot_dim) {
      role = p.interleaved ? 2 : r >= half ? 1 : 0;
      if (role == 0) partner = lane + half / 8;
      if (role == 1) partner = lane - half / 8;
      const int64_t pos = p.positions[t];
      const bool known = pos >= 0 && pos < p.n_pos;
      const float* row = p.cos_sin + (known ? pos : 0) * p.rot_dim;
      const float bad = __uint_as_float(0x7FC00000u);
      const int i0 = p.interleaved ? r / 2 : role == 1 ? r - half : r;
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        if (i == 0 || !p.interleaved) {
          const f32x4 cv = *reinterpret_cast<const f32x4*>(row + i0 + i);
          const f32x4 sv = *reinterpret_cast<const f32x4*>(row + half + i0 + i);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            c8[i + j] = known ? cv[j] : bad;
            s8[i + j] = known ? sv[j] : bad;
          }
        }
      }
    }
  }
  const int64_t slot = p.slots[t];
  const bool stored = slot >= 0 && slot < p.slots_end;
  const int64_t page = slot >> p.page_shift;
  const int in_page = (int)(slot & ((int64_t(1) << p.page_shift) - 1));

  const int rows = p.hq + p.hk + p.hv;
  for (int r0 = part * RPW; r0 < rows; r0 += p.parts * RPW) {
    const int r = r0 + sub;
    const bool live = r < rows;
    const bool is_q = r < p.hq, is_k = !is_q && r < p.hq + p.hk;
    const int h = is_q ? r : is_k ? r - p.hq : r - p.hq - p.hk;
    const uint16_t* src = is_q ? p.q + t * p.q_st + h * p.q_sh
                        : is_k ? p.k + t * p.k_st + h * p.k_sh
                               : p.v + t * p.v_st + h * p.v_sh;
    u32x4 x = {0, 0, 0, 0};
    if (live) x = STREAM ? wload<u32x4>(src + e0) : *reinterpret_cast<const u32x4*>(src + e0);
    u32x4 y = rotate8(x, c8, s8, live && (is_q || is_k) ? role : -1, partner);
    if (live && is_q) *reinterpret_cast<u32x4*>(p.q_out + t * p.qo_st + h * p.qo_sh + e0) = y;
    if (live && is_k && p.k_out)
      *reinterpret_cast<u32x4*>(p.k_out + t * p.ko_st + h * p.ko_sh + e0) = y;
    const bool put = live && !is_q && stored;
    const int64_t at = page * p.c_sp + h * p.c_sh + (int64_t)in_page * p.c_st + e0;
    char* dst = is_k ? p.ck : p.cv;
    if constexpr (!FP8) {
      if (put) *reinterpret_cast<u32x4*>(dst + 2 * at) = y;
    } else {
      float f[8];
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_to_f32(y[i] & 0xFFFFu);
        f[2 * i + 1] = bf16_to_f32(y[i] >> 16);
        amax = fmaxf(amax, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
      }
#pragma unroll
      for (int off = 1; off < GROUP; off <<= 1) amax = fmaxf(amax, __shfl_xor(amax, off));
      const int e = pow2_scale_exp(amax);
      if (put) {
        const float a[4] = {f[0], f[1], f[2], f[3]}, b[4] = {f[4], f[5], f[6], f[7]};
        const u32x2 code = {e4m3x4_exp(a, e), e4m3x4_exp(b, e)};
        *reinterpret_cast<u32x2*>(dst + at) = code;
        if (c % GROUP == 0) {
          uint8_t* sc = is_k ? p.cks : p.cvs;
          const int64_t i =
              ((page * p.hk + h) * (int64_t(1) << p.page_shift) + in_page) * NG + c / GROUP;
          sc[i] = (uint8_t)(e + 127);
          if (p.cks2) p.cks2[i] = (uint8_t)(e + 127);
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_kv_append(const moe_kv_cache& c, const moe_rope* rope, int64_t tokens,
                            const int64_t* slots, const int32_t* positions, const moe_rows& k,
                            const moe_rows* v, int heads_q, const moe_rows* q,
                            const moe_rows* q_out, const moe_rows* k_out, hipStream_t st) {
  if (tokens == 0) return hipSuccess;
  AppendArgs a{};
  a.k = k.p; a.k_st = k.stride_token; a.k_sh = k.stride_head;
  if (v) { a.v = v->p; a.v_st = v->stride_token; a.v_sh = v->stride_head; }
  if (q) { a.q = q->p; a.q_st = q->stride_token; a.q_sh = q->stride_head; }
  if (q) { a.q_out = q_out->p; a.qo_st = q_out->stride_token; a.qo_sh = q_out->stride_head; }
  if (k_out) { a.k_out = k_out->p; a.ko_st = k_out->stride_token; a.ko_sh = k_out->stride_head; }
  a.ck = static_cast<char*>(c.k); a.cv = static_cast<char*>(c.v);
  a.cks = c.k_scale; a.cvs = c.v_scale;
  a.cks2 = !v && c.v_scale != c.k_scale ? c.v_scale : nullptr;
  a.c_sp = c.stride_page; a.c_sh = c.stride_head; a.c_st = c.stride_token;
  a.slots_end = c.pages * c.page_size;
  a.page_shift = __builtin_ctz((unsigned)c.page_size);
  a.slots = slots; a.positions = positions; a.tokens = tokens;
  if (rope) {
    a.cos_sin = rope->cos_sin; a.n_pos = rope->positions; a.rot_dim = rope->rot_dim;
    a.rot_offset = rope->rot_offset; a.interleaved = rope->interleaved;
  }
  a.hq = q ? heads_q : 0; a.hk = c.heads; a.hv = v ? c.heads : 0;
  const int rpw = 64 / (c.head_dim / 8);
  const int steps = (a.hq + a.hk + a.hv + rpw - 1) / rpw;
  // Waves that share a token's heads: as many as make 4096 waves (4 per SIMD),
  // or 16384 where each still has 4 steps.  4099 tokens of 48 rows of 128 elements:
  // 22.3 us with one wave a token, 20.4 with three; 1000 such tokens 7.3 us
  // with four waves a token, 8.6 with twelve.
  a.parts = (int)std::clamp<int64_t>(
      std::max<int64_t>(4096 / tokens, std::min<int64_t>(16384 / tokens, steps / 4)), 1, steps);
  // Rows of a projection that has just been written sit in the caches (256
  // MB), unless they are most of it: 200 MB of rows take 67 us read past the
  // caches and 94 through them, 50 MB the same, 12 MB 9.8 and 7.3.
  const bool stream = tokens * (a.hq + a.hk + a.hv) * c.head_dim * 2 > (int64_t(64) << 20);
  const int64_t waves = tokens * a.parts;
#define MOE_APPEND_S(D, F)                                                                   \
  do {                                                                                       \
    if (stream)                                                                              \
      hipLaunchKernelGGL((kv_append_kernel<D, F, true>), grid, dim3(256), 0, st, a);         \
    else                                                                                     \
      hipLaunchKernelGGL((kv_append_kernel<D, F, false>), grid, dim3(256), 0, st, a);        \
  } while (0)
#define MOE_APPEND(D)                                                                        \
  case D:                                                                                    \
    if (c.format == MOE_KV_FP8) MOE_APPEND_S(D, true); else MOE_APPEND_S(D, false);          \
    break;
  return launch_workgroups((waves + 3) / 4, [&](uint32_t first, dim3 grid) {
    a.first = first;
    switch (c.head_dim) {
      MOE_APPEND(64) MOE_APPEND(128) MOE_APPEND(256) MOE_APPEND(512)
    }
  });
#undef MOE_APPEND
#undef MOE_APPEND_S
}

}  // namespace moe
