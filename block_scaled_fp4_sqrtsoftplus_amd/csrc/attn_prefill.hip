// Attention over packed prompts (include/moe_attn.h, moe_attn_prefill).
//
// Mathematics: one pass over the keys with the running maximum m and sum l of
// a softmax in base 2: m' = max(m, s2), p = 2^(s2 - m'), o = o 2^(m - m') + p v,
// s2 = scale log2(e) q.k, out = o / l.
//
// Matrix form: S^T = K Q^T and O^T = V^T P^T on 32x32x16 bf16 MFMA.  A wave
// owns 32 rows; lane % 32 is the row in both products, so m, l and the
// rescaling are per lane (and its partner lane + 32), and the P that the first
// product leaves is the second's operand register for register: lane half hh =
// lane / 32 holds keys 16 c + 4 hh + (0..3) and 16 c + 8 + 4 hh + (0..3) of a
// 32-key tile in 8 consecutive registers, and the second product contracts 16 keys in
// whatever order both operands share.  Its V^T operand, 4 keys of one column
// per register pair, comes out of row-major V in LDS by the transposing LDS
// read.
//
// Rows: the heads of one key-value head's group are packed into the row
// index (row = token * group + head in the group), so a workgroup's rows span
// few tokens: short prompts fill their tiles and little is computed above the
// diagonal.
#include <algorithm>

#include "attn_internal.h"

namespace moe {

namespace {

struct PrefillArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* out;
  float* lse;
  int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh, o_st, o_sh;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int64_t tokens, tokens_kv;
  int batch, hq, hkv, group, causal, window;
  uint32_t q_flip;        // sign bits to flip in q: scale2 is |scale| log2(e)
  float scale2;
};

struct Seq {
  int b, q0, qn, k0, kn, tile;
};

__device__ __forceinline__ int clamped(const int32_t* cu, int i, int64_t most) {
  return (int)min((int64_t)max(cu[i], 0), most);
}

// The sequence and row tile of tile number `tile` (BM rows each; long rows of
// a sequence, which see the most keys, come first).
template <int BM>
__device__ __forceinline__ bool find_tile(const PrefillArgs& p, int tile, Seq& s) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 64) {
    const int b = b0 + lane;
    int n = 0;
    if (b < p.batch) {
      const int64_t rows =
          (int64_t)max(clamped(p.cu_q, b + 1, p.tokens) - clamped(p.cu_q, b, p.tokens), 0) *
          p.group;
      n = (int)((rows + BM - 1) / BM);
    }
    int incl = n;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(incl, off);
      if (lane >= off) incl += o;
    }
    const uint64_t past = __ballot(base + incl > tile);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int tiles = __builtin_amdgcn_readlane(n, l);
      const int t0 = base + __builtin_amdgcn_readlane(incl, l) - tiles;
      s.b = __builtin_amdgcn_readfirstlane(b0 + l);
      s.tile = tiles - 1 - (tile - t0);
      s.q0 = clamped(p.cu_q, s.b, p.tokens);
      s.qn = clamped(p.cu_q, s.b + 1, p.tokens) - s.q0;
      s.k0 = clamped(p.cu_k, s.b, p.tokens_kv);
      s.kn = max(clamped(p.cu_k, s.b + 1, p.tokens_kv) - s.k0, 0);
      return true;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// 16-byte chunk c of row r of a K or V tile in LDS: the position inside the row is permuted
// so that the reads below touch every bank once.  K: a wave reads one chunk
// of 32 rows.  V: the transposing read takes 4 chunks of 4 rows.

// 16-byte chunk c of row r of a K or V tile in LDS sits at chunk c ^ swz(r) of
// the row, so that the reads below touch every bank once.  K: 16 lanes read
// one chunk of 16 rows.  V: the transposing read takes 4 chunks of 4 rows.
template <int D>
__device__ __forceinline__ int k_swz(int r) {
  return D == 64 ? (r >> 1) & 7 : r & 15;
}
template <int D>
__device__ __forceinline__ int v_swz(int r) {
  return D == 64 ? 4 * ((r >> 1) & 1) : 4 * (r & 3);
}
template <int D>
__device__ __forceinline__ int k_at(int r, int c) {
  return (r * (D / 8) + ((c & 15) ^ k_swz<D>(r))) * 16 + (c & ~15) * 16;
}
template <int D>
__device__ __forceinline__ int v_at(int r, int c) {
  return (r * (D / 8) + ((c & 15) ^ v_swz<D>(r))) * 16 + (c & ~15) * 16;
}

// SPLIT waves share 32 rows (each has a D / SPLIT slice of both products'
// columns, and they add their parts of S through LDS); 4 such groups make the
// workgroup.  OCC: workgroups per CU the registers are held to, in waves per SIMD.
template <int D, int BN, int SPLIT, int OCC>
__global__ __launch_bounds__(256 * SPLIT, OCC) void attn_prefill_kernel(PrefillArgs p) {
  constexpr int BM = 128;
  constexpr int TH = 256 * SPLIT;
  constexpr int NF = D / 16 / SPLIT;         // K fragments of a wave per 32 keys
  constexpr int ND = D / 32 / SPLIT;         // its column blocks of O
  constexpr int NK = BN / 32;                // 32-key tiles per step
  constexpr int C = D / 8;                   // 16-byte chunks per row
  constexpr int LD = BN * C / TH;           // chunks a thread stages per tensor
  constexpr int TB = BN * D * 2;             // bytes of one tile
  constexpr int XB = SPLIT > 1 ? 4 * SPLIT * NK * 4096 : 0;   // the waves' parts of S
  __shared__ __align__(16) char lds[4 * TB + XB];   // K, K, V, V, S
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave = wv / SPLIT, part = wv % SPLIT;   // row group, slice of the columns
  const int col = lane & 31, hh = lane >> 5;

  // workgroups go to the 8 XCDs in turn: a key-value head stays on one XCD
  int h, tile;
  {
    const int w = blockIdx.x;
    if (p.hkv % 8 == 0) {
      const int per = p.hkv / 8, i = w >> 3;
      h = (w & 7) * per + i % per;
      tile = i / per;
    } else {
      h = w % p.hkv;
      tile = w / p.hkv;
    }
  }
  Seq s;
  if (!find_tile<BM>(p, tile, s)) return;

  // this lane's row, and the keys it keeps: [row_lo, row_hi)
  const int64_t rows = (int64_t)s.qn * p.group;
  const int64_t row0 = (int64_t)s.tile * BM;
  const int64_t row = row0 + wave * 32 + col;
  const bool live = row < rows;
  const int tok = (int)(min(row, rows - 1) / p.group);
  const int head = h * p.group + (int)(min(row, rows - 1) - (int64_t)tok * p.group);
  const int end = s.kn - s.qn + tok + 1;
  const int row_hi = p.causal ? max(min(end, s.kn), 0) : s.kn;
  const int row_lo = p.window > 0 ? max(end - p.window, 0) : 0;
  // the same over the workgroup's rows and over the wave's
  const int tok_a = (int)(row0 / p.group);
  const int tok_z = (int)((min(row0 + BM, rows) - 1) / p.group);
  const int wtok_a = (int)(min(row0 + wave * 32, rows - 1) / p.group);
  const int wtok_z = (int)(min(row0 + wave * 32 + 31, rows - 1) / p.group);
  auto hi_of = [&](int t) { return p.causal ? max(min(s.kn - s.qn + t + 1, s.kn), 0) : s.kn; };
  auto lo_of = [&](int t) { return p.window > 0 ? max(s.kn - s.qn + t + 1 - p.window, 0) : 0; };
  const int key_lo = lo_of(tok_a) / BN * BN, key_hi = hi_of(tok_z);
  const int all_lo = lo_of(wtok_z), all_hi = hi_of(wtok_a);   // kept by every row of the wave
  const int any_lo = lo_of(wtok_a), any_hi = hi_of(wtok_z);   // kept by some row of it

  bf16x8 qf[NF];
  {
    const uint16_t* qp = p.q + (s.q0 + tok) * p.q_st + head * p.q_sh;
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      u32x4 w = *reinterpret_cast<const u32x4*>(qp + 16 * (part * NF + j) + 8 * hh);
      w ^= p.q_flip;
      qf[j] = __builtin_bit_cast(bf16x8, w);
    }
  }
  f32x16 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m = kNoMax, l = 0.f;

  // Staging: chunk i of a thread is chunk tid + TH i of the tile, in row
  // r0 + RS i.  Its place in the row is permuted on the global side, since the
  // load writes LDS in lane order.  Rows past the last key repeat it (their
  // weights are zero, and the row is finite).
  constexpr int RS = TH / C;
  const char* kb = reinterpret_cast<const char*>(p.k + s.k0 * p.k_st + h * p.k_sh);
  const char* vb = reinterpret_cast<const char*>(p.v + s.k0 * p.v_st + h * p.v_sh);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  const int r0 = tid / C, c0 = tid % C;
  auto fetch = [&](int which, int buf, int key0) {   // which: 0 K, 1 V
    const char* base = which ? vb : kb;
    const int64_t st = 2 * (which ? p.v_st : p.k_st);
    const uint32_t to = lds0 + (2 * which + buf) * TB + wv * 1024;
    const bool whole = key0 + BN <= s.kn;
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const int c = c0 ^ (which ? v_swz<D>(r0 + RS * i) : k_swz<D>(r0 + RS * i));
      if (whole)
        load_lds16(to + i * TH * 16, base + (key0 + RS * i) * st, (uint32_t)(r0 * (int)st + 16 * c));
      else
        load_lds16(to + i * TH * 16, base + key0 * st,
                   (uint32_t)(min(r0 + RS * i, s.kn - 1 - key0) * (int)st + 16 * c));
    }
  };
  const int steps = key_hi > key_lo ? (key_hi - key_lo + BN - 1) / BN : 0;
  if (steps > 0) {
    fetch(0, 0, key_lo);
    fetch(1, 0, key_lo);
  }
  step_barrier();
  for (int it = 0; it < steps; ++it) {
    const int key0 = key_lo + it * BN;
    const int buf = it & 1;
    const bool mine = key0 < any_hi && key0 + BN > any_lo;   // wave-uniform
    if (it + 1 < steps) {
      fetch(0, buf ^ 1, key0 + BN);
      fetch(1, buf ^ 1, key0 + BN);
    }
    // LDS places of this lane's first chunks: the swizzle is an exclusive or,
    // so the other chunks' places are these with some bits flipped.  For large
    // heads they are worked out anew in each step: kept over the loop they would
    // take registers that it does not have (smaller ones are 5% faster with
    // them kept).
    int ka = buf * TB + k_at<D>(col, hh);
    const int vr = 4 * hh + ((lane & 15) >> 2);
    int va = (2 + buf) * TB + v_at<D>(vr, ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1)) + (lane & 1) * 8;
    if constexpr (D >= 256) asm volatile("" : "+v"(ka), "+v"(va));
    f32x16 sc[NK];
    if (mine) {
#pragma unroll
      for (int t = 0; t < NK; ++t) {
#pragma unroll
        for (int i = 0; i < 16; ++i) sc[t][i] = 0.f;
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          // chunk 2 (part NF + j) + hh of row 32 t + col
          const int c = 2 * j;
          const bf16x8 kf = __builtin_bit_cast(
              bf16x8, *reinterpret_cast<const u32x4*>(lds + (ka ^ ((c & 15) * 16)) + (c & ~15) * 16 +
                                                      part * NF * 32 + 32 * t * D * 2));
          sc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[j], sc[t], 0, 0, 0);
        }
      }
    }
    if constexpr (SPLIT == 2) {
      float* x = reinterpret_cast<float*>(lds + 4 * TB);
      if (mine) {
#pragma unroll
        for (int t = 0; t < NK; ++t)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<f32x4*>(x + ((wv * NK + t) * 4 + i / 4) * 256 + lane * 4) =
                f32x4{sc[t][i], sc[t][i + 1], sc[t][i + 2], sc[t][i + 3]};
      }
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // loads stay in flight
      if (mine) {
#pragma unroll
        for (int t = 0; t < NK; ++t)
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const f32x4 y = *reinterpret_cast<const f32x4*>(
                x + (((wv ^ 1) * NK + t) * 4 + i / 4) * 256 + lane * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[t][i + e] += y[e];
          }
      }
    }
    if (mine) {
      if (!(key0 >= all_lo && key0 + BN <= all_hi)) {
#pragma unroll
        for (int t = 0; t < NK; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = key0 + 32 * t + 8 * (i >> 2) + 4 * hh + (i & 3);
            if (key >= row_hi || key < row_lo) sc[t][i] = -INFINITY;
          }
      }
      float mx = sc[0][0];
#pragma unroll
      for (int t = 0; t < NK; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, sc[t][i]);
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      mx *= p.scale2;
      if (__ballot(mx > m + kLag)) {
        const float mn = fmaxf(m, mx);
        const float a = exp2_fast(m - mn);
        m = mn;
        l *= a;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[d][i] *= a;
      }
#pragma unroll
      for (int t = 0; t < NK; ++t) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          sc[t][i] = exp2_fast(fmaf(sc[t][i], p.scale2, -m));
          l += sc[t][i];
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          u32x4 pw;
#pragma unroll
          for (int i = 0; i < 4; ++i) pw[i] = pack_bf16(sc[t][8 * c + 2 * i], sc[t][8 * c + 2 * i + 1]);
          const bf16x8 pf = __builtin_bit_cast(bf16x8, pw);
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            // chunks 4 (part ND + d) + .. of rows 32 t + 16 c + vr and 8 below
            const int ch = 4 * d;
            const char* v0 = lds + (va ^ ((ch & 15) * 16)) + (ch & ~15) * 16 + part * ND * 64 +
                             (32 * t + 16 * c) * D * 2;
            const bf16x8 vf = read_tr(v0, v0 + 8 * D * 2);
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf, o[d], 0, 0, 0);
          }
        }
      }
    }
    step_barrier();
  }

  l += __shfl_xor(l, 32);
  if (!live) return;
  const float inv = l > 0.f ? 1.0f / l : 0.f;
  uint16_t* dst = p.out + (s.q0 + tok) * p.o_st + head * p.o_sh;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const u32x2 w = {pack_bf16(o[d][i] * inv, o[d][i + 1] * inv),
                       pack_bf16(o[d][i + 2] * inv, o[d][i + 3] * inv)};
      *reinterpret_cast<u32x2*>(dst + 32 * (part * ND + d) + 2 * i + 4 * hh) = w;
    }
  if (p.lse && hh == 0 && part == 0)
    p.lse[(int64_t)(s.q0 + tok) * p.hq + head] =
        l > 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

hipError_t launch_attn_prefill(const moe_attn_config& c, const moe_rows& q, const moe_rows& k,
                               const moe_rows& v, const int32_t* cu_q, const int32_t* cu_k,
                               const moe_rows& out, float* lse, hipStream_t st) {
  if (c.batch == 0 || c.tokens == 0) return hipSuccess;
  PrefillArgs a{};
  a.q = q.p; a.q_st = q.stride_token; a.q_sh = q.stride_head;
  a.k = k.p; a.k_st = k.stride_token; a.k_sh = k.stride_head;
  a.v = v.p; a.v_st = v.stride_token; a.v_sh = v.stride_head;
  a.out = out.p; a.o_st = out.stride_token; a.o_sh = out.stride_head;
  a.lse = lse;
  a.cu_q = cu_q; a.cu_k = cu_k;
  a.tokens = c.tokens; a.tokens_kv = c.tokens_kv;
  a.batch = c.batch; a.hq = c.heads_q; a.hkv = c.heads_kv; a.group = c.heads_q / c.heads_kv;
  a.causal = c.causal; a.window = c.window;
  a.q_flip = c.scale < 0.f ? 0x80008000u : 0u;
  a.scale2 = (c.scale < 0.f ? -c.scale : c.scale) * kLog2e;
  // at most one partly filled tile per sequence
  const int64_t tiles =
      c.tokens * a.group / 128 + std::min<int64_t>(c.batch, c.tokens);
  const dim3 grid((unsigned)(tiles * c.heads_kv));
#define MOE_PREFILL(D, BN, SPLIT, OCC)                                                        \
  case D:                                                                                     \
    hipLaunchKernelGGL((attn_prefill_kernel<D, BN, SPLIT, OCC>), grid, dim3(256 * SPLIT), 0, st, \
                       a);                                                                    \
    break;
  switch (c.head_dim) {
    MOE_PREFILL(64, 64, 1, 2)
    MOE_PREFILL(128, 64, 1, 2)
    MOE_PREFILL(256, 32, 1, 2)
    MOE_PREFILL(512, 32, 2, 2)
    default: return hipErrorInvalidValue;
  }
#undef MOE_PREFILL
  return hipGetLastError();
}

}  // namespace moe
