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
//
// P is rounded to bf16 as v is, its sum taken before: outputs are 2.0e-3 from the
// exact ones in the 2-norm, of which their own rounding is 1.6e-3.  P as the sum of
// two bf16 values would be a second product with V, half as many matrix
// instructions again where they are the bound.
//
// Measured (TFLOP/s count what the mask leaves): 8192 tokens, 32 heads of 128 on 8
// 502 to 519 us (1094 to 1060 TFLOP/s): matrix units busy for 58% of the cycles at a clock that the load
// brings down to 1.6 to 1.8 GHz, no LDS bank conflict; where the exponentials
// and loads stand between the products makes no difference there any more.  Six packed prompts 77 us
// (708), 2048 tokens of 64 heads on one 512-element head that is keys and
// values 304 us (903), 200 tokens of 16 heads of 64 7.6 us, all latencies.
#include <algorithm>
#include <type_traits>

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
  uint32_t first;         // the launch's first workgroup
  uint32_t q_flip;        // sign bits to flip in q: scale2 is |scale| log2(e)
  float scale2;
};

struct Seq {
  int q0, qn, k0, kn, tile;
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
    int n = 0, q0 = 0, q1 = 0, k0 = 0, k1 = 0;   // a sequence per lane
    if (b < p.batch) {
      q0 = clamped(p.cu_q, b, p.tokens);
      q1 = clamped(p.cu_q, b + 1, p.tokens);
      k0 = clamped(p.cu_k, b, p.tokens_kv);
      k1 = clamped(p.cu_k, b + 1, p.tokens_kv);
      const int64_t rows = (int64_t)max(q1 - q0, 0) * p.group;
      n = (int)((rows + BM - 1) / BM);
    }
    const int incl = wave_scan(n);
    const uint64_t past = __ballot(base + incl > tile);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int tiles = __builtin_amdgcn_readlane(n, l);
      const int t0 = base + __builtin_amdgcn_readlane(incl, l) - tiles;
      s.tile = tiles - 1 - (tile - t0);
      s.q0 = __builtin_amdgcn_readlane(q0, l);
      s.qn = __builtin_amdgcn_readlane(q1, l) - s.q0;
      s.k0 = __builtin_amdgcn_readlane(k0, l);
      s.kn = max(__builtin_amdgcn_readlane(k1, l) - s.k0, 0);
      return true;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

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

// RG row groups of 32 rows; SPLIT waves share a group (each has a D / SPLIT
// slice of both products' columns, and they add their parts of S through
// LDS).  BN: keys per step.  BUFS: LDS tiles of K and of V, BUFS - 1 of them on
// their way while one is read (with ONE, where v is k, of the one tensor: three).
// PIPE: a step takes the weights of its scores while the matrix units take the
// next step's scores.  AHEAD: products by which LDS reads run ahead of their use,
// where their order is fixed by hand.  WAVES: waves per SIMD that the registers are
// held to, where the LDS holds as many (256-element heads: 96 KB, one wave and more registers).
template <int D, int BN, int RG, int SPLIT, int BUFS, bool PIPE, int AHEAD, int WAVES, bool ONE>
__global__ __launch_bounds__(64 * RG * SPLIT, WAVES) void attn_prefill_kernel(PrefillArgs p) {
  constexpr int BM = 32 * RG;
  constexpr int TH = 64 * RG * SPLIT;
  constexpr int NF = D / 16 / SPLIT;         // K fragments of a wave per 32 keys
  constexpr int ND = D / 32 / SPLIT;         // its column blocks of O
  constexpr int NK = BN / 32;                // 32-key tiles per step
  constexpr int C = D / 8;                   // 16-byte chunks per row
  constexpr int LD = BN * C / TH;            // chunks a thread stages per tensor
  constexpr int TB = BN * D * 2;             // bytes of one tile
  constexpr int V0 = ONE ? 0 : BUFS * TB;    // the tiles of V
  constexpr int X0 = (ONE ? BUFS : 2 * BUFS) * TB;   // the waves' parts of S
  constexpr int XB = SPLIT > 1 ? RG * SPLIT * NK * 4096 : 0;
  __shared__ __align__(16) char lds[X0 + XB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave = wv / SPLIT, part = wv % SPLIT;   // row group, slice of the columns
  const int col = lane & 31, hh = lane >> 5;

  // 512-element heads work what depends on the lane out anew each time, from the one
  // register that holds it
  auto here = [&]() {
    int l = lane;
    asm volatile("" : "+v"(l));
    return l;
  };

  // workgroups go to the 8 XCDs in turn: a key-value head stays on one XCD
  int h, tile;
  {
    const int w = p.first + blockIdx.x;
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
  const int64_t my_row = min(row0 + wave * 32 + col, rows - 1);
  const int my_tok = (int)(my_row / p.group);
  const int end = s.kn - s.qn + my_tok + 1;
  const int row_hi = p.causal ? max(min(end, s.kn), 0) : s.kn;
  const int row_lo = p.window > 0 ? max(end - p.window, 0) : 0;
  // the same over the workgroup's rows and over the wave's
  const int tok_a = (int)(row0 / p.group);
  const int tok_z = (int)((min(row0 + BM, rows) - 1) / p.group);
  const int wtok_a = (int)(min(row0 + wave * 32, rows - 1) / p.group);
  const int wtok_z = (int)(min(row0 + wave * 32 + 31, rows - 1) / p.group);
  auto hi_of = [&](int t) { return p.causal ? max(min(s.kn - s.qn + t + 1, s.kn), 0) : s.kn; };
  auto lo_of = [&](int t) { return p.window > 0 ? max(s.kn - s.qn + t + 1 - p.window, 0) : 0; };
  const int key_first = lo_of(tok_a), key_lo = key_first / BN * BN, key_hi = hi_of(tok_z);
  const int all_lo = lo_of(wtok_z), all_hi = hi_of(wtok_a);   // kept by every row of the wave

  bf16x8 qf[NF];
  {
    const int head = h * p.group + (int)(my_row - (int64_t)my_tok * p.group);
    const uint16_t* qp = p.q + (s.q0 + my_tok) * p.q_st + head * p.q_sh;
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
  float m = kNoMax, l = 0.f, l2 = 0.f;   // two sums: shorter chains

  // Staging: chunk i of a thread is chunk tid + TH i of the tile, in row
  // r0 + RS i.  Its place in the row is permuted on the global side, since the
  // load writes LDS in lane order.  Rows past the last key repeat it, and rows
  // before the first key that the workgroup's rows keep repeat that one: their weights are
  // zero, but 0 * NaN is not, and the keys repeated are finite while what
  // lies outside every window may hold anything.
  constexpr int RS = TH / C;
  const char* kb = reinterpret_cast<const char*>(p.k + s.k0 * p.k_st + h * p.k_sh);
  const char* vb = reinterpret_cast<const char*>(p.v + s.k0 * p.v_st + h * p.v_sh);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  const int r0 = D == 512 ? wv : tid / C;
  // chunk i of a tile whose rows are all keys
  auto fetch_one = [&](int which, int buf, int key0, int i) {
    const int c0 = D == 512 ? here() : tid % C;
    const int64_t st = 2 * (which ? p.v_st : p.k_st);
    const int c = c0 ^ (which ? v_swz<D>(r0 + RS * i) : k_swz<D>(r0 + RS * i));
    load_lds16(lds0 + (which ? V0 : 0) + buf * TB + wv * 1024 + i * TH * 16,
               (which ? vb : kb) + (key0 + RS * i) * st, (uint32_t)(r0 * (int)st + 16 * c));
  };
  auto fetch = [&](int which, int buf, int key0) {   // which: 0 K, 1 V
    const char* base = which ? vb : kb;
    const int64_t st = 2 * (which ? p.v_st : p.k_st);
    const uint32_t to = lds0 + (which ? V0 : 0) + buf * TB + wv * 1024;
    if (key0 >= key_first && key0 + BN <= s.kn) {
#pragma unroll
      for (int i = 0; i < LD; ++i) fetch_one(which, buf, key0, i);
    } else {
#pragma unroll 1
      for (int i = 0; i < LD; ++i) {
        const int c0 = D == 512 ? here() : tid % C;
        const int c = c0 ^ (which ? v_swz<D>(r0 + RS * i) : k_swz<D>(r0 + RS * i));
        load_lds16(to + i * TH * 16, base + key0 * st,
                   (uint32_t)(min(max(r0 + RS * i, key_first - key0), s.kn - 1 - key0) * (int)st + 16 * c));
      }
    }
  };
  // LDS places of this lane's first chunks: the permutation is an exclusive or,
  // so the other chunks' places are these with some bits flipped.  For large
  // heads they are worked out anew in each step: kept over the loop they would
  // take registers that it does not have.
  const int k_once = k_at<D>(col, hh);
  const int v_once = v_at<D>(4 * hh + ((lane & 15) >> 2), ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1)) +
                     (lane & 1) * 8;
  auto k_lane = [&]() {
    if constexpr (D < 512) return k_once;
    const int l = here();
    return k_at<D>(l & 31, l >> 5);
  };
  auto v_lane = [&]() {
    if constexpr (D < 512) return v_once;
    const int l = here();
    return v_at<D>(4 * (l >> 5) + ((l & 15) >> 2), ((l >> 4) & 1) * 2 + ((l & 3) >> 1)) + (l & 1) * 8;
  };
  constexpr int QK = NK * NF, PV = 2 * NK * ND, NE = 16 * NK;
  auto read_k = [&](int ka, int i) {   // operand of QK product i: tile i % NK, columns i / NK
    const int t = i % NK, c = 2 * (i / NK);   // chunk 2 (part NF + ..) + hh of row 32 t + col
    return __builtin_bit_cast(
        bf16x8, *reinterpret_cast<const u32x4*>(lds + (ka ^ ((c & 15) * 16)) + (c & ~15) * 16 +
                                                part * NF * 32 + 32 * t * D * 2));
  };
  auto read_v = [&](int va, int i) {   // operand of PV product i: keys i / ND, columns i % ND
    const int ch = 4 * (i % ND);       // chunk 4 (part ND + ..) of rows 16 (i / ND) + .. and 8 below
    const int at = va ^ ((ch & 15) * 16);
    const char* v0 = lds + (ch & ~15) * 16 + part * ND * 64 + 16 * (i / ND) * D * 2;
    return read_tr(v0 + at, v0 + (at ^ (v_swz<D>(8) * 16)) + 8 * D * 2);
  };
  float* xs = reinterpret_cast<float*>(lds + X0);
  auto hand_over = [&](const f32x16(&sc)[NK]) {   // SPLIT 2: this wave's part for the other
    const int l = here();
#pragma unroll
    for (int t = 0; t < NK; ++t)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<f32x4*>(xs + ((wv * NK + t) * 4 + i / 4) * 256 + l * 4) =
            f32x4{sc[t][i], sc[t][i + 1], sc[t][i + 2], sc[t][i + 3]};
  };
  auto take_over = [&](f32x16(&sc)[NK]) {
    const int l = here();
#pragma unroll
    for (int t = 0; t < NK; ++t)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const f32x4 y =
            *reinterpret_cast<const f32x4*>(xs + (((wv ^ 1) * NK + t) * 4 + i / 4) * 256 + l * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[t][i + e] += y[e];
      }
  };
  // whether every row of the wave keeps all of a step's keys; if not, the mask
  auto inner = [&](int key0) { return key0 >= all_lo && key0 + BN <= all_hi; };
  auto mask = [&](int key0, f32x16(&sc)[NK]) {
    int first = key0 + 4 * (here() >> 5);
    asm volatile("" : "+v"(first));    // its places are not kept over the loop
#pragma unroll
    for (int t = 0; t < NK; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int key = first + 32 * t + 8 * (i >> 2) + (i & 3);
        if (key >= row_hi || key < row_lo) sc[t][i] = -INFINITY;
      }
  };
  auto largest = [&](const f32x16(&sc)[NK]) {
    float x[4];
#pragma unroll
    for (int i = 0; i < 16 * NK; ++i)
      x[i % 4] = i < 4 ? sc[i / 16][i % 16] : fmaxf(x[i % 4], sc[i / 16][i % 16]);
    return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
  };
  // takes the largest score of this lane's half of the row's keys
  auto raise = [&](float mx) {
    mx = halves_max(mx) * p.scale2;
    if (__ballot(mx > m + kLag)) {
      const float mn = fmaxf(m, mx);
      const float a = exp2_fast(m - mn);
      m = mn;
      l *= a;
      l2 *= a;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= a;
    }
  };

  const int steps = key_hi > key_lo ? (key_hi - key_lo + BN - 1) / BN : 0;
  auto q_arrived = [&]() {
#pragma unroll
    for (int j = 0; j < NF; ++j) arrived(__builtin_bit_cast(u32x4, qf[j]));
  };
  u32x4 pw[2 * NK];
  // the weight of element e of the step, in three parts that may be apart
  auto weight_arg = [&](f32x16(&sc)[NK], int e) {
    sc[e / 16][e % 16] = fmaf(sc[e / 16][e % 16], p.scale2, -m);
  };
  auto weight_exp = [&](f32x16(&sc)[NK], int e) {
    sc[e / 16][e % 16] = exp2_fast(sc[e / 16][e % 16]);
  };
  auto weight_sum = [&](const f32x16(&sc)[NK], int e) {
    const float w = sc[e / 16][e % 16];
    if (e & 1) {
      l2 += w;
      pw[e / 8][e / 2 % 4] = pack_bf16(sc[e / 16][e % 16 - 1], w);
    } else {
      l += w;
    }
  };
  auto weight = [&](f32x16(&sc)[NK], int e) {
    weight_arg(sc, e);
    weight_exp(sc, e);
    weight_sum(sc, e);
  };
  auto scores = [&](int buf, f32x16(&to)[NK]) {
    int ka = buf * TB + k_lane();
    if constexpr (D >= 256) asm volatile("" : "+v"(ka));
#pragma unroll
    for (int t = 0; t < NK; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) to[t][i] = 0.f;
#pragma unroll
    for (int i = 0; i < QK; ++i)
      to[i % NK] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(read_k(ka, i), qf[i / NK], to[i % NK], 0, 0, 0);
  };
  auto values = [&](int buf) {
    int va = V0 + buf * TB + v_lane();
    if constexpr (D >= 256) asm volatile("" : "+v"(va));
#pragma unroll
    for (int i = 0; i < PV; ++i)
      o[i % ND] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          read_v(va, i), __builtin_bit_cast(bf16x8, pw[i / ND]), o[i % ND], 0, 0, 0);
  };
  if constexpr (PIPE) {
    // K runs one step ahead of V.  At step it, K of it + 1 and V of it are in
    // LDS, K up to it + BUFS - 1 and V up to it + BUFS - 2 on their way.
    f32x16 sc[NK], nx[NK];
    if (steps > 0) {
#pragma unroll
      for (int i = 0; i < BUFS; ++i) {
        if (i < steps) fetch(0, i, key_lo + i * BN);
        if (i < BUFS - 1 && i < steps) fetch(1, i, key_lo + i * BN);
      }
      q_arrived();
      step_barrier<0>();
      scores(0, sc);
      if (!inner(key_lo)) mask(key_lo, sc);
      raise(largest(sc));
      step_barrier<0>();
    }
    int kb_next = 1 % BUFS, vb_now = 0;      // tiles of K of it + 1, V of it
    // WHOLE: every row of the tiles it asks for is a key's, and the next step's scores
    // need no mask.  Then the loads are dealt out behind the QK products (a
    // wave that issues them at once waits for the address unit, which takes
    // them one by one) and the next maximum behind the PV products.
    auto step = [&](int it, f32x16(&sc)[NK], f32x16(&nx)[NK], auto whole) {
      constexpr bool WHOLE = decltype(whole)::value;
      const int key0 = key_lo + it * BN;
      const int vb_free = vb_now == 0 ? BUFS - 1 : vb_now - 1;
      const int kb_free = kb_next == 0 ? BUFS - 1 : kb_next - 1;
      if constexpr (!WHOLE) {
        if (it + BUFS < steps) fetch(0, kb_free, key0 + BUFS * BN);
        if (it + BUFS - 1 < steps) fetch(1, vb_free, key0 + (BUFS - 1) * BN);
      }
      // One stream of matrix instructions in an order fixed by hand: the QK
      // products of the next step, the weights of this one dealt out
      // behind them, then the PV products.
      int ka = kb_next * TB + k_lane(), va = V0 + vb_now * TB + v_lane();
      asm volatile("" : "+v"(ka), "+v"(va));
      auto read = [&](int i) { return i < QK ? read_k(ka, i) : read_v(va, i - QK); };
      // the elements behind product i
      auto from = [](int i) { return (i < 0 ? 0 : i) * NE / QK; };
#pragma unroll
      for (int t = 0; t < NK; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) nx[t][i] = 0.f;
      bf16x8 f[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) f[i] = read(i);
#pragma unroll
      for (int i = 0; i < QK; ++i) {
        nx[i % NK] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i % AHEAD], qf[i / NK], nx[i % NK], 0, 0, 0);
        f[i % AHEAD] = read(i + AHEAD);
        // three products' elements at once, so that no part waits for the one before it
#pragma unroll
        for (int e = from(i - 2); e < from(i - 1); ++e) weight_sum(sc, e);
#pragma unroll
        for (int e = from(i - 1); e < from(i); ++e) weight_exp(sc, e);
#pragma unroll
        for (int e = from(i); e < from(i + 1); ++e) weight_arg(sc, e);
        if constexpr (WHOLE) {
#pragma unroll
          for (int j = i * 2 * LD / QK; j < (i + 1) * 2 * LD / QK; ++j) {
            if (j < LD) fetch_one(0, kb_free, key0 + BUFS * BN, j);
            else fetch_one(1, vb_free, key0 + (BUFS - 1) * BN, j - LD);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int e = from(QK - 1); e < NE; ++e) weight_exp(sc, e);
      float mx[4];
#pragma unroll
      for (int i = 0; i < PV; ++i) {
        o[i % ND] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            f[(QK + i) % AHEAD], __builtin_bit_cast(bf16x8, pw[i / ND]), o[i % ND], 0, 0, 0);
        if (i + AHEAD < PV) f[(QK + i) % AHEAD] = read(QK + i + AHEAD);
        if (i < 2) {                         // the last two products' weights
#pragma unroll
          for (int e = from(QK - 2 + i); e < from(QK - 1 + i); ++e) weight_sum(sc, e);
        }
        if constexpr (WHOLE) {
#pragma unroll
          for (int e = i * NE / PV; e < (i + 1) * NE / PV; ++e)
            mx[e % 4] = e < 4 ? nx[e / 16][e % 16] : fmaxf(mx[e % 4], nx[e / 16][e % 16]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (WHOLE) {
        raise(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
      } else {
        if (!WHOLE && !inner(key0 + BN)) mask(key0 + BN, nx);
        raise(largest(nx));
      }
      kb_next = kb_next + 1 == BUFS ? 0 : kb_next + 1;
      vb_now = vb_now + 1 == BUFS ? 0 : vb_now + 1;
      // what this step has asked for may stay on its way
      if constexpr (WHOLE) step_barrier<(BUFS - 2) * 2 * LD>(); else step_barrier<0>();
    };
    auto whole = [&](int it) {
      return it + BUFS < steps && key_lo + (it + BUFS + 1) * BN <= s.kn && inner(key_lo + (it + 1) * BN);
    };
    int it = 0;
    while (it + 1 < steps) {
      for (; whole(it) && whole(it + 1); it += 2) {   // two at a time: scores change places
        step(it, sc, nx, std::true_type{});
        step(it + 1, nx, sc, std::true_type{});
      }
      if (it + 1 < steps) {
        step(it, sc, nx, std::false_type{});
#pragma unroll
        for (int t = 0; t < NK; ++t) sc[t] = nx[t];
        ++it;
      }
    }
    if (steps > 0) {
#pragma unroll
      for (int e = 0; e < NE; ++e) weight(sc, e);
      values(vb_now);
    }
  } else if constexpr (SPLIT == 2) {
    // Half of a step is matrix products (its scores, and with V of the step
    // before), half vector instructions (the other wave's part of the scores,
    // the weights).  The second four waves, which share the SIMDs of the first, are half
    // a step late, so that products run beside weights: 335 us instead of 350 at
    // 2048 tokens of 64 heads on one.  Tiles of K take turns in kb, kb_next
    // .., the tile of V is vb; with ONE that is K's of the step before.
    f32x16 sc[NK];
    int kb = 0, vb = 0;   // tiles of K and V that are read
    if (steps > 0) fetch(0, 0, key_lo);
    q_arrived();
    step_barrier<0>();
    auto products = [&](auto first) __attribute__((always_inline)) {
      constexpr bool LAG = !decltype(first)::value;
      int ka = kb * TB + k_lane(), va = V0 + vb * TB + v_lane();
      asm volatile("" : "+v"(ka), "+v"(va));
      auto read = [&](int i) { return i < QK ? read_k(ka, i) : read_v(va, i - QK); };
      constexpr int N = LAG ? QK + PV : QK;
#pragma unroll
      for (int t = 0; t < NK; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) sc[t][i] = 0.f;
      bf16x8 f[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) f[i] = read(i);
#pragma unroll
      for (int i = 0; i < QK; ++i) {
        sc[i % NK] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i % AHEAD], qf[i / NK], sc[i % NK], 0, 0, 0);
        if (i + AHEAD < N) f[i % AHEAD] = read(i + AHEAD);
        __builtin_amdgcn_sched_barrier(0);
      }
      hand_over(sc);
#pragma unroll
      for (int i = QK; i < N; ++i) {
        o[(i - QK) % ND] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            f[i % AHEAD], __builtin_bit_cast(bf16x8, pw[(i - QK) / ND]), o[(i - QK) % ND], 0, 0, 0);
        if (i + AHEAD < N) f[i % AHEAD] = read(i + AHEAD);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto weights = [&](int key0) __attribute__((always_inline)) {
      take_over(sc);
      if (!inner(key0)) mask(key0, sc);
      raise(largest(sc));
#pragma unroll
      for (int e = 0; e < NE; ++e) weight(sc, e);
    };
    // one step of early or late waves: both pass the same two barriers
    auto step = [&](int it, auto first, auto late) __attribute__((always_inline)) {
      constexpr bool LATE = decltype(late)::value;
      const int key0 = key_lo + it * BN;
      const int kb_next = kb + 1 == (ONE ? 3 : 2) ? 0 : kb + 1;
      const int vb_next = ONE ? kb : vb ^ 1;
      if (it + 1 < steps) fetch(0, kb_next, key0 + BN);
      if constexpr (!ONE) fetch(1, vb_next, key0);
      if constexpr (!LATE) products(first);
      else if constexpr (!decltype(first)::value) weights(key0 - BN);
      lds_barrier();
      if constexpr (LATE) products(first); else weights(key0);
      kb = kb_next;
      vb = vb_next;
      step_barrier<0>();
    };
    auto walk = [&](auto late) __attribute__((always_inline)) {
      step(0, std::true_type{}, late);
      for (int it = 1; it < steps; ++it) step(it, std::false_type{}, late);
    };
    if (steps > 0) {
      if (wv < 4) {
        walk(std::false_type{});
      } else {
        walk(std::true_type{});
        weights(key_lo + (steps - 1) * BN);
      }
      values(vb);
    }
  } else {
    if (steps > 0) {
      fetch(0, 0, key_lo);
      fetch(1, 0, key_lo);
    }
    q_arrived();
    step_barrier<0>();
    for (int it = 0; it < steps; ++it) {
      const int key0 = key_lo + it * BN;
      const int buf = it & 1;
      if (it + 1 < steps) {
        fetch(0, buf ^ 1, key0 + BN);
        fetch(1, buf ^ 1, key0 + BN);
      }
      f32x16 sc[NK];
      scores(buf, sc);
      if (!inner(key0)) mask(key0, sc);
      raise(largest(sc));
#pragma unroll
      for (int e = 0; e < NE; ++e) weight(sc, e);
      values(buf);
      step_barrier<0>();
    }
  }

  l += l2;
  l += __shfl_xor(l, 32);
  // the row again, so that the loop need not hold it
  const int ln = here();
  const int64_t row = row0 + wave * 32 + (ln & 31);
  if (row >= rows) return;
  const int tok = (int)(row / p.group);
  const int head = h * p.group + (int)(row - (int64_t)tok * p.group);
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  uint16_t* dst = p.out + (s.q0 + tok) * p.o_st + head * p.o_sh;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
      // 4 columns of two eighths each: the row's other lane takes the second
      // eighth's for the first one's, so that each stores one of 16 bytes
      const u32x2 x = __builtin_amdgcn_permlane32_swap(pack_bf16(o[d][i] * inv, o[d][i + 1] * inv),
                                                       pack_bf16(o[d][i + 4] * inv, o[d][i + 5] * inv),
                                                       false, false);
      const u32x2 y = __builtin_amdgcn_permlane32_swap(pack_bf16(o[d][i + 2] * inv, o[d][i + 3] * inv),
                                                       pack_bf16(o[d][i + 6] * inv, o[d][i + 7] * inv),
                                                       false, false);
      *reinterpret_cast<u32x4*>(dst + 32 * (part * ND + d) + 2 * i + 8 * (ln >> 5)) =
          u32x4{x[0], y[0], x[1], y[1]};
    }
  if (p.lse && ln < 32 && part == 0)
    p.lse[(int64_t)(s.q0 + tok) * p.hq + head] =
        l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
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
#define MOE_PREFILL(D, BN, RG, SPLIT, BUFS, PIPE, AHEAD, WAVES, ONE)                          \
  {                                                                                           \
    /* at most one partly filled tile per sequence */                                         \
    const int64_t tiles = c.tokens * a.group / (32 * RG) + std::min<int64_t>(c.batch, c.tokens); \
    return launch_workgroups(tiles * c.heads_kv, [&](uint32_t first, dim3 grid) {             \
      a.first = first;                                                                        \
      hipLaunchKernelGGL((attn_prefill_kernel<D, BN, RG, SPLIT, BUFS, PIPE, AHEAD, WAVES, ONE>), grid, \
                         dim3(64 * RG * SPLIT), 0, st, a);                                    \
    });                                                                                       \
  }
  // Weights beside the next step's products, or not (PIPE), in us: 64-element heads,
  // 8192 tokens 343 and 315 (without it four workgroups share a CU); 128, 8192 tokens
  // 542 and 560; 256, 4096 tokens 168 and 215.  One tensor as keys and values,
  // loaded once: 331 instead of 356 for 2048 tokens of 64 heads of 512.
  switch (c.head_dim) {
    case 64: MOE_PREFILL(64, 64, 4, 1, 2, false, 4, 2, false)
    case 128: MOE_PREFILL(128, 64, 4, 1, 2, true, 3, 2, false)
    case 256: MOE_PREFILL(256, 32, 4, 1, 3, true, 2, 2, false)
    case 512:
      if (v.p == k.p && v.stride_token == k.stride_token && v.stride_head == k.stride_head)
        MOE_PREFILL(512, 32, 4, 2, 3, false, 2, 2, true)
      else
        MOE_PREFILL(512, 32, 4, 2, 2, false, 2, 2, false)
    default: return hipErrorInvalidValue;
  }
#undef MOE_PREFILL
}

}  // namespace moe
