// Attention of new tokens over the paged key-value cache (include/moe_attn.h,
// moe_attn_decode).
//
// Mathematics: every wave walks its keys once with the running maximum m and
// sum l of a softmax in base 2 (s2 = scale log2(e) q.k):
//   m' = max(m, s2), p = 2^(s2 - m'), a = 2^(m - m'), l = a l + sum p,
//   o = a o + p v;
// pieces (m_i, l_i, o_i) join as m = max m_i, l = sum 2^(m_i - m) l_i,
// o = sum 2^(m_i - m) o_i / l, first the waves of a workgroup through LDS,
// then the splits of a sequence in a second kernel.
//
// Matrix form: the rows of one key-value head (q_len * group of them, 16 to a
// tile) are the columns of both products, S^T = K Q^T and O^T = V^T P^T on
// 16x16x32 bf16 MFMA, so that m, l and the rescaling are per lane (lane % 16
// is the row), and the P that comes out of the first product is, register
// for register, the operand of the second: with lane group g = lane / 16 the first leaves keys
// 4 g .. 4 g + 3 of two 16-key tiles in a lane, and the second contracts over
// any order of keys that both of its operands share.  K and V go from memory
// to registers without LDS: K's operand is 16 bytes of one key per lane; V's
// needs 8 keys of one column per lane, which a lane gets by loading the same 8
// columns of its 8 keys (a wave then covers whole rows) and transposing 8 x 8
// in registers.
#include <algorithm>

#include "attn_internal.h"

namespace moe {

namespace {

constexpr int kTileKeys = 128;     // unit of the split over a sequence's keys
constexpr int kSplitTarget = 1024; // workgroups the tiles are dealt to

struct DecodeArgs {
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int64_t q_st, q_sh, o_st, o_sh;
  const char* k;
  const char* v;
  const uint8_t* ks;
  const uint8_t* vs;
  int64_t sp, sh, st;      // bytes
  int64_t pages;
  const int32_t* table;
  const int32_t* seq_lens;
  int table_width, page_shift;
  int batch, q_len, hq, hkv, group, rows, rgroups;
  int window;
  float scale2;            // scale * log2(e)
  int target;              // splits over all sequences, for one head and row group
  int slots;               // grid bound: target + batch
  float* part_o;           // [slots][hkv][rows][D]
  float* part_m;           // [slots][hkv][rows] maximum (base 2)
  float* part_l;           // ... and sum
  int2* meta;              // [batch] first slot, splits
};

// Keys a sequence's rows may reach: [lo, len), and how many 128-key tiles
// that is, counted from lo rounded down to a step of 32.
struct Range {
  int lo, len, tiles;
};
__device__ __forceinline__ Range range_of(const DecodeArgs& p, int raw_len) {
  Range r;
  const int64_t cap = (int64_t)p.table_width << p.page_shift;
  r.len = (int)min((int64_t)max(raw_len, 0), cap);
  if (p.pages == 0) r.len = 0;
  r.lo = 0;
  if (p.window > 0) {
    const int64_t lo = (int64_t)r.len - p.q_len + 1 - p.window;   // first row's window start
    r.lo = (int)max(lo, (int64_t)0);
  }
  const int span = r.len - (r.lo & ~31);
  r.tiles = r.len > r.lo ? (span + kTileKeys - 1) / kTileKeys : 0;
  return r;
}

// Which sequence and split a slot is: tiles are dealt c to a split, c the
// ceiling of all tiles over `target`; a sequence has at least one split, so
// that an empty one still has its rows written.  Every wave works it out for
// itself, 64 sequences at a time.
struct Piece {
  int b, split, splits, slot0, c;
};
__device__ __forceinline__ int wave_sum(int x) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) x += __shfl_xor(x, off);
  return x;
}
__device__ __forceinline__ bool find_piece(const DecodeArgs& p, int slot, Piece& out) {
  const int lane = threadIdx.x & 63;
  int64_t total = 0;
  int mine = 0;   // tiles of the last 64 sequences looked at
  for (int b0 = 0; b0 < p.batch; b0 += 64) {
    mine = b0 + lane < p.batch ? range_of(p, p.seq_lens[b0 + lane]).tiles : 0;
    total += wave_sum(mine);
  }
  const int c = (int)max((total + p.target - 1) / p.target, (int64_t)1);
  int base = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 64) {
    if (p.batch > 64)
      mine = b0 + lane < p.batch ? range_of(p, p.seq_lens[b0 + lane]).tiles : 0;
    const int n = b0 + lane < p.batch ? max((mine + c - 1) / c, 1) : 0;
    int incl = n;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(incl, off);
      if (lane >= off) incl += o;
    }
    const uint64_t past = __ballot(base + incl > slot);
    if (past) {
      const int l = __builtin_ctzll(past);
      out.b = __builtin_amdgcn_readfirstlane(b0 + l);
      out.splits = __builtin_amdgcn_readlane(n, l);
      out.slot0 = base + __builtin_amdgcn_readlane(incl, l) - out.splits;
      out.split = slot - out.slot0;
      out.c = __builtin_amdgcn_readfirstlane(c);
      return true;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

__device__ __forceinline__ float scale_of(uint32_t byte) {   // 2^(byte - 127)
  return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}

// 4 E4M3 bytes times 2^.. -> 4 bf16 (exact: an E4M3 value times a power of two)
__device__ __forceinline__ u32x2 fp8x4_to_bf16(uint32_t w, float s) {
  u32x2 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true));
  return r;
}

// D: head size; RT: 16-row tiles of a workgroup, one per wave (1, 2 or 4);
// the 4 / RT waves of one tile take every (4 / RT)th step of 32 keys.
template <int D, bool FP8, int RT>
__global__ __launch_bounds__(256) void attn_decode_kernel(DecodeArgs p) {
  constexpr int KP = 4 / RT;
  constexpr int NF = D / 32;                  // K fragments per 16-key tile
  constexpr int DV = D < 128 ? D / 16 : 8;    // columns of V per lane and block
  constexpr int NB = D / (16 * DV);           // blocks of 16 * DV columns
  constexpr int NG = D < 128 ? 1 : D / 128;   // FP8 scales per row
  constexpr int EB = FP8 ? 1 : 2;             // bytes per element
  constexpr int VW = DV * EB / 4;             // dwords of V per lane, row and block
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int rt = wave % RT, kp = wave / RT;

  const int per_slot = p.hkv * p.rgroups;
  const int slot = blockIdx.x / per_slot;
  const int rest = blockIdx.x - slot * per_slot;
  const int rg = rest / p.hkv, h = rest - rg * p.hkv;
  Piece pc;
  if (!find_piece(p, slot, pc)) return;
  const Range rng = range_of(p, __builtin_amdgcn_readfirstlane(p.seq_lens[pc.b]));
  const int len = rng.len, lo = rng.lo;
  const int first = (lo & ~31) + pc.split * pc.c * kTileKeys;
  const int last = (int)min((int64_t)len, (int64_t)first + (int64_t)pc.c * kTileKeys);

  // this lane's row: token, head and the keys it keeps [row_lo, row_hi)
  const int row = (rg * RT + rt) * 16 + col;
  const bool row_live = row < p.rows;
  const int tok = row_live ? row / p.group : 0;
  const int head = row_live ? h * p.group + row - tok * p.group : 0;
  const int64_t qrow = (int64_t)pc.b * p.q_len + tok;
  const int row_hi = len - p.q_len + 1 + tok;
  const int row_lo = p.window > 0 ? row_hi - p.window : 0;
  // every row keeps the keys of [all_lo, all_hi)
  const int all_hi = len - p.q_len + 1;
  const int all_lo = p.window > 0 ? len - p.window : 0;

  bf16x8 qf[NF];
#pragma unroll
  for (int j = 0; j < NF; ++j) {
    // the columns of fragment j that this lane group holds; for FP8, fragments
    // 2 i and 2 i + 1 share one 16-byte load of K
    const int d = FP8 ? 64 * (j >> 1) + 16 * g + 8 * (j & 1) : 32 * j + 8 * g;
    u32x4 w = {0, 0, 0, 0};
    if (row_live) w = *reinterpret_cast<const u32x4*>(p.q + qrow * p.q_st + head * p.q_sh + d);
    qf[j] = __builtin_bit_cast(bf16x8, w);
  }
  f32x4 o[NB][DV];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < DV; ++i) o[b][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = kNoMax, l = 0.f;

  const int32_t* trow = p.table + (int64_t)pc.b * p.table_width;
  const char* kh = p.k + h * p.sh;
  const char* vh = p.v + h * p.sh;
  const int page_mask = (1 << p.page_shift) - 1;

  for (int key0 = first + 32 * kp; key0 < last; key0 += 32 * KP) {
    bool have[2];
    int64_t off[2], srow[2];   // byte offset of the tile's first row; its index among scale rows
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int kt = key0 + 16 * t;
      have[t] = kt < len && kt + 16 > lo;
      int pid = have[t] ? trow[kt >> p.page_shift] : 0;
      have[t] = have[t] && pid >= 0 && pid < p.pages;
      pid = have[t] ? pid : 0;
      off[t] = pid * p.sp + (int64_t)(kt & page_mask) * p.st;
      srow[t] = (((int64_t)pid * p.hkv + h) << p.page_shift) + (kt & page_mask);
    }
    const bool inner = have[0] && have[1] && key0 >= all_lo && key0 + 32 <= all_hi;

    // K, 16 keys a tile, and V
    f32x4 s[2];
    u32x4 kr[2][FP8 ? NF / 2 : NF];
    uint32_t ksc[2][NG];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const char* kb = kh + off[t] + col * p.st;
#pragma unroll
      for (int j = 0; j < (FP8 ? NF / 2 : NF); ++j)
        kr[t][j] = *reinterpret_cast<const u32x4*>(kb + 64 * j + 16 * g);
      if constexpr (FP8) {
#pragma unroll
        for (int n = 0; n < NG; ++n) ksc[t][n] = p.ks[(srow[t] + col) * NG + n];
      }
    }
    uint32_t vr[8][NB][VW];
    uint32_t vsc[2][NG];      // the 4 rows' scale bytes of tile t, row-major [4][NG]
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const char* vb = vh + off[t] + (4 * g + r) * p.st + col * (DV * EB);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if constexpr (VW == 4) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(vb + b * 16 * DV * EB);
#pragma unroll
            for (int i = 0; i < 4; ++i) vr[4 * t + r][b][i] = w[i];
          } else if constexpr (VW == 2) {
            const u32x2 w = *reinterpret_cast<const u32x2*>(vb + b * 16 * DV * EB);
            vr[4 * t + r][b][0] = w[0];
            vr[4 * t + r][b][1] = w[1];
          } else {
            vr[4 * t + r][b][0] = *reinterpret_cast<const uint32_t*>(vb + b * 16 * DV * EB);
          }
        }
      }
      if constexpr (FP8) {
        const uint32_t* sb = reinterpret_cast<const uint32_t*>(p.vs + (srow[t] + 4 * g) * NG);
#pragma unroll
        for (int n = 0; n < NG; ++n) vsc[t][n] = sb[n];
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      s[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        bf16x8 kf;
        if constexpr (FP8) {
          const float sc = scale_of(ksc[t][(64 * (j >> 1)) / 128]);
          const u32x2 a = fp8x4_to_bf16(kr[t][j >> 1][2 * (j & 1)], sc);
          const u32x2 b = fp8x4_to_bf16(kr[t][j >> 1][2 * (j & 1) + 1], sc);
          kf = __builtin_bit_cast(bf16x8, u32x4{a[0], a[1], b[0], b[1]});
        } else {
          kf = __builtin_bit_cast(bf16x8, kr[t][j]);
        }
        s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[j], s[t], 0, 0, 0);
      }
    }

    float pr[8];
    float mx = kNoMax;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) pr[4 * t + i] = s[t][i] * p.scale2;
    if (!inner) {
      // masked scores, and rows of V that no score keeps are not used whatever
      // they hold (0 * NaN)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = key0 + 16 * t + 4 * g + i;
          if (!(have[t] && key < row_hi && key >= row_lo)) pr[4 * t + i] = -INFINITY;
          const bool used = have[t] && key < len && key >= lo;
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int w = 0; w < VW; ++w) vr[4 * t + i][b][w] = used ? vr[4 * t + i][b][w] : 0u;
          if constexpr (FP8) {
#pragma unroll
            for (int n = 0; n < NG; ++n) {
              const int at = i * NG + n;   // byte of vsc[t]
              const uint32_t one = 127u << (8 * (at & 3)), all = 0xFFu << (8 * (at & 3));
              vsc[t][at >> 2] = used ? vsc[t][at >> 2] : (vsc[t][at >> 2] & ~all) | one;
            }
          }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = fmaxf(mx, pr[i]);
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    if (__ballot(mx > m)) {
      const float mn = fmaxf(m, mx);
      const float a = exp2_fast(m - mn);
      m = mn;
      l *= a;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < DV; ++i) o[b][i] *= a;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) pr[i] = exp2_fast(pr[i] - m);
    l += ((pr[0] + pr[1]) + (pr[2] + pr[3])) + ((pr[4] + pr[5]) + (pr[6] + pr[7]));
    const u32x4 pw = {pack_bf16(pr[0], pr[1]), pack_bf16(pr[2], pr[3]), pack_bf16(pr[4], pr[5]),
                      pack_bf16(pr[6], pr[7])};
    const bf16x8 pf = __builtin_bit_cast(bf16x8, pw);

#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint32_t x[8][DV / 2];     // 8 keys x DV columns of bf16
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if constexpr (FP8) {
          const int at = (r & 3) * NG + (NG == 1 ? 0 : b);
          const float sc = scale_of((vsc[r >> 2][at >> 2] >> (8 * (at & 3))) & 0xFFu);
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            const u32x2 y = fp8x4_to_bf16(vr[r][b][w], sc);
            x[r][2 * w] = y[0];
            x[r][2 * w + 1] = y[1];
          }
        } else {
#pragma unroll
          for (int w = 0; w < VW; ++w) x[r][w] = vr[r][b][w];
        }
      }
#pragma unroll
      for (int i = 0; i < DV; ++i) {
        u32x4 f;
        const uint32_t sel = (i & 1) ? 0x07060302u : 0x05040100u;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          f[j] = __builtin_amdgcn_perm(x[2 * j + 1][i >> 1], x[2 * j][i >> 1], sel);
        o[b][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f), pf,
                                                          o[b][i], 0, 0, 0);
      }
    }
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);

  // join the waves of one row tile: half of them hand theirs to the others
  if constexpr (KP > 1) {
    constexpr int SZ = NB * DV * 4 * 64;        // floats of o per wave
    __shared__ float lds[RT * (KP / 2) * (SZ + 128)];
#pragma unroll
    for (int half = KP / 2; half >= 1; half >>= 1) {
      if (kp >= half && kp < 2 * half) {
        float* to = lds + (rt * (KP / 2) + kp - half) * (SZ + 128);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < DV; ++i)
            *reinterpret_cast<f32x4*>(to + ((b * DV + i) * 64 + lane) * 4) = o[b][i];
        to[SZ + lane] = m;
        to[SZ + 64 + lane] = l;
      }
      __syncthreads();
      if (kp < half) {
        const float* from = lds + (rt * (KP / 2) + kp) * (SZ + 128);
        const float m2 = from[SZ + lane], l2 = from[SZ + 64 + lane];
        const float mn = fmaxf(m, m2);
        const float a = exp2_fast(m - mn), c = exp2_fast(m2 - mn);
        m = mn;
        l = l * a + l2 * c;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < DV; ++i) {
            const f32x4 y = *reinterpret_cast<const f32x4*>(from + ((b * DV + i) * 64 + lane) * 4);
            o[b][i] = o[b][i] * a + y * c;
          }
      }
      __syncthreads();
    }
    if (kp > 0) return;
  }

  if (pc.split == 0 && h == 0 && rg == 0 && threadIdx.x == 0)
    p.meta[pc.b] = make_int2(pc.slot0, pc.splits);
  if (!row_live) return;
  if (pc.splits == 1) {
    const float inv = l > 0.f ? 1.0f / l : 0.f;
    uint16_t* dst = p.out + qrow * p.o_st + head * p.o_sh;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        uint32_t w[DV / 2];
#pragma unroll
        for (int i = 0; i < DV / 2; ++i)
          w[i] = pack_bf16(o[b][2 * i][r] * inv, o[b][2 * i + 1][r] * inv);
        uint16_t* to = dst + b * 16 * DV + (4 * g + r) * DV;
        if constexpr (DV == 8)
          *reinterpret_cast<u32x4*>(to) = u32x4{w[0], w[1], w[2], w[3]};
        else
          *reinterpret_cast<u32x2*>(to) = u32x2{w[0], w[1]};
      }
    if (p.lse && g == 0)
      p.lse[qrow * p.hq + head] = l > 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
  } else {
    const int64_t at = ((int64_t)slot * p.hkv + h) * p.rows + row;
    float* dst = p.part_o + at * D;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < DV; i += 4)
          *reinterpret_cast<f32x4*>(dst + b * 16 * DV + (4 * g + r) * DV + i) =
              f32x4{o[b][i][r], o[b][i + 1][r], o[b][i + 2][r], o[b][i + 3][r]};
    if (g == 0) {
      p.part_m[at] = m;
      p.part_l[at] = l;
    }
  }
}

// Joins the splits of a sequence: one wave per (sequence, head, row); rows of a
// sequence with one split are written already.
template <int D>
__global__ __launch_bounds__(256) void attn_decode_join_kernel(DecodeArgs p) {
  constexpr int EPL = D / 64;     // elements per lane
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t per_b = (int64_t)p.hkv * p.rows;
  const int64_t b = w / per_b;
  if (b >= p.batch) return;
  const int rest = (int)(w - b * per_b);
  const int h = rest / p.rows, row = rest - h * p.rows;
  const int2 mt = p.meta[b];
  if (mt.y <= 1) return;
  const int64_t stride = (int64_t)p.hkv * p.rows;
  const int64_t at0 = (int64_t)mt.x * stride + (int64_t)h * p.rows + row;
  float m = kNoMax;
  for (int i = lane; i < mt.y; i += 64) m = fmaxf(m, p.part_m[at0 + i * stride]);
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) m = fmaxf(m, __shfl_xor(m, off));
  float l = 0.f, o[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) o[e] = 0.f;
  for (int i = 0; i < mt.y; ++i) {
    const int64_t at = at0 + i * stride;
    const float a = exp2_fast(p.part_m[at] - m);
    l = fmaf(a, p.part_l[at], l);
#pragma unroll
    for (int e = 0; e < EPL; ++e) o[e] = fmaf(a, p.part_o[at * D + lane * EPL + e], o[e]);
  }
  const float inv = l > 0.f ? 1.0f / l : 0.f;
  const int tok = row / p.group;
  const int head = h * p.group + row - tok * p.group;
  const int64_t qrow = b * p.q_len + tok;
  uint16_t* dst = p.out + qrow * p.o_st + head * p.o_sh + lane * EPL;
  if constexpr (EPL == 1) {
    *dst = (uint16_t)(pack_bf16(o[0] * inv, 0.f) & 0xFFFFu);
  } else {
#pragma unroll
    for (int e = 0; e < EPL; e += 2)
      *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16(o[e] * inv, o[e + 1] * inv);
  }
  if (p.lse && lane == 0) p.lse[qrow * p.hq + head] = l > 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
}

int row_tiles(int rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

struct DecodePlan {
  int rows, rgroups, target, slots;
};
DecodePlan plan_of(const moe_attn_config& c) {
  DecodePlan d;
  d.rows = c.q_len * (c.heads_q / c.heads_kv);
  const int rt = row_tiles(d.rows);
  d.rgroups = (d.rows + 16 * rt - 1) / (16 * rt);
  d.target = std::max(1, kSplitTarget / (c.heads_kv * d.rgroups));
  d.slots = d.target + c.batch;
  return d;
}
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

size_t attn_decode_ws_bytes(const moe_attn_config& c) {
  const DecodePlan d = plan_of(c);
  const size_t rows = (size_t)d.slots * c.heads_kv * d.rows;
  return up256(rows * c.head_dim * 4) + 2 * up256(rows * 4) + up256((size_t)c.batch * 8);
}

hipError_t launch_attn_decode(const moe_attn_config& c, const moe_rows& q, const moe_kv_cache& kv,
                              const int32_t* table, int table_width, const int32_t* seq_lens,
                              const moe_rows& out, float* lse, void* ws, hipStream_t st) {
  if (c.batch == 0) return hipSuccess;
  const DecodePlan d = plan_of(c);
  DecodeArgs a{};
  a.q = q.p; a.q_st = q.stride_token; a.q_sh = q.stride_head;
  a.out = out.p; a.o_st = out.stride_token; a.o_sh = out.stride_head;
  a.lse = lse;
  const int eb = kv.format == MOE_KV_FP8 ? 1 : 2;
  a.k = static_cast<const char*>(kv.k); a.v = static_cast<const char*>(kv.v);
  a.ks = kv.k_scale; a.vs = kv.v_scale;
  a.sp = kv.stride_page * eb; a.sh = kv.stride_head * eb; a.st = kv.stride_token * eb;
  a.pages = kv.pages;
  a.table = table; a.table_width = table_width; a.seq_lens = seq_lens;
  a.page_shift = __builtin_ctz((unsigned)kv.page_size);
  a.batch = c.batch; a.q_len = c.q_len; a.hq = c.heads_q; a.hkv = c.heads_kv;
  a.group = c.heads_q / c.heads_kv;
  a.rows = d.rows; a.rgroups = d.rgroups; a.target = d.target; a.slots = d.slots;
  a.window = c.window; a.scale2 = c.scale * kLog2e;
  const size_t rows = (size_t)d.slots * c.heads_kv * d.rows;
  char* w = static_cast<char*>(ws);
  a.part_o = reinterpret_cast<float*>(w); w += up256(rows * c.head_dim * 4);
  a.part_m = reinterpret_cast<float*>(w); w += up256(rows * 4);
  a.part_l = reinterpret_cast<float*>(w); w += up256(rows * 4);
  a.meta = reinterpret_cast<int2*>(w);
  const dim3 grid((unsigned)d.slots * c.heads_kv * d.rgroups);
  const int rt = row_tiles(d.rows);
  const bool f8 = kv.format == MOE_KV_FP8;
#define MOE_DECODE_RT(D, F, R) \
  hipLaunchKernelGGL((attn_decode_kernel<D, F, R>), grid, dim3(256), 0, st, a)
#define MOE_DECODE(D)                                                                         \
  case D:                                                                                     \
    if (f8) {                                                                                 \
      if (rt == 1) MOE_DECODE_RT(D, true, 1);                                                 \
      else if (rt == 2) MOE_DECODE_RT(D, true, 2);                                            \
      else MOE_DECODE_RT(D, true, 4);                                                         \
    } else {                                                                                  \
      if (rt == 1) MOE_DECODE_RT(D, false, 1);                                                \
      else if (rt == 2) MOE_DECODE_RT(D, false, 2);                                           \
      else MOE_DECODE_RT(D, false, 4);                                                        \
    }                                                                                         \
    break;
  switch (c.head_dim) {
    MOE_DECODE(64) MOE_DECODE(128) MOE_DECODE(256) MOE_DECODE(512)
    default: return hipErrorInvalidValue;
  }
#undef MOE_DECODE
#undef MOE_DECODE_RT
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t waves = (int64_t)c.batch * c.heads_kv * d.rows;
  const dim3 jgrid((unsigned)((waves + 3) / 4));
#define MOE_JOIN(D) \
  case D: hipLaunchKernelGGL((attn_decode_join_kernel<D>), jgrid, dim3(256), 0, st, a); break;
  switch (c.head_dim) { MOE_JOIN(64) MOE_JOIN(128) MOE_JOIN(256) MOE_JOIN(512) }
#undef MOE_JOIN
  return hipGetLastError();
}

}  // namespace moe
