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
// in registers.  P is rounded to bf16 as v is: kept as the sum of two bf16
// values (16 bits) the output is nearer to the exact one by less than its own
// rounding (1.7e-3 instead of 2.3e-3 in the 2-norm), for 1 to 13% of the time.
//
// Bound by the reads of K and V, each row once.  Measured: 64 sequences of up to
// 4096 keys, 8 heads of 128 in bf16 106 us (6.1 TB/s; the join kernel takes 4.5 of
// them); one sequence of 131071 keys in FP8 49 us (5.5 TB/s); 32 sequences of up to 4096
// keys, 64 query heads on one 512-element head that is keys and values 47 us
// (2.2 TB/s: 35 and a join of 7.6, with 31 MB of partial results between
// them); 300 keys of 8 heads 7.8 us, a chain of latencies.
#include <algorithm>

#include "attn_internal.h"

namespace moe {

namespace {

// Pieces the work is cut into, over all heads and row groups: two workgroups a CU for the kernel without LDS
// (of 256, 512, 768 and 1024 pieces the best or within 1% of it for 64 ragged
// sequences, one long one and 256-element heads; 1024 take 3% and 10% more on the first two).  The one with LDS cuts
// each sequence by itself, which adds up to a piece per sequence, head and row
// group.  With one head and row group the pieces make room for those (of up to 128 sequences), so that all
// stay below the CUs of a kernel with one workgroup on each (69 instead
// of 48 us at 32 sequences on one 512-element head without).  With several heads or row groups
// they do not: room for a piece of each makes pieces longer and was slower, though the
// workgroups pass 256 without it.  Four new tokens on one 512-element head, 32 ragged sequences 127 us
// and 132 with the room; two heads of 512 99 and 105; four new tokens on 4 heads of 128 61 and 78; 256 elements 47 and
// 49; eight heads of 512 alone gained, 195 and 182.
constexpr int kPieces = 512;
int pieces_rows(int batch) { return std::max(256 - batch, 128); }

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
  int pieces;              // the work's, for one head and row group; 0: one per sequence
  uint32_t first;          // the launch's first workgroup
  int tile_shift;          // keys per tile, the unit of the cut: 2^tile_shift
  float* part_o;           // [pieces + batch][hkv][rows][D]
  float* part_m;           // [pieces + batch][hkv][rows] maximum (base 2)
  float* part_l;           // ... and sum
  int2* meta;              // [batch] first slot, splits
};

// An entry of a table that no kernel writes, at a wave-uniform index: a scalar load.
__device__ __forceinline__ int entry(const int32_t* t, int64_t i) {
  return *(const __attribute__((address_space(4))) int32_t*)(t + i);
}

// Keys a sequence's rows may reach: [lo, len), and how many tiles that is, counted from lo rounded down to a step of 32 (1 for none).
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
  r.tiles = r.len > r.lo ? (span + (1 << p.tile_shift) - 1) >> p.tile_shift : 1;
  return r;
}

// The work of all sequences, laid end to end in tiles, is cut into pieces, one
// per workgroup (of a head and row group).  An empty sequence counts a tile,
// so that a piece writes its rows.
// ACROSS: pieces of equal length; one covers the end of a sequence, whole ones and
// the start of another.  Sequence b's part of piece w is a split with slot w +
// b: every step along the work raises one of the two, so slots differ, and
// those of a sequence are consecutive.
// Otherwise each sequence is cut by itself into pieces of at most the same
// length, which are its splits and slots: more uneven, but a part of a
// sequence costs the kernel for many rows as much as 200 keys (its rows of q, its first
// tiles, its partial result).
struct Piece {
  int w;            // piece
  uint32_t per;     // tiles per piece
  uint32_t at, end; // first tile, and past the last one
  int b, tile, len; // the sequence of the first one, the tile's place there, seq_lens[b]
};
// Every wave works its piece out for itself, 64 sequences at a time.
template <bool ACROSS>
__device__ __forceinline__ bool find_piece(const DecodeArgs& p, int w, Piece& out) {
  const int lane = threadIdx.x & 63;
  if (p.pieces == 0) {                 // nothing is cut: piece w is sequence w
    out.w = 0;
    out.per = 1u << 30;
    out.b = w;
    out.tile = 0;
    out.len = entry(p.seq_lens, w);
    out.at = 0;
    out.end = range_of(p, out.len).tiles;
    return true;
  }
  uint32_t total = 0;   // the host has checked that it stays below 2^31
  int raw = 0, mine = 0, incl = 0;   // the last 64 sequences looked at
  auto look = [&](int b0) {
    raw = b0 + lane < p.batch ? p.seq_lens[b0 + lane] : 0;
    mine = b0 + lane < p.batch ? range_of(p, raw).tiles : 0;
    incl = wave_scan(mine);
  };
  for (int b0 = 0; b0 < p.batch; b0 += 64) {
    look(b0);
    total += __builtin_amdgcn_readlane(incl, 63);
  }
  out.w = w;
  out.per = __builtin_amdgcn_readfirstlane((total + p.pieces - 1) / p.pieces);
  if constexpr (!ACROSS) {
    uint32_t base = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 64) {
      if (p.batch > 64) look(b0);
      const int n = (int)((mine + out.per - 1) / out.per);   // 0 past the last sequence
      incl = wave_scan(n);
      const uint64_t past = __ballot(base + incl > (uint32_t)w);
      if (past) {
        const int l = __builtin_ctzll(past);
        out.b = __builtin_amdgcn_readfirstlane(b0 + l);
        out.len = __builtin_amdgcn_readlane(raw, l);
        out.tile = __builtin_amdgcn_readfirstlane(
            (w - (int)(base + __builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(n, l))) *
            (int)out.per);
        out.at = out.tile;
        out.end = min(out.at + out.per, (uint32_t)__builtin_amdgcn_readlane(mine, l));
        return true;
      }
      base += __builtin_amdgcn_readlane(incl, 63);
    }
    return false;
  }
  out.at = (uint32_t)min((uint64_t)w * out.per, (uint64_t)total);
  out.end = min(out.at + out.per, total);
  if (out.at >= total) return false;
  uint32_t base = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 64) {
    if (p.batch > 64) look(b0);
    const uint64_t past = __ballot(base + incl > out.at);
    if (past) {
      const int l = __builtin_ctzll(past);
      out.b = __builtin_amdgcn_readfirstlane(b0 + l);
      out.len = __builtin_amdgcn_readlane(raw, l);
      out.tile = (int)(out.at - base) -
                 (__builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(mine, l));
      return true;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// One sequence's part of a piece.
struct Part {
  int b, slot, splits;
  bool starts;      // holds the sequence's first tile
  Range rng;
  int first, last;  // keys
};
template <bool ACROSS>
__device__ __forceinline__ Part part_of(const DecodeArgs& p, const Piece& pc) {
  Part x;
  x.b = pc.b;
  x.slot = ACROSS ? pc.w + pc.b : pc.w;
  x.rng = range_of(p, pc.len);
  const uint32_t begin = pc.at - pc.tile;   // the sequence's first tile in all the work, or 0
  x.splits = __builtin_amdgcn_readfirstlane(
      (int)((begin + x.rng.tiles - 1) / pc.per - begin / pc.per) + 1);
  x.starts = pc.tile == 0;
  const int n = min((int)(pc.end - pc.at), x.rng.tiles - pc.tile);
  x.first = (x.rng.lo & ~31) + (pc.tile << p.tile_shift);
  x.last = (int)min((int64_t)x.rng.len, (int64_t)x.first + ((int64_t)n << p.tile_shift));
  return x;
}
__device__ __forceinline__ void advance(const DecodeArgs& p, const Part& x, Piece& pc) {
  pc.at += x.rng.tiles - pc.tile;          // past the end where the part is the piece's last
  pc.tile = 0;
  ++pc.b;
  if (pc.at < pc.end) pc.len = entry(p.seq_lens, pc.b);
}

// Pages of 64 consecutive 16-key tiles, one per lane (-1: no key of the tile is
// read), with the next 64 on their way: a step gets its page from a lane instead
// of waiting for a load.
struct Pages {
  const int32_t* row;
  int len, lo, base, now, next;
  __device__ __forceinline__ int load(const DecodeArgs& p, int tile) const {
    const int64_t key = 16 * ((int64_t)tile + (threadIdx.x & 63));
    if (!(key < len && key + 16 > lo)) return -1;
    const int id = row[key >> p.page_shift];
    return id >= 0 && id < p.pages ? id : -1;
  }
  __device__ __forceinline__ Pages(const DecodeArgs& p, const Part& pt)
      : row(p.table + (int64_t)pt.b * p.table_width), len(pt.rng.len), lo(pt.rng.lo),
        base(pt.first >> 4) {
    now = load(p, base);
    next = load(p, base + 64);
  }
  // the page of the tile that key begins or lies in; keys do not go back past a window
  __device__ __forceinline__ int at(const DecodeArgs& p, int key) {
    const int t = key >> 4;
    if (t >= base + 64) {
      base += 64;
      now = next;
      next = load(p, base + 64);
    }
    return __builtin_amdgcn_readlane(now, t - base);
  }
};

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

// Joins the KP waves that share a row tile (rt of RT): half of them hand their
// maximum, sum and NQ quads to the others through LDS, until wave 0 has all.
// lds: RT * KP / 2 * (NQ * 256 + 128) floats.
template <int KP, int RT, int NQ>
__device__ __forceinline__ void join_waves(float* lds, int kp, int rt, float& m, float& l,
                                           f32x4* o) {
  constexpr int SZ = NQ * 256 + 128;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int half = KP / 2; half >= 1; half >>= 1) {
    if (kp >= half && kp < 2 * half) {
      float* to = lds + (rt * (KP / 2) + kp - half) * SZ;
#pragma unroll
      for (int i = 0; i < NQ; ++i) *reinterpret_cast<f32x4*>(to + (i * 64 + lane) * 4) = o[i];
      to[NQ * 256 + lane] = m;
      to[NQ * 256 + 64 + lane] = l;
    }
    __syncthreads();
    if (kp < half) {
      const float* from = lds + (rt * (KP / 2) + kp) * SZ;
      const float m2 = from[NQ * 256 + lane], l2 = from[NQ * 256 + 64 + lane];
      const float mn = fmaxf(m, m2);
      const float a = exp2_fast(m - mn), c = exp2_fast(m2 - mn);
      m = mn;
      l = l * a + l2 * c;
#pragma unroll
      for (int i = 0; i < NQ; ++i)
        o[i] = o[i] * a + *reinterpret_cast<const f32x4*>(from + (i * 64 + lane) * 4) * c;
    }
    __syncthreads();
  }
}

// Writes a row tile's result: the output where its sequence has one split,
// else the split's partial result.  A lane has NQ quads of its row: columns
// col(i) .. + 3, values val(i).
template <int D, int NQ, class Col, class Val>
__device__ __forceinline__ void finish(const DecodeArgs& p, const Part& pc, int h, int rg,
                                       int row, bool row_live, int64_t qrow, int head, int g,
                                       float m, float l, Col col, Val val) {
  if (pc.starts && h == 0 && rg == 0 && threadIdx.x == 0)
    p.meta[pc.b] = make_int2(pc.slot, pc.splits);
  if (!row_live) return;
  if (pc.splits == 1) {
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    uint16_t* dst = p.out + qrow * p.o_st + head * p.o_sh;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const f32x4 x = val(i) * inv;
      *reinterpret_cast<u32x2*>(dst + col(i)) = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
    }
    if (p.lse && g == 0)
      p.lse[qrow * p.hq + head] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
  } else {
    const int64_t idx = ((int64_t)pc.slot * p.hkv + h) * p.rows + row;
    float* dst = p.part_o + idx * D;
#pragma unroll
    for (int i = 0; i < NQ; ++i) *reinterpret_cast<f32x4*>(dst + col(i)) = val(i);
    if (g == 0) {
      p.part_m[idx] = m;
      p.part_l[idx] = l;
    }
  }
}

// Up to 16 rows for a key-value head: each of 4 waves takes every fourth step of 32 keys,
// from memory to registers.
template <int D, bool FP8>
__global__ __launch_bounds__(256, 2) void attn_decode_kernel(DecodeArgs p) {
  constexpr int KP = 4;
  constexpr int NF = D / 32;                  // K fragments per 16-key tile
  constexpr int DV = D < 128 ? D / 16 : 8;    // columns of V per lane and block
  constexpr int NB = D / (16 * DV);           // blocks of 16 * DV columns
  constexpr int NG = D < 128 ? 1 : D / 128;   // FP8 scales per row
  constexpr int EB = FP8 ? 1 : 2;             // bytes per element
  constexpr int VW = DV * EB / 4;             // dwords of V per lane, row and block
  constexpr int NL = FP8 ? NF / 2 : NF;       // 16-byte loads of K per lane and tile
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int kp = wave;

  const uint32_t wg = p.first + blockIdx.x;
  const int piece = wg / p.hkv;
  const int h = wg - piece * p.hkv;
  constexpr int rg = 0;
  Piece pc;
  if (!find_piece<true>(p, piece, pc)) return;
  while (pc.at < pc.end) {
  const Part pt = part_of<true>(p, pc);
  advance(p, pt, pc);
  const int len = pt.rng.len, lo = pt.rng.lo, first = pt.first, last = pt.last;

  // this lane's row: token, head and the keys it keeps [row_lo, row_hi)
  const int row = col;
  const bool row_live = row < p.rows;
  const int tok = row_live ? row / p.group : 0;
  const int head = row_live ? h * p.group + row - tok * p.group : 0;
  const int64_t qrow = (int64_t)pt.b * p.q_len + tok;
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

  Pages pages(p, pt);
  const char* kh = p.k + h * p.sh;
  const char* vh = p.v + h * p.sh;
  const int page_mask = (1 << p.page_shift) - 1;

  for (int key0 = first + 32 * kp; key0 < last; key0 += 32 * KP) {
    bool have[2];
    int64_t off[2], srow[2];   // byte offset of the tile's first row; its index among scale rows
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int kt = key0 + 16 * t;
      int pid = pages.at(p, kt);
      have[t] = pid >= 0;
      pid = max(pid, 0);
      off[t] = pid * p.sp + (int64_t)(kt & page_mask) * p.st;
      srow[t] = (((int64_t)pid * p.hkv + h) << p.page_shift) + (kt & page_mask);
    }
    const bool inner = have[0] && have[1] && key0 >= all_lo && key0 + 32 <= all_hi;

    // K, 16 keys a tile, and V
    f32x4 s[2];
    u32x4 kr[2][NL];
    uint32_t ksc[2][NG];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if constexpr (D * EB >= 128) {
        // whole 128-byte lines of 8 rows a load, then into operand order
        const char* kb = kh + off[t] + (col & 7) * p.st + 64 * (col >> 3) + 16 * g;
#pragma unroll
        for (int j = 0; j < NL; j += 2) {
          kr[t][j] = wload<u32x4>(kb + 64 * j);
          kr[t][j + 1] = wload<u32x4>(kb + 64 * j + 8 * p.st);
        }
      } else {
        const char* kb = kh + off[t] + col * p.st;
        kr[t][0] = *reinterpret_cast<const u32x4*>(kb + 16 * g);
      }
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
            const u32x4 w = wload<u32x4>(vb + b * 16 * DV * EB);
#pragma unroll
            for (int i = 0; i < 4; ++i) vr[4 * t + r][b][i] = w[i];
          } else if constexpr (VW == 2) {
            const u32x2 w = wload<u32x2>(vb + b * 16 * DV * EB);
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
      if constexpr (D * EB >= 128)
#pragma unroll
        for (int j = 0; j < NL; j += 2) line_pair_to_steps(kr[t][j], kr[t][j + 1]);
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
    mx = quarters_max(mx);
    if (__ballot(mx > m + kLag)) {
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

  __shared__ float lds[KP / 2 * (NB * DV * 256 + 128)];
  join_waves<KP, 1, NB * DV>(lds, kp, 0, m, l, &o[0][0]);
  if (kp > 0) continue;

  // quad i: block b, row r of V's operand, columns 4 c of the lane's DV
  constexpr int QD = DV / 4;
  finish<D, NB * 4 * QD>(
      p, pt, h, rg, row, row_live, qrow, head, g, m, l,
      [&](int i) { return i / (4 * QD) * 16 * DV + (4 * g + i / QD % 4) * DV + i % QD * 4; },
      [&](int i) {
        const int b = i / (4 * QD), r = i / QD % 4, c = i % QD * 4;
        return f32x4{o[b][c][r], o[b][c + 1][r], o[b][c + 2][r], o[b][c + 3][r]};
      });
  }
}

// Position of 16-byte chunk c of row r in an LDS tile whose rows serve as keys
// (16 lanes read one chunk of 16 rows, the next 16 the neighbouring chunk) and
// as values (the transposing read takes 2 chunks of 8 rows).  A 16-byte read
// takes lanes 0-3, 12-15 and 20-27 together, then 4-11, 16-19 and 28-31: rows
// 4 to 11 share the upper places of the permutation, so that these too touch
// every bank once.
template <int D>
__device__ __forceinline__ int kv_at(int r, int c) {
  const int x = D == 64 ? ((((r >> 1) ^ (r >> 2 & 2)) & 3) << 1) | ((r >> 3) & 1)
                        : (((r ^ (r >> 1 & 4)) & 7) << 1) | ((r >> 3) & 1);
  // the permutation stays in 16 chunks, so that the rest is a constant offset
  return (r * (D / 8) + ((c & 15) ^ x)) * 16 + (c & ~15) * 16;
}

// More than 16 rows for a key-value head: RT row tiles of 16 (2 or 4), one per
// wave, share K and V through LDS, and KP waves share a row tile, 32 keys of a
// step each.  A step's tiles are loaded while the one before is computed:
// bf16 straight into LDS, FP8 through registers, turned into bf16 once for all waves.
// ONE: one tensor serves as keys and values, and is loaded once.
// At 32 sequences of up to 4096 keys with 64 rows on one 512-element head: 35 us, of
// which a workgroup's start (its piece, q, the first tiles) takes 7, eight steps
// of 64 KB 23 (5 TB/s over all CUs) and its partial result 5.  32 rows a workgroup and twice the
// steps write half as many partial results, but take 10 us more.
template <int D, bool FP8, int RT, int KP, bool ONE>
__global__ __launch_bounds__(64 * RT * KP, (ONE || D < 512) ? 2 : 1) void attn_decode_rows_kernel(
    DecodeArgs p) {
  constexpr int KT = 32 * KP;                 // keys per step
  constexpr int NF = D / 32;
  constexpr int NB = D / 16;
  constexpr int C = D / 8;                    // 16-byte bf16 chunks per row
  constexpr int NG = D < 128 ? 1 : D / 128;
  constexpr int TB = KT * D * 2;
  constexpr int NT = ONE ? 1 : 2;
  constexpr int AHEAD = D == 512 && KP == 2 ? 2 : 4;   // registers
  constexpr int LD = C / (2 * RT);            // chunks a thread stages per tensor
  constexpr int JOIN = KP > 1 ? RT * (KP / 2) * (NB * 256 + 128) * 4 : 0;
  constexpr int LDS = 2 * NT * TB > JOIN ? 2 * NT * TB : JOIN;
  __shared__ __align__(16) char lds[LDS];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int rt = wave % RT, kp = wave / RT;

  const int per_piece = p.hkv * p.rgroups;
  const uint32_t wg = p.first + blockIdx.x;
  const int piece = wg / per_piece;
  const int rest = wg - piece * per_piece;
  const int rg = rest / p.hkv, h = rest - rg * p.hkv;
  Piece pc;
  if (!find_piece<false>(p, piece, pc)) return;
  while (pc.at < pc.end) {
  const Part pt = part_of<false>(p, pc);
  advance(p, pt, pc);
  const int len = pt.rng.len, lo = pt.rng.lo, first = pt.first, last = pt.last;

  const bool tile_live = (rg * RT + rt) * 16 < p.rows;
  const int row = (rg * RT + rt) * 16 + col;
  const bool row_live = row < p.rows;
  const int tok = row_live ? row / p.group : 0;
  const int head = row_live ? h * p.group + row - tok * p.group : 0;
  const int64_t qrow = (int64_t)pt.b * p.q_len + tok;
  const int row_hi = len - p.q_len + 1 + tok;
  const int row_lo = p.window > 0 ? row_hi - p.window : 0;
  const int all_hi = len - p.q_len + 1;
  const int all_lo = p.window > 0 ? len - p.window : 0;

  bf16x8 qf[NF];
#pragma unroll
  for (int j = 0; j < NF; ++j) {
    u32x4 w = {0, 0, 0, 0};
    if (row_live)
      w = *reinterpret_cast<const u32x4*>(p.q + qrow * p.q_st + head * p.q_sh + 32 * j + 8 * g);
    qf[j] = __builtin_bit_cast(bf16x8, w);
  }
  f32x4 o[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) o[b] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = kNoMax, l = 0.f;

  Pages pages(p, pt);
  const int page_mask = (1 << p.page_shift) - 1;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  // a wave stages rows wave * WR .. of a step, in one 16-key tile and so one page
  constexpr int WR = 32 / RT;                 // rows per wave
  constexpr int RI = WR / LD;                 // rows per load of the wave
  static_assert(16 % WR == 0 && RI * LD == WR, "a wave's rows stay in one page");
  bool have[2], have_next[2];                 // whether the wave's two tiles of a step have keys
  u32x2 reg[FP8 ? NT : 1][FP8 ? LD : 1];      // FP8: codes of a step on their way
  uint32_t rsc[FP8 ? NT : 1][FP8 ? LD : 1];   // and their scale bytes
  // the chunk of its row that belongs at this lane's place of tile row tr
  auto chunk = [&](int tr, int c) { return (kv_at<D>(tr, c) >> 4) - tr * C; };
  auto fetch = [&](int buf, int key0) {
    int sr = lane / C % RI, sc = lane % C;    // row among a load's, chunk of it
    asm volatile("" : "+v"(sr), "+v"(sc));    // as below: no places kept over the loop
    const int kr = key0 + wave * WR;          // the wave's first key
    const int pid = pages.at(p, kr);
    have_next[0] = pages.at(p, key0 + 32 * kp) >= 0;
    have_next[1] = pages.at(p, key0 + 32 * kp + 16) >= 0;
    const int64_t off = (int64_t)max(pid, 0) * p.sp + h * p.sh + (int64_t)(kr & page_mask) * p.st;
    const int64_t srow = (((int64_t)max(pid, 0) * p.hkv + h) << p.page_shift) + (kr & page_mask);
    const int ra = pid >= 0 ? max(lo - kr, 0) : 0;                // rows [ra, rz) are read;
    const int rz = pid >= 0 ? max(min(len - kr, WR), 0) : 0;      // the others are zeros
    if constexpr (FP8) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const char* base = (t ? p.v : p.k) + off;
        const uint8_t* sb = (t ? p.vs : p.ks) + srow * NG;
#pragma unroll
        for (int i = 0; i < LD; ++i) {
          const int r = RI * i + sr;
          const int c = chunk(wave * WR + r, sc);
          reg[t][i] = u32x2{0, 0};
          rsc[t][i] = 127;
          if (r >= ra && r < rz) {
            reg[t][i] = *reinterpret_cast<const u32x2*>(base + (uint32_t)(r * (int)p.st + 8 * c));
            rsc[t][i] = sb[(uint32_t)(r * NG + c / 16)];
          }
        }
      }
    } else if (ra == 0 && rz == WR) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const char* base = (t ? p.v : p.k) + off;
        const uint32_t to = lds0 + (2 * t + buf) * TB + wave * WR * D * 2;
#pragma unroll
        for (int i = 0; i < LD; ++i)
          load_lds16(to + RI * i * D * 2, base + RI * i * p.st,
                     (uint32_t)(sr * (int)p.st + 16 * chunk(wave * WR + RI * i + sr, sc)));
      }
    } else {
#pragma unroll 1
      for (int j = 0; j < NT * LD; ++j) {
        const int t = j / LD, i = j % LD;
        const int r = RI * i + sr;
        u32x4 w = {0, 0, 0, 0};
        if (r >= ra && r < rz)
          w = *reinterpret_cast<const u32x4*>((t ? p.v : p.k) + off + r * p.st +
                                              16 * chunk(wave * WR + r, sc));
        *reinterpret_cast<u32x4*>(lds + (2 * t + buf) * TB + (wave * WR + RI * i) * D * 2 +
                                  lane * 16) = w;
      }
    }
  };
  auto put = [&](int buf) {                   // FP8: the fetched codes as bf16 into LDS
    if constexpr (FP8) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < LD; ++i) {
          const float s = scale_of(rsc[t][i]);
          const u32x2 a = fp8x4_to_bf16(reg[t][i][0], s), b = fp8x4_to_bf16(reg[t][i][1], s);
          *reinterpret_cast<u32x4*>(lds + (2 * t + buf) * TB + (wave * WR + RI * i) * D * 2 +
                                    lane * 16) = u32x4{a[0], a[1], b[0], b[1]};
        }
    }
  };

  if (first < last) fetch(0, first);
  put(0);
#pragma unroll
  for (int j = 0; j < NF; ++j) arrived(__builtin_bit_cast(u32x4, qf[j]));
  step_barrier<0>();
  int buf = 0;
  for (int key0 = first; key0 < last; key0 += KT, buf ^= 1) {
    const bool more = key0 + KT < last;
    have[0] = have_next[0];
    have[1] = have_next[1];
    if (more) fetch(buf ^ 1, key0 + KT);
    const int mykey = key0 + 32 * kp;
    // LDS places of this lane's chunks: kv_at's permutation is an exclusive or,
    // so chunk 4 j + g (keys) and 2 b + .. (values) are the lane's first one
    // with the bits of j or b flipped.  Worked out anew in each step: kept
    // over the loop they would take registers the loop does not have.
    const int vr = 32 * kp + 4 * g + (col >> 2);
    int ka = buf * TB + kv_at<D>(32 * kp + col, g);
    int va = (ONE ? 0 : 2 * TB) + buf * TB + kv_at<D>(vr, (col & 3) >> 1) + (col & 1) * 8;
    asm volatile("" : "+v"(ka), "+v"(va));
    if (tile_live && (KP == 1 || mykey < last)) {
      // LDS reads run AHEAD products before their use, in an order fixed by hand
      constexpr int QK = 2 * NF;
      auto read = [&](int i) {
        if (i < QK) {                         // tile i % 2, columns i / 2
          const int j = i / 2;
          return __builtin_bit_cast(
              bf16x8, *reinterpret_cast<const u32x4*>(lds + (ka ^ ((j & 3) * 64)) +
                                                      (j >> 2) * 256 + (i % 2) * 16 * D * 2));
        }
        const int b = i - QK;
        const char* v0 = lds + (va ^ ((b & 7) * 32)) + (b >> 3) * 256;
        return read_tr(v0, v0 + 16 * D * 2);
      };
      bf16x8 f[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) f[i] = read(i);
      f32x4 s[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) s[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < QK; ++i) {
        s[i % 2] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[i % AHEAD], qf[i / 2], s[i % 2], 0, 0, 0);
        f[i % AHEAD] = read(i + AHEAD);
        __builtin_amdgcn_sched_barrier(0);
      }
      float pr[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) pr[i] = s[i >> 2][i & 3] * p.scale2;
      if (!(have[0] && have[1] && mykey >= all_lo && mykey + 32 <= all_hi)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int key = mykey + 16 * (i >> 2) + 4 * g + (i & 3);
          if (!(have[i >> 2] && key < row_hi && key >= row_lo)) pr[i] = -INFINITY;
        }
      }
      float mx = pr[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) mx = fmaxf(mx, pr[i]);
      mx = quarters_max(mx);
      if (__ballot(mx > m + kLag)) {
        const float mn = fmaxf(m, mx);
        const float a = exp2_fast(m - mn);
        m = mn;
        l *= a;
#pragma unroll
        for (int b = 0; b < NB; ++b) o[b] *= a;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) pr[i] = exp2_fast(pr[i] - m);
      l += ((pr[0] + pr[1]) + (pr[2] + pr[3])) + ((pr[4] + pr[5]) + (pr[6] + pr[7]));
      const u32x4 pw = {pack_bf16(pr[0], pr[1]), pack_bf16(pr[2], pr[3]),
                        pack_bf16(pr[4], pr[5]), pack_bf16(pr[6], pr[7])};
      const bf16x8 pf = __builtin_bit_cast(bf16x8, pw);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        o[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[(QK + b) % AHEAD], pf, o[b], 0, 0, 0);
        if (b + AHEAD < NB) f[(QK + b) % AHEAD] = read(QK + b + AHEAD);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (more) put(buf ^ 1);
    step_barrier<0>();
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if constexpr (KP > 1) {
    join_waves<KP, RT, NB>(reinterpret_cast<float*>(lds), kp, rt, m, l, o);
    if (kp > 0) continue;
  }
  finish<D, NB>(
      p, pt, h, rg, row, row_live, qrow, head, g, m, l,
      [&](int i) { return 16 * i + 4 * g; }, [&](int i) { return o[i]; });
  }
}

// Joins the splits of a sequence: one workgroup per (sequence, head, row);
// rows of a sequence with one split are written already.  A group of D / 4 lanes takes a split's
// row, the groups every (1024 / D)th split, and their sums meet in LDS.
template <int D>
__global__ __launch_bounds__(256) void attn_decode_join_kernel(DecodeArgs p) {
  constexpr int GL = D / 4, NGR = 256 / GL;
  __shared__ f32x4 so[NGR][GL];
  __shared__ float sm[NGR], sl[NGR];
  const uint32_t per_b = (uint32_t)(p.hkv * p.rows);
  const uint32_t wg = p.first + blockIdx.x;
  const uint32_t b = wg / per_b;
  const int rest = (int)(wg - b * per_b);
  const int h = rest / p.rows, row = rest - h * p.rows;
  const int2 mt = p.meta[b];
  if (mt.y <= 1) return;
  const int64_t at0 = (int64_t)mt.x * per_b + (int64_t)h * p.rows + row;
  const int gr = threadIdx.x / GL, gl = threadIdx.x % GL;
  // a group's own running maximum: no load waits for another's
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  float l = 0.f, m = kNoMax;
#pragma unroll 4
  for (int i = gr; i < mt.y; i += NGR) {
    const int64_t at = at0 + (int64_t)i * per_b;
    const float mi = p.part_m[at], li = p.part_l[at];
    const f32x4 oi = *reinterpret_cast<const f32x4*>(p.part_o + at * D + gl * 4);
    const float mn = fmaxf(m, mi);
    const float a = exp2_fast(m - mn), c = exp2_fast(mi - mn);
    m = mn;
    l = l * a + li * c;
    o = o * a + oi * c;
  }
  so[gr][gl] = o;
  if (gl == 0) {
    sm[gr] = m;
    sl[gr] = l;
  }
  __syncthreads();
  if (gr > 0) return;
  float top = sm[0];
#pragma unroll
  for (int i = 1; i < NGR; ++i) top = fmaxf(top, sm[i]);
  o = f32x4{0.f, 0.f, 0.f, 0.f};
  l = 0.f;
#pragma unroll
  for (int i = 0; i < NGR; ++i) {
    const float a = exp2_fast(sm[i] - top);
    o += so[i][gl] * a;
    l += sl[i] * a;
  }
  m = top;
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  o *= inv;
  const int tok = row / p.group;
  const int head = h * p.group + row - tok * p.group;
  const int64_t qrow = (int64_t)b * p.q_len + tok;
  *reinterpret_cast<u32x2*>(p.out + qrow * p.o_st + head * p.o_sh + gl * 4) =
      u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
  if (p.lse && gl == 0)
    p.lse[qrow * p.hq + head] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
}

// Row tiles of a workgroup; 1: the kernel without LDS, which for up to 16 rows
// takes 107 us where the other takes 132 (64 sequences of up to 4096 keys, 4 rows
// of 128 elements a head), with FP8 51 and 116 (one of 131071).  512-element heads have no registers for it.
// Two tiles for 17 to 32 rows, and twice as many keys a step: 64 us instead of
// 77 with four (32 sequences of 4096 keys, 32 rows of 128 elements); with 256
// elements four, since a twofold step takes most of the LDS and leaves one
// workgroup on a CU (16 sequences of 4096: 70 us with two, 62 with four).
int row_tiles(int rows, int dim) {
  return dim == 512 ? 4 : rows <= 16 ? 1 : rows <= 32 && dim < 256 ? 2 : 4;
}

struct DecodePlan {
  int rows, rgroups, pieces;
  int64_t slots;
};
// Whether no sequence is cut: a workgroup takes one whole, and the call is one
// kernel.  A cut costs a second launch and the join; without it a workgroup
// reads a sequence's keys and values of a head (`bytes` at most) at the rate of one CU.
// Measured, whole and cut: 300 keys of 128 elements 7.8 and 9.7 us, 8
// sequences of 450 11.6 and 10.7, 500 keys of 256 elements 17.8 and 14.0; with
// a workgroup for every CU, 32 sequences of 500 keys 14.5 and 18.9, of 1000
// 21.4 and 23.2; in the many-row kernel 3 of 120 16.9 and 18.8, 4 of 500 39 and 19.
bool whole_sequences(int64_t bytes, int64_t workgroups, bool many_rows) {
  const int64_t most = workgroups >= 256 ? 512 : many_rows ? 128 : 192;
  return bytes <= most * 1024;
}
DecodePlan plan_of(const moe_attn_config& c) {
  DecodePlan d;
  d.rows = c.q_len * (c.heads_q / c.heads_kv);
  const int rt = row_tiles(d.rows, c.head_dim);
  d.rgroups = (d.rows + 16 * rt - 1) / (16 * rt);
  d.pieces = std::max(1, (rt == 1 ? kPieces : pieces_rows(c.batch)) / (c.heads_kv * d.rgroups));
  d.slots = (int64_t)d.pieces + c.batch;
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
  a.rows = d.rows; a.rgroups = d.rgroups;
  const bool one = kv.k == kv.v && (eb == 2 || kv.k_scale == kv.v_scale);
  const bool whole = whole_sequences(
      ((int64_t)table_width << a.page_shift) * c.head_dim * eb * (one ? 1 : 2),
      (int64_t)c.batch * c.heads_kv * d.rgroups, row_tiles(d.rows, c.head_dim) > 1);
  a.pieces = whole ? 0 : d.pieces;
  a.tile_shift = row_tiles(d.rows, c.head_dim) == 1 ? 7 : 6;
  a.window = c.window; a.scale2 = c.scale * kLog2e;
  const size_t rows = (size_t)d.slots * c.heads_kv * d.rows;
  char* w = static_cast<char*>(ws);
  a.part_o = reinterpret_cast<float*>(w); w += up256(rows * c.head_dim * 4);
  a.part_m = reinterpret_cast<float*>(w); w += up256(rows * 4);
  a.part_l = reinterpret_cast<float*>(w); w += up256(rows * 4);
  a.meta = reinterpret_cast<int2*>(w);
  const int64_t cut = row_tiles(d.rows, c.head_dim) == 1 ? d.pieces : d.slots;
  const int64_t workgroups = (whole ? c.batch : cut) * c.heads_kv * d.rgroups;
  const int rt = row_tiles(d.rows, c.head_dim);
  const bool f8 = kv.format == MOE_KV_FP8;
#define MOE_ROWS(D, F, R, KP, O)                                                              \
  hipLaunchKernelGGL((attn_decode_rows_kernel<D, F, R, KP, O>), grid, dim3(64 * R * KP), 0, st, a)
#define MOE_ROWS_ANY(D, F, R)                                                                 \
  do {                                                                                        \
    if (one) MOE_ROWS(D, F, R, (D == 512 ? 2 : 4 / R), true);                                 \
    else MOE_ROWS(D, F, R, 4 / R, false);                                                     \
  } while (0)
#define MOE_DIRECT(D, F)                                                                      \
  hipLaunchKernelGGL((attn_decode_kernel<D, F>), grid, dim3(256), 0, st, a)
#define MOE_FEW(D, F)                                                                         \
  do {                                                                                        \
    if (rt == 1) MOE_DIRECT(D, F);                                                            \
    else if (rt == 2) MOE_ROWS_ANY(D, F, 2);                                                  \
    else MOE_ROWS_ANY(D, F, 4);                                                               \
  } while (0)
#define MOE_DECODE(D)                                                                         \
  case D:                                                                                     \
    if (f8) MOE_FEW(D, true); else MOE_FEW(D, false);                                         \
    break;
  hipError_t e = launch_workgroups(workgroups, [&](uint32_t first, dim3 grid) {
    a.first = first;
    switch (c.head_dim) {
      MOE_DECODE(64) MOE_DECODE(128)
      case 256:
        if (rt == 1) {
          if (f8) MOE_DIRECT(256, true); else MOE_DIRECT(256, false);
          break;
        }
        if (f8) MOE_ROWS_ANY(256, true, 4); else MOE_ROWS_ANY(256, false, 4);
        break;
      case 512:
        if (f8) MOE_ROWS_ANY(512, true, 4); else MOE_ROWS_ANY(512, false, 4);
        break;
    }
  });
#undef MOE_DECODE
#undef MOE_FEW
#undef MOE_DIRECT
#undef MOE_ROWS_ANY
#undef MOE_ROWS
  if (e != hipSuccess || whole) return e;
#define MOE_JOIN(D) \
  case D: hipLaunchKernelGGL((attn_decode_join_kernel<D>), grid, dim3(256), 0, st, a); break;
  return launch_workgroups((int64_t)c.batch * c.heads_kv * d.rows, [&](uint32_t first, dim3 grid) {
    a.first = first;
    switch (c.head_dim) { MOE_JOIN(64) MOE_JOIN(128) MOE_JOIN(256) MOE_JOIN(512) }
  });
#undef MOE_JOIN
}

}  // namespace moe
