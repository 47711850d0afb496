// Kernels of attention over the paged key-value cache: new tokens that see everything
// before them (attn_decode.hip), and with TREE those of a drafted tree, or of a window with
// first tokens that stay visible (attn_tree.hip).
#pragma once

#include <algorithm>
#include <climits>

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
  const uint64_t* masks;   // TREE: [batch][q_len], or null: rows are causal
  int sinks;               // TREE: first tokens that stay visible
  uint32_t q_flip;         // attn_tree_rows.hip: sign bits to flip in q, where scale2 is |scale| log2(e)
  uint32_t total;          // ... its workgroups
  int row_groups;          // ... and their groups of 32 rows
};

// An entry of a table that no kernel writes, at a wave-uniform index: a scalar load.
__device__ __forceinline__ int entry(const int32_t* t, int64_t i) {
  return *(const __attribute__((address_space(4))) int32_t*)(t + i);
}

// Keys a sequence's rows may reach: [lo, len), and how many tiles that is, counted from lo rounded down to a step of 32 (1 for none).
// TREE: the rows also reach the first tokens, and the walk leaves the keys between out: place v of
// it is key v below `front` and key v + gap from there on (both multiples of 32), for v < end.
// ctx: keys before the new tokens (below 0: the first rows stand before the sequence).
struct Range {
  int lo, len, tiles;
  int ctx, front, gap, end;
  __device__ __forceinline__ int key_of(int v) const { return v < front ? v : v + gap; }
};
template <bool TREE>
__device__ __forceinline__ Range range_of(const DecodeArgs& p, int raw_len) {
  Range r;
  const int64_t cap = (int64_t)p.table_width << p.page_shift;
  r.len = (int)min((int64_t)max(raw_len, 0), cap);
  if constexpr (TREE) {
    r.ctx = p.masks ? r.len : r.len - p.q_len;
    r.len = (int)min((int64_t)r.ctx + p.q_len, cap);
    if (p.pages == 0) r.len = 0;
    r.lo = p.window > 0 ? max(r.ctx + 1 - p.window, 0) : 0;   // of a row at the context's end
    const int near = r.lo & ~31;
    r.front = (max(min(min(p.sinks, r.ctx), r.lo), 0) + 31) & ~31;
    r.gap = max(near - r.front, 0);
    r.end = r.len - r.gap;
    r.tiles = r.end > 0 ? (r.end + (1 << p.tile_shift) - 1) >> p.tile_shift : 1;
    return r;
  }
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

// TREE: what this lane's row, and any row, keeps among the new tokens (a bit each) and before them.
struct Seen {
  uint64_t mine, any;
  int row_lo, row_sinks;    // of the context the row keeps [row_lo, ctx) and [0, row_sinks)
  int lo, sinks;            // some row does
  int all_lo;               // every row that keeps anything keeps [all_lo, ctx)
  bool keeps;               // the row has a place in its sequence
};
__device__ __forceinline__ uint64_t low_bits(int n) {
  return n <= 0 ? 0 : n >= 64 ? ~uint64_t(0) : (uint64_t(1) << n) - 1;
}
// Bit i of x, as 0 or 1; 0 past the last one, any value below 0.
__device__ __forceinline__ uint32_t bit_of(uint64_t x, int i) {
  const uint32_t w = i < 32 ? (uint32_t)x : (uint32_t)(x >> 32);
  return i < 64 ? w >> (i & 31) & 1 : 0;
}
// f over all lanes, in all of them; `none` is f's neutral value.
template <class F>
__device__ __forceinline__ int wave_all(int x, int none, F f) {
  x = f(x, __builtin_amdgcn_update_dpp(none, x, 0x111, 0xF, 0xF, false));   // row_shr 1, 2, 4, 8
  x = f(x, __builtin_amdgcn_update_dpp(none, x, 0x112, 0xF, 0xF, false));
  x = f(x, __builtin_amdgcn_update_dpp(none, x, 0x114, 0xF, 0xF, false));
  x = f(x, __builtin_amdgcn_update_dpp(none, x, 0x118, 0xF, 0xF, false));
  x = f(x, __builtin_amdgcn_update_dpp(none, x, 0x142, 0xA, 0xF, false));   // lane 15 of a row to the next
  x = f(x, __builtin_amdgcn_update_dpp(none, x, 0x143, 0xC, 0xF, false));   // lane 31 to rows 2 and 3
  return __builtin_amdgcn_readlane(x, 63);
}
__device__ __forceinline__ Seen seen_of(const DecodeArgs& p, const Range& r, int b, int tok,
                                        bool row_live) {
  const int lane = threadIdx.x & 63;       // a new token per lane
  uint64_t m = 0;
  int pos = r.ctx + lane;                  // its position
  bool live = lane < p.q_len;
  if (p.masks) {
    if (live) m = p.masks[(int64_t)b * p.q_len + lane] & low_bits(p.q_len);
    live = m != 0;
    pos = r.ctx + __popcll(m) - 1;
  } else if (live) {
    live = pos >= 0;
    // its window, and first tokens that are new themselves
    m = low_bits(lane + 1);
    if (p.window > 0) m &= ~low_bits(lane + 1 - p.window) | low_bits(p.sinks - r.ctx);
  }
  m &= low_bits(r.len - r.ctx) & ~low_bits(-r.ctx);
  auto either = [](int a, int b) { return a | b; };
  const int any_lo = wave_all((int)(uint32_t)m, 0, either);
  const int any_hi = wave_all((int)(uint32_t)(m >> 32), 0, either);
  Seen s;
  s.any = (uint64_t)(uint32_t)any_hi << 32 | (uint32_t)any_lo;
  int first = INT_MAX, last = -1;          // rows' positions, which a window goes by
  const bool some = __ballot(live) != 0;
  if (p.window > 0) {
    first = wave_all(live ? pos : INT_MAX, INT_MAX, [](int a, int b) { return min(a, b); });
    last = wave_all(live ? pos : -1, -1, [](int a, int b) { return max(a, b); });
  }
  const int at = __shfl(pos, tok);
  const int there = __shfl((int)live, tok);   // by all lanes: any may be asked
  s.keeps = row_live && there;
  s.mine = (uint64_t)__shfl((uint32_t)(m >> 32), tok) << 32 | __shfl((uint32_t)m, tok);
  const int sinks = max(min(p.sinks, r.ctx), 0);
  auto start = [&](int q) { return p.window > 0 ? max(q + 1 - p.window, 0) : 0; };
  s.row_lo = s.keeps ? start(at) : INT_MAX;
  s.row_sinks = s.keeps ? sinks : 0;
  s.lo = __builtin_amdgcn_readfirstlane(some ? start(first) : INT_MAX);
  s.sinks = __builtin_amdgcn_readfirstlane(some ? sinks : 0);
  s.all_lo = __builtin_amdgcn_readfirstlane(some ? start(last) : INT_MAX);
  if (!s.keeps) s.mine = 0;
  return s;
}
// Whether the row, or any row, keeps a key of the sequence.  Without branches: lanes differ.
__device__ __forceinline__ bool row_keeps(const Seen& s, const Range& r, int key) {
  const uint32_t context = (uint32_t)(key >= s.row_lo) | (uint32_t)(key < s.row_sinks);
  return (key < r.ctx ? context : bit_of(s.mine, key - r.ctx)) != 0;
}
__device__ __forceinline__ bool any_keeps(const Seen& s, const Range& r, int key) {
  const uint32_t context = (uint32_t)(key >= s.lo) | (uint32_t)(key < s.sinks);
  return (key < r.ctx ? context : bit_of(s.any, key - r.ctx)) != 0;
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
template <bool ACROSS, bool TREE>
__device__ __forceinline__ bool find_piece(const DecodeArgs& p, int w, Piece& out) {
  const int lane = threadIdx.x & 63;
  if (p.pieces == 0) {                 // nothing is cut: piece w is sequence w
    out.w = 0;
    out.per = 1u << 30;
    out.b = w;
    out.tile = 0;
    out.len = entry(p.seq_lens, w);
    out.at = 0;
    out.end = range_of<TREE>(p, out.len).tiles;
    return true;
  }
  uint32_t total = 0;   // the host has checked that it stays below 2^31
  int raw = 0, mine = 0, incl = 0;   // the last 64 sequences looked at
  auto look = [&](int b0) {
    raw = b0 + lane < p.batch ? p.seq_lens[b0 + lane] : 0;
    mine = b0 + lane < p.batch ? range_of<TREE>(p, raw).tiles : 0;
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
  int first, last;  // keys (TREE: places of the walk)
};
template <bool ACROSS, bool TREE>
__device__ __forceinline__ Part part_of(const DecodeArgs& p, const Piece& pc) {
  Part x;
  x.b = pc.b;
  x.slot = ACROSS ? pc.w + pc.b : pc.w;
  x.rng = range_of<TREE>(p, pc.len);
  const uint32_t begin = pc.at - pc.tile;   // the sequence's first tile in all the work, or 0
  x.splits = __builtin_amdgcn_readfirstlane(
      (int)((begin + x.rng.tiles - 1) / pc.per - begin / pc.per) + 1);
  x.starts = pc.tile == 0;
  const int n = min((int)(pc.end - pc.at), x.rng.tiles - pc.tile);
  x.first = (TREE ? 0 : x.rng.lo & ~31) + (pc.tile << p.tile_shift);
  x.last = (int)min((int64_t)(TREE ? x.rng.end : x.rng.len),
                    (int64_t)x.first + ((int64_t)n << p.tile_shift));
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
template <bool TREE>
struct Pages {
  const int32_t* row;
  int len, lo, base, now, next;
  int front, gap;
  __device__ __forceinline__ int load(const DecodeArgs& p, int tile) const {
    int64_t key = 16 * ((int64_t)tile + (threadIdx.x & 63));
    if (!(key < len && key + 16 > lo)) return -1;
    if (TREE && key >= front) key += gap;
    const int id = row[key >> p.page_shift];
    return id >= 0 && id < p.pages ? id : -1;
  }
  __device__ __forceinline__ Pages(const DecodeArgs& p, const Part& pt)
      : row(p.table + (int64_t)pt.b * p.table_width), len(TREE ? pt.rng.end : pt.rng.len),
        lo(TREE ? 0 : pt.rng.lo), base(pt.first >> 4), front(pt.rng.front), gap(pt.rng.gap) {
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

// Up to 16 rows for a key-value head (TREE: in each of its row groups): each of 4 waves takes every fourth step of 32 keys,
// from memory to registers.
template <int D, bool FP8, bool TREE>
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
  const int per_piece = TREE ? p.hkv * p.rgroups : p.hkv;
  const int piece = wg / per_piece;
  const int rest = wg - piece * per_piece;
  const int rg = TREE ? rest / p.hkv : 0, h = rest - rg * p.hkv;
  Piece pc;
  if (!find_piece<true, TREE>(p, piece, pc)) return;
  while (pc.at < pc.end) {
  const Part pt = part_of<true, TREE>(p, pc);
  advance(p, pt, pc);
  const int len = pt.rng.len, lo = pt.rng.lo, first = pt.first, last = pt.last;

  // this lane's row: token, head and the keys it keeps [row_lo, row_hi)
  const int row = TREE ? rg * 16 + col : col;
  const bool row_live = row < p.rows;
  const int tok = row_live ? row / p.group : 0;
  const int head = row_live ? h * p.group + row - tok * p.group : 0;
  const int64_t qrow = (int64_t)pt.b * p.q_len + tok;
  const int row_hi = len - p.q_len + 1 + tok;
  const int row_lo = p.window > 0 ? row_hi - p.window : 0;

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

  Pages<TREE> pages(p, pt);
  Seen seen;                                  // after the loads of q and pages have gone out
  if constexpr (TREE) seen = seen_of(p, pt.rng, pt.b, tok, row_live);
  const int all_hi = TREE ? pt.rng.ctx : len - p.q_len + 1;   // every row keeps [all_lo, all_hi)
  const int all_lo = TREE ? seen.all_lo : p.window > 0 ? len - p.window : 0;
  const char* kh = p.k + h * p.sh;
  const char* vh = p.v + h * p.sh;
  const int page_mask = (1 << p.page_shift) - 1;

  for (int at0 = first + 32 * kp; at0 < last; at0 += 32 * KP) {
    const int key0 = TREE ? pt.rng.key_of(at0) : at0;
    bool have[2];
    int64_t off[2], srow[2];   // byte offset of the tile's first row; its index among scale rows
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int kt = key0 + 16 * t;
      int pid = pages.at(p, at0 + 16 * t);
      have[t] = pid >= 0;
      pid = max(pid, 0);
      off[t] = pid * p.sp + (int64_t)(kt & page_mask) * p.st;
      srow[t] = (((int64_t)pid * p.hkv + h) << p.page_shift) + (kt & page_mask);
    }
    const bool inner = have[0] && have[1] && ((key0 >= all_lo && key0 + 32 <= all_hi) ||
                                              (TREE && key0 + 32 <= seen.sinks));

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
          const bool kept = TREE ? row_keeps(seen, pt.rng, key) : key < row_hi && key >= row_lo;
          if (!(have[t] && kept)) pr[4 * t + i] = -INFINITY;
          const bool used = have[t] && (TREE ? any_keeps(seen, pt.rng, key) : key < len && key >= lo);
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
  if constexpr (TREE) {                       // a row without a place keeps nothing, whatever its q
    if (!seen.keeps) {
      m = kNoMax;
      l = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < DV; ++i) o[b][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }

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
template <int D, bool FP8, int RT, int KP, bool ONE, bool TREE>
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
  if (!find_piece<false, TREE>(p, piece, pc)) return;
  while (pc.at < pc.end) {
  const Part pt = part_of<false, TREE>(p, pc);
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

  Pages<TREE> pages(p, pt);
  Seen seen;                                  // after the loads of q and pages have gone out
  if constexpr (TREE) seen = seen_of(p, pt.rng, pt.b, tok, row_live);
  const int all_hi = TREE ? pt.rng.ctx : len - p.q_len + 1;   // every row keeps [all_lo, all_hi)
  const int all_lo = TREE ? seen.all_lo : p.window > 0 ? len - p.window : 0;
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
    const int pid = pages.at(p, key0 + wave * WR);
    // the wave's first key
    const int kr = TREE ? pt.rng.key_of(key0 + wave * WR) : key0 + wave * WR;
    have_next[0] = pages.at(p, key0 + 32 * kp) >= 0;
    have_next[1] = pages.at(p, key0 + 32 * kp + 16) >= 0;
    const int64_t off = (int64_t)max(pid, 0) * p.sp + h * p.sh + (int64_t)(kr & page_mask) * p.st;
    const int64_t srow = (((int64_t)max(pid, 0) * p.hkv + h) << p.page_shift) + (kr & page_mask);
    const int ra = pid >= 0 ? max(lo - kr, 0) : 0;                // rows [ra, rz) are read;
    const int rz = pid >= 0 ? max(min(len - kr, WR), 0) : 0;      // the others are zeros
    const bool whole = TREE ? pid >= 0 && ((kr >= seen.lo && kr + WR <= pt.rng.ctx) ||
                                           kr + WR <= seen.sinks)
                            : ra == 0 && rz == WR;
    auto is_read = [&](int r) {
      return TREE ? pid >= 0 && any_keeps(seen, pt.rng, kr + r) : r >= ra && r < rz;
    };
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
          if (TREE ? whole || is_read(r) : is_read(r)) {
            reg[t][i] = *reinterpret_cast<const u32x2*>(base + (uint32_t)(r * (int)p.st + 8 * c));
            rsc[t][i] = sb[(uint32_t)(r * NG + c / 16)];
          }
        }
      }
    } else if (whole) {
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
        if (is_read(r))
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
      const int base = TREE ? pt.rng.key_of(mykey) : mykey;
      if (!(have[0] && have[1] && ((base >= all_lo && base + 32 <= all_hi) ||
                                   (TREE && base + 32 <= seen.sinks)))) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int key = base + 16 * (i >> 2) + 4 * g + (i & 3);
          const bool kept = TREE ? row_keeps(seen, pt.rng, key) : key < row_hi && key >= row_lo;
          if (!(have[i >> 2] && kept)) pr[i] = -INFINITY;
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
  if constexpr (TREE) {                       // a row without a place keeps nothing, whatever its q
    if (!seen.keeps) {
      m = kNoMax;
      l = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b) o[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
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

size_t decode_ws_bytes(const moe_attn_config& c) {
  const DecodePlan d = plan_of(c);
  const size_t rows = (size_t)d.slots * c.heads_kv * d.rows;
  return up256(rows * c.head_dim * 4) + 2 * up256(rows * 4) + up256((size_t)c.batch * 8);
}

// The arguments that do not depend on the cut of the work.
DecodeArgs decode_args(const moe_attn_config& c, const moe_rows& q, const moe_kv_cache& kv,
                       const int32_t* table, int table_width, const int32_t* seq_lens,
                       const moe_rows& out, float* lse) {
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
  a.window = c.window; a.scale2 = c.scale * kLog2e;
  return a;
}

// Keys of a sequence that its rows may reach, by the table's width and the window.
template <bool TREE>
int64_t longest_walk(const moe_attn_config& c, const DecodeArgs& a) {
  const int64_t longest = (int64_t)a.table_width << a.page_shift;
  if (!TREE || c.window == 0) return longest;
  return std::min(longest, (int64_t)c.window + a.sinks + c.q_len + 64);
}

// Row groups of 16 for the kernel without LDS where there are more rows, but so few keys and
// workgroups that it is one launch which ends sooner than the others, though every group reads
// the keys again; 0: the others.  8 nodes of 32 heads on 8 of 128, 300 keys, with the masks: 12.3
// us, cut and joined 14.7.
int narrow_groups(const moe_attn_config& c, int64_t bytes) {
  const int64_t rows = (int64_t)c.q_len * (c.heads_q / c.heads_kv), groups = (rows + 15) / 16;
  const int64_t workgroups = c.batch * c.heads_kv * groups;
  return c.head_dim < 512 && rows > 16 && workgroups <= 512 && whole_sequences(bytes, 0, false) ? (int)groups : 0;
}

// (a template, so that sources which do not launch it hold no such kernels)
template <bool TREE>
hipError_t launch_join(const moe_attn_config& c, DecodeArgs a, hipStream_t st) {
#define MOE_JOIN(D) \
  case D: hipLaunchKernelGGL((attn_decode_join_kernel<D>), grid, dim3(256), 0, st, a); break;
  return launch_workgroups((int64_t)c.batch * c.heads_kv * a.rows, [&](uint32_t first, dim3 grid) {
    a.first = first;
    switch (c.head_dim) { MOE_JOIN(64) MOE_JOIN(128) MOE_JOIN(256) MOE_JOIN(512) }
  });
#undef MOE_JOIN
}

// masks, sinks: see DecodeArgs.
template <bool TREE>
hipError_t launch_decode(const moe_attn_config& c, const moe_rows& q, const moe_kv_cache& kv,
                         const int32_t* table, int table_width, const int32_t* seq_lens,
                         const uint64_t* masks, int sinks, const moe_rows& out, float* lse,
                         void* ws, hipStream_t st) {
  if (c.batch == 0) return hipSuccess;
  const DecodePlan d = plan_of(c);
  DecodeArgs a = decode_args(c, q, kv, table, table_width, seq_lens, out, lse);
  a.masks = masks; a.sinks = sinks;
  a.rows = d.rows; a.rgroups = d.rgroups;
  const int eb = kv.format == MOE_KV_FP8 ? 1 : 2;
  const bool one = kv.k == kv.v && (eb == 2 || kv.k_scale == kv.v_scale);
  const int64_t bytes = longest_walk<TREE>(c, a) * c.head_dim * eb * (one ? 1 : 2);
  const int narrow = TREE ? narrow_groups(c, bytes) : 0;
  if (narrow) a.rgroups = narrow;
  const int rt = narrow ? 1 : row_tiles(d.rows, c.head_dim);
  const bool whole = narrow || whole_sequences(bytes, (int64_t)c.batch * c.heads_kv * d.rgroups, rt > 1);
  a.pieces = whole ? 0 : d.pieces;
  a.tile_shift = rt == 1 ? 7 : 6;
  const size_t rows = (size_t)d.slots * c.heads_kv * d.rows;
  char* w = static_cast<char*>(ws);
  a.part_o = reinterpret_cast<float*>(w); w += up256(rows * c.head_dim * 4);
  a.part_m = reinterpret_cast<float*>(w); w += up256(rows * 4);
  a.part_l = reinterpret_cast<float*>(w); w += up256(rows * 4);
  a.meta = reinterpret_cast<int2*>(narrow ? ws : w);
  const int64_t cut = rt == 1 ? d.pieces : d.slots;
  const int64_t workgroups = (whole ? c.batch : cut) * c.heads_kv * a.rgroups;
  const bool f8 = kv.format == MOE_KV_FP8;
#define MOE_ROWS(D, F, R, KP, O)                                                              \
  hipLaunchKernelGGL((attn_decode_rows_kernel<D, F, R, KP, O, TREE>), grid, dim3(64 * R * KP), 0, st, a)
#define MOE_ROWS_ANY(D, F, R)                                                                 \
  do {                                                                                        \
    if (one) MOE_ROWS(D, F, R, (D == 512 ? 2 : 4 / R), true);                                 \
    else MOE_ROWS(D, F, R, 4 / R, false);                                                     \
  } while (0)
#define MOE_DIRECT(D, F)                                                                      \
  hipLaunchKernelGGL((attn_decode_kernel<D, F, TREE>), grid, dim3(256), 0, st, a)
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
  return launch_join<TREE>(c, a, st);
}

}  // namespace

}  // namespace moe
