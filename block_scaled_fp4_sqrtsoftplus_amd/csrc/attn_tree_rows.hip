// Tree attention over the paged cache where a key-value head has many rows:
// a group of heads times up to 64 drafted tokens (include/moe_serving.h,
// moe_attn_tree).
//
// Mathematics: one pass over the keys with a softmax's running maximum and
// sum, as attn_decode.hip; masks as attn_tree.hip.
//
// Matrix form: that of attn_prefill.hip, S^T = K Q^T and O^T = V^T P^T on
// 32x32x16 MFMA, a wave per 32 rows (two waves with half of the columns each
// for 512-element heads, which add their scores through LDS).  Four row groups
// share K and V in LDS.  The kernels for few rows have 16 to a wave, which
// reads all of K and V from LDS for half as many products: LDS then is the
// bound.  Keys come through the block table 16 rows at a time, bf16 straight
// into LDS, FP8 through registers, turned into bf16 once for all waves.
#include "attn_decode_kernels.h"
#include "attn_tiles.h"

namespace moe {

namespace {

// One workgroup's work: a part of a sequence's walk.  `slots` workgroups (of a
// head and row group) take all sequences, each cut by itself into parts of
// equal length: at most `per` tiles, the least for which the slots suffice
// (in steps of an eighth).  slots 0: a workgroup per sequence.
struct Cut {
  int b, slot, splits;
  bool starts;
  int tile, tiles;    // of the walk
};
__device__ __forceinline__ bool find_cut(const DecodeArgs& p, int w, Cut& c) {
  const int lane = threadIdx.x & 63;
  if (p.pieces == 0) {
    c = Cut{w, 0, 1, true, 0, range_of<true>(p, entry(p.seq_lens, w)).tiles};
    return true;
  }
  uint32_t total = 0;
  int mine = 0;              // the last 64 sequences looked at
  auto look = [&](int b0) {
    mine = b0 + lane < p.batch ? range_of<true>(p, p.seq_lens[b0 + lane]).tiles : 0;
  };
  for (int b0 = 0; b0 < p.batch; b0 += 64) {
    look(b0);
    total += __builtin_amdgcn_readlane(wave_scan(mine), 63);
  }
  uint32_t per = (total + p.pieces - 1) / p.pieces;
  for (;; per += (per + 7) / 8) {
    per = __builtin_amdgcn_readfirstlane(per);
    int parts = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 64) {
      if (p.batch > 64) look(b0);
      parts += __builtin_amdgcn_readlane(wave_scan((int)((mine + per - 1) / per)), 63);
    }
    if (parts <= p.pieces || per >= total) break;   // pieces >= batch: a part each fits
  }
  int base = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 64) {
    if (p.batch > 64) look(b0);
    const int n = (int)((mine + per - 1) / per);
    const int incl = wave_scan(n);
    const uint64_t past = __ballot(base + incl > w);
    if (past) {
      const int l = __builtin_ctzll(past);
      c.b = b0 + l;
      c.splits = __builtin_amdgcn_readlane(n, l);
      const int i = w - (base + __builtin_amdgcn_readlane(incl, l) - c.splits);
      const int all = __builtin_amdgcn_readlane(mine, l);
      c.slot = w;
      c.starts = i == 0;
      c.tile = (int)((int64_t)all * i / c.splits);
      c.tiles = (int)((int64_t)all * (i + 1) / c.splits) - c.tile;
      return true;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// Where 16-key tiles of the walk lie, 64 of them and the next 64, a tile per
// lane: a step gets the places of its tiles from lanes, with no page to wait for
// and no product to form.
template <bool FP8>
struct WalkTiles {
  struct Group {
    uint32_t lo, hi;       // byte offset of the tile's first row in k and v
    uint32_t slo, shi;     // FP8: its row among the scales
    uint64_t ok;           // tiles whose page is there
  };
  const int32_t* row;
  Range rng;
  int base, h;
  Group now, next;
  __device__ __forceinline__ Group load(const DecodeArgs& p, int tile) const {
    const int64_t v = 16 * ((int64_t)tile + (threadIdx.x & 63));
    int id = -1;
    int64_t key = v;
    if (v < rng.end) {
      if (key >= rng.front) key += rng.gap;
      id = row[key >> p.page_shift];
    }
    const bool ok = id >= 0 && id < p.pages;
    const int64_t page = ok ? id : 0;
    const int in_page = (int)(key & ((1 << p.page_shift) - 1));
    const int64_t off = page * p.sp + h * p.sh + in_page * p.st;
    const int64_t srow = FP8 ? ((page * p.hkv + h) << p.page_shift) + in_page : 0;
    return Group{(uint32_t)off, (uint32_t)(off >> 32), (uint32_t)srow, (uint32_t)(srow >> 32), __ballot(ok)};
  }
  __device__ __forceinline__ WalkTiles(const DecodeArgs& p, const Range& r, int b, int head, int tile)
      : row(p.table + (int64_t)b * p.table_width), rng(r), base(tile), h(head) {
    now = load(p, base);
    next = load(p, base + 64);
  }
  // no tile before this one is asked for any more
  __device__ __forceinline__ void advance(const DecodeArgs& p, int tile) {
    if (tile < base + 64) return;
    base += 64;
    now = next;
    next = load(p, base + 64);
  }
  __device__ __forceinline__ int64_t offset(int tile) const {
    const int i = tile - base;
    return (int64_t)(((uint64_t)__builtin_amdgcn_readlane(now.hi, i) << 32) | (uint32_t)__builtin_amdgcn_readlane(now.lo, i));
  }
  __device__ __forceinline__ int64_t scale_row(int tile) const {
    const int i = tile - base;
    return (int64_t)(((uint64_t)__builtin_amdgcn_readlane(now.shi, i) << 32) | (uint32_t)__builtin_amdgcn_readlane(now.slo, i));
  }
  // bits of the tiles from this one on
  __device__ __forceinline__ uint32_t ok(int tile) const { return (uint32_t)(now.ok >> (tile - base)); }
};

// ONE: one tensor serves as keys and values, and is loaded once (512-element
// heads, whose tiles have one permutation for both reads).
template <int D, bool FP8, bool ONE>
__global__ __launch_bounds__(D == 512 ? 512 : 256, 2) void attn_tree_rows_kernel(DecodeArgs p) {
  constexpr int RG = 4, SPLIT = D == 512 ? 2 : 1;
  constexpr int BN = D >= 256 ? 32 : 64;     // keys per step
  constexpr int BM = 32 * RG, TH = 64 * RG * SPLIT;
  constexpr int NF = D / 16 / SPLIT;         // K fragments of a wave per 32 keys
  constexpr int ND = D / 32 / SPLIT;         // its column blocks of O
  constexpr int NK = BN / 32;                // 32-key tiles per step
  constexpr int C = D / 8;                   // 16-byte bf16 chunks per row
  constexpr int LD = BN * C / TH;            // chunks a thread stages per tensor
  constexpr int RS = TH / C;                 // rows between them
  constexpr int NG = D < 128 ? 1 : D / 128;
  constexpr int NT = ONE ? 1 : 2;
  constexpr int TB = BN * D * 2;             // bytes of one tile
  constexpr int X0 = 2 * NT * TB;
  constexpr int XB = SPLIT > 1 ? RG * SPLIT * NK * 4096 : 0;
  __shared__ __align__(16) char lds[X0 + XB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave = wv / SPLIT, part = wv % SPLIT;   // row group, slice of the columns
  const int col = lane & 31, hh = lane >> 5;

  // Workgroups go to the 8 XCDs in turn: those on the same keys stay together on one
  const uint32_t wg = p.first + blockIdx.x;
  const uint32_t per_xcd = (p.total + 7) / 8;
  const uint32_t at = (wg & 7) * per_xcd + (wg >> 3);
  if ((wg >> 3) >= per_xcd || at >= p.total) return;
  const int per_piece = p.hkv * p.rgroups;
  const int w = at / per_piece, rest = at - w * per_piece;
  const int h = rest / p.rgroups, rg = rest - h * p.rgroups;
  Cut cut;
  if (!find_cut(p, w, cut)) return;
  const Range rng = range_of<true>(p, entry(p.seq_lens, cut.b));

  const int row = rg * BM + wave * 32 + col;
  const bool row_live = row < p.rows;
  const int tok = row_live ? row / p.group : 0;
  const int head = row_live ? h * p.group + row - tok * p.group : 0;
  const int64_t qrow = (int64_t)cut.b * p.q_len + tok;
  const Seen seen = seen_of(p, rng, cut.b, tok, row_live);

  bf16x8 qf[NF];
#pragma unroll
  for (int j = 0; j < NF; ++j) {
    u32x4 x = {0, 0, 0, 0};
    if (seen.keeps)
      x = *reinterpret_cast<const u32x4*>(p.q + qrow * p.q_st + head * p.q_sh +
                                          16 * (part * NF + j) + 8 * hh);
    qf[j] = __builtin_bit_cast(bf16x8, x ^ p.q_flip);
  }
  f32x16 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m = kNoMax, l = 0.f, l2 = 0.f;   // two sums: shorter chains

  const int first = cut.tile << p.tile_shift;
  const int last = min(rng.end, first + (cut.tiles << p.tile_shift));
  const int steps = last > first ? (last - first + BN - 1) / BN : 0;
  WalkTiles<FP8> tiles(p, rng, cut.b, h, first >> 4);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;

  // Staging: chunk i of a thread lies in row r0 + RS i of the tile, whose wave's
  // rows are in one 16-key tile of the walk.  Its place in the row is permuted
  // on the global side, since the load writes LDS in lane order.
  const int r0 = D == 512 ? wv : tid / C;
  const int wr0 = D == 512 ? wv : wv * (64 / C);   // the wave's first row
  u32x2 reg[FP8 ? NT : 1][FP8 ? LD : 1];      // FP8: codes of a step on their way
  uint32_t rsc[FP8 ? NT : 1][FP8 ? LD : 1];   // and their scale bytes
  // whether every key of a step is there and kept by some row, in the context
  auto whole = [&](int at0) {
    bool all = true;
#pragma unroll
    for (int t = 0; t < NK; ++t) {
      const int base = rng.key_of(at0 + 32 * t);
      all = all && ((base >= seen.lo && base + 32 <= rng.ctx) || base + 32 <= seen.sinks);
    }
    constexpr uint32_t bits = (1u << (BN / 16)) - 1;
    return all && (tiles.ok(at0 >> 4) & bits) == bits;
  };
  const int c_once = tid % C;
  auto chunk = [&](int t, int r) {
    int c0 = c_once;
    if constexpr (D >= 256) asm volatile("" : "+v"(c0));   // no places kept over the loop
    return c0 ^ (t ? v_swz<D>(r) : k_swz<D>(r));
  };
  const int st = (int)p.st;
  auto fetch = [&](int buf, int at0) {
    tiles.advance(p, at0 >> 4);
    if (whole(at0)) {
#pragma unroll
      for (int i = 0; i < LD; ++i) {
        const int tile = (at0 + wr0 + RS * i) >> 4;     // of the wave's rows of this load
        const int64_t off = tiles.offset(tile);
        const int r = (r0 + RS * i) & 15;               // this lane's row of the 16
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const char* base = (t ? p.v : p.k) + off;
          const int c = chunk(t, r0 + RS * i);
          if constexpr (FP8) {
            reg[t][i] = *reinterpret_cast<const u32x2*>(base + (uint32_t)(r * st + 8 * c));
            rsc[t][i] = (t ? p.vs : p.ks)[tiles.scale_row(tile) * NG + (uint32_t)(r * NG + c / 16)];
          } else {
            load_lds16(lds0 + (2 * t + buf) * TB + wv * 1024 + i * TH * 16, base, (uint32_t)(r * st + 16 * c));
          }
        }
      }
      return;
    }
    // keys that no row keeps, and those of pages that are not there, are zeros
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const int place = at0 + ((wr0 + RS * i) & ~15), tile = place >> 4;
      const int64_t off = tiles.offset(tile);
      const int r = (r0 + RS * i) & 15;
      const bool read = (tiles.ok(tile) & 1) != 0 && any_keeps(seen, rng, rng.key_of(place) + r);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const char* base = (t ? p.v : p.k) + off;
        const int c = chunk(t, r0 + RS * i);
        if constexpr (FP8) {
          reg[t][i] = u32x2{0, 0};
          rsc[t][i] = 127;
          if (read) {
            reg[t][i] = *reinterpret_cast<const u32x2*>(base + (uint32_t)(r * st + 8 * c));
            rsc[t][i] = (t ? p.vs : p.ks)[tiles.scale_row(tile) * NG + (uint32_t)(r * NG + c / 16)];
          }
        } else {
          u32x4 x = {0, 0, 0, 0};
          if (read) x = *reinterpret_cast<const u32x4*>(base + (uint32_t)(r * st + 16 * c));
          *reinterpret_cast<u32x4*>(lds + (2 * t + buf) * TB + wv * 1024 + i * TH * 16 + lane * 16) = x;
        }
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
          *reinterpret_cast<u32x4*>(lds + (2 * t + buf) * TB + wv * 1024 + i * TH * 16 + lane * 16) =
              u32x4{a[0], a[1], b[0], b[1]};
        }
    }
  };

  // LDS places of this lane's first chunks: the permutation is an exclusive or,
  // so the other chunks' places are these with some bits flipped.
  constexpr int QK = NK * NF, PV = 2 * NK * ND, NE = 16 * NK;
  auto read_k = [&](int ka, int i) {   // operand of QK product i: tile i % NK, columns i / NK
    const int t = i % NK, c = 2 * (i / NK);
    return __builtin_bit_cast(
        bf16x8, *reinterpret_cast<const u32x4*>(lds + (ka ^ ((c & 15) * 16)) + (c & ~15) * 16 +
                                                part * NF * 32 + 32 * t * D * 2));
  };
  auto read_v = [&](int va, int i) {   // operand of PV product i: keys i / ND, columns i % ND
    const int ch = 4 * (i % ND);
    const int x = va ^ ((ch & 15) * 16);
    const char* v0 = lds + (ch & ~15) * 16 + part * ND * 64 + 16 * (i / ND) * D * 2;
    return read_tr(v0 + x, v0 + (x ^ (v_swz<D>(8) * 16)) + 8 * D * 2);
  };
  float* xs = reinterpret_cast<float*>(lds + X0);

  if (steps > 0) fetch(0, first);
  put(0);
#pragma unroll
  for (int j = 0; j < NF; ++j) arrived(__builtin_bit_cast(u32x4, qf[j]));
  step_barrier<0>();
  for (int it = 0; it < steps; ++it) {
    const int at0 = first + it * BN, buf = it & 1;
    const uint32_t ok = tiles.ok(at0 >> 4);   // before they move on
    bool inner = (ok & ((1u << (BN / 16)) - 1)) == (1u << (BN / 16)) - 1;
#pragma unroll
    for (int t = 0; t < NK; ++t) {
      const int base = rng.key_of(at0 + 32 * t);
      inner = inner && ((base >= seen.all_lo && base + 32 <= rng.ctx) || base + 32 <= seen.sinks);
    }
    if (it + 1 < steps) fetch(buf ^ 1, at0 + BN);
    int ka = buf * TB + k_at<D>(col, hh);
    int va = (ONE ? 0 : 2 * TB) + buf * TB +
             v_at<D>(4 * hh + ((lane & 15) >> 2), ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1)) +
             (lane & 1) * 8;
    asm volatile("" : "+v"(ka), "+v"(va));
    f32x16 sc[NK];
#pragma unroll
    for (int t = 0; t < NK; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) sc[t][i] = 0.f;
#pragma unroll
    for (int i = 0; i < QK; ++i)
      sc[i % NK] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(read_k(ka, i), qf[i / NK], sc[i % NK], 0, 0, 0);
    if constexpr (SPLIT == 2) {
#pragma unroll
      for (int t = 0; t < NK; ++t)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<f32x4*>(xs + ((wv * NK + t) * 4 + i / 4) * 256 + lane * 4) =
              f32x4{sc[t][i], sc[t][i + 1], sc[t][i + 2], sc[t][i + 3]};
      lds_barrier();
#pragma unroll
      for (int t = 0; t < NK; ++t)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const f32x4 y =
              *reinterpret_cast<const f32x4*>(xs + (((wv ^ 1) * NK + t) * 4 + i / 4) * 256 + lane * 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[t][i + e] += y[e];
        }
    }
    if (!inner) {
#pragma unroll
      for (int t = 0; t < NK; ++t) {
        const int base = rng.key_of(at0 + 32 * t) + 4 * hh;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const bool there = ok >> (2 * t + (i >> 3)) & 1;
          const bool kept = there & row_keeps(seen, rng, base + 8 * (i >> 2) + (i & 3));
          sc[t][i] = kept ? sc[t][i] : -INFINITY;
        }
      }
    }
    float mx[4];
#pragma unroll
    for (int i = 0; i < NE; ++i)
      mx[i % 4] = i < 4 ? sc[i / 16][i % 16] : fmaxf(mx[i % 4], sc[i / 16][i % 16]);
    const float top = halves_max(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]))) * p.scale2;
    if (__ballot(top > m + kLag)) {
      const float mn = fmaxf(m, top);
      const float a = exp2_fast(m - mn);
      m = mn;
      l *= a;
      l2 *= a;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= a;
    }
    u32x4 pw[2 * NK];
#pragma unroll
    for (int e = 0; e < NE; e += 2) {
      const float a = exp2_fast(fmaf(sc[e / 16][e % 16], p.scale2, -m));
      const float b = exp2_fast(fmaf(sc[e / 16][e % 16 + 1], p.scale2, -m));
      l += a;
      l2 += b;
      pw[e / 8][e / 2 % 4] = pack_bf16(a, b);
    }
#pragma unroll
    for (int i = 0; i < PV; ++i)
      o[i % ND] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          read_v(va, i), __builtin_bit_cast(bf16x8, pw[i / ND]), o[i % ND], 0, 0, 0);
    if (it + 1 < steps) put(buf ^ 1);
    step_barrier<0>();
  }

  l += l2;
  l += __shfl_xor(l, 32);
  if (cut.starts && h == 0 && rg == 0 && tid == 0) p.meta[cut.b] = make_int2(cut.slot, cut.splits);
  if (!row_live) return;
  if (!seen.keeps) {                          // a row without a place keeps nothing, whatever its q
    m = kNoMax;
    l = 0.f;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  }
  if (cut.splits == 1) {
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    uint16_t* dst = p.out + qrow * p.o_st + head * p.o_sh;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<u32x2*>(dst + 32 * (part * ND + d) + 2 * i + 4 * hh) =
            u32x2{pack_bf16(o[d][i] * inv, o[d][i + 1] * inv),
                  pack_bf16(o[d][i + 2] * inv, o[d][i + 3] * inv)};
    if (p.lse && hh == 0 && part == 0)
      p.lse[qrow * p.hq + head] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
  } else {
    const int64_t idx = ((int64_t)cut.slot * p.hkv + h) * p.rows + row;
    float* dst = p.part_o + idx * D;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<f32x4*>(dst + 32 * (part * ND + d) + 2 * i + 4 * hh) =
            f32x4{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
    if (hh == 0 && part == 0) {
      p.part_m[idx] = m;
      p.part_l[idx] = l;
    }
  }
}

// Joins the parts of sequences that are cut: a row per D / 4 lanes, parts one
// after another.  There are many rows and few parts, unlike in attn_decode's join (17.6 us where this takes
// 7.1, 26 nodes of 32 sequences).
template <int D>
__global__ __launch_bounds__(256) void attn_tree_join_kernel(DecodeArgs p) {
  constexpr int GL = D / 4, ROWS = 256 / GL;
  const uint32_t per_b = (uint32_t)(p.hkv * p.rows);
  const uint32_t groups = (per_b + ROWS - 1) / ROWS;
  const uint32_t wg = p.first + blockIdx.x;
  const uint32_t b = wg / groups;
  const int2 mt = p.meta[b];
  if (mt.y <= 1) return;
  const uint32_t hr = (wg - b * groups) * ROWS + threadIdx.x / GL;   // head and row
  if (hr >= per_b) return;
  const int gl = threadIdx.x % GL;
  const int64_t at0 = (int64_t)mt.x * per_b + hr;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  float l = 0.f, m = kNoMax;
#pragma unroll 4
  for (int i = 0; i < mt.y; ++i) {
    const int64_t at = at0 + (int64_t)i * per_b;
    const float mi = p.part_m[at], li = p.part_l[at];
    const f32x4 oi = *reinterpret_cast<const f32x4*>(p.part_o + at * D + gl * 4);
    const float mn = fmaxf(m, mi);
    const float a = exp2_fast(m - mn), c = exp2_fast(mi - mn);
    m = mn;
    l = l * a + li * c;
    o = o * a + oi * c;
  }
  o *= l == 0.f ? 0.f : 1.0f / l;
  const int h = hr / p.rows, row = hr - h * p.rows;
  const int tok = row / p.group, head = h * p.group + row - tok * p.group;
  const int64_t qrow = (int64_t)b * p.q_len + tok;
  *reinterpret_cast<u32x2*>(p.out + qrow * p.o_st + head * p.o_sh + gl * 4) =
      u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
  if (p.lse && gl == 0)
    p.lse[qrow * p.hq + head] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
}

}  // namespace

bool tree_rows_apply(const moe_attn_config& c) { return c.q_len * (c.heads_q / c.heads_kv) > 64; }

namespace {

// Workgroups that the GPU holds at once: two on a CU, of 512-element heads one.
int at_once(int dim) { return dim == 512 ? 256 : 512; }

struct TreePlan {
  int rows, rgroups;
  int64_t slots;       // parts of sequences at most; batch: none is cut
};
TreePlan tree_plan(const moe_attn_config& c) {
  TreePlan t;
  t.rows = c.q_len * (c.heads_q / c.heads_kv);
  t.rgroups = (t.rows + 127) / 128;
  t.slots = std::max<int64_t>(c.batch, at_once(c.head_dim) / ((int64_t)c.heads_kv * t.rgroups));
  return t;
}

}  // namespace

size_t tree_rows_ws_bytes(const moe_attn_config& c) {
  const TreePlan t = tree_plan(c);
  if (t.slots <= c.batch) return up256((size_t)c.batch * 8) + 256;
  const size_t rows = (size_t)t.slots * c.heads_kv * t.rows;
  return up256(rows * c.head_dim * 4) + 2 * up256(rows * 4) + up256((size_t)c.batch * 8);
}

hipError_t launch_tree_rows(const moe_attn_config& c, int sinks, const moe_rows& q,
                            const moe_kv_cache& kv, const int32_t* table, int table_width,
                            const int32_t* lens, const uint64_t* masks, const moe_rows& out,
                            float* lse, void* ws, hipStream_t st) {
  const TreePlan t = tree_plan(c);
  DecodeArgs a = decode_args(c, q, kv, table, table_width, lens, out, lse);
  a.masks = masks; a.sinks = sinks;
  a.rows = t.rows; a.rgroups = t.rgroups;
  a.q_flip = c.scale < 0.f ? 0x80008000u : 0u;
  a.scale2 = (c.scale < 0.f ? -c.scale : c.scale) * kLog2e;
  a.tile_shift = 6;
  char* w = static_cast<char*>(ws);
  const bool one = kv.k == kv.v && (kv.format != MOE_KV_FP8 || kv.k_scale == kv.v_scale);
  const bool f8 = kv.format == MOE_KV_FP8;
  const bool cut = t.slots > c.batch &&
                   !whole_sequences(longest_walk<true>(c, a) * c.head_dim * (f8 ? 1 : 2) * (one ? 1 : 2),
                                    (int64_t)c.batch * c.heads_kv * t.rgroups, true);
  if (cut) {
    const size_t rows = (size_t)t.slots * c.heads_kv * t.rows;
    a.part_o = reinterpret_cast<float*>(w); w += up256(rows * c.head_dim * 4);
    a.part_m = reinterpret_cast<float*>(w); w += up256(rows * 4);
    a.part_l = reinterpret_cast<float*>(w); w += up256(rows * 4);
  }
  a.meta = reinterpret_cast<int2*>(w);
  a.pieces = cut ? (int)t.slots : 0;
  const int64_t total = (cut ? t.slots : c.batch) * c.heads_kv * t.rgroups;
  a.total = (uint32_t)total;
#define MOE_TREE_ROWS(D, F, O)                                                                 \
  hipLaunchKernelGGL((attn_tree_rows_kernel<D, F, O>), grid, dim3(D == 512 ? 512 : 256), 0, st, a)
#define MOE_TREE(D)                                                                            \
  case D:                                                                                      \
    if (f8) { if (D == 512 && one) MOE_TREE_ROWS(D, true, D == 512); else MOE_TREE_ROWS(D, true, false); }   \
    else { if (D == 512 && one) MOE_TREE_ROWS(D, false, D == 512); else MOE_TREE_ROWS(D, false, false); }    \
    break;
  const hipError_t e = launch_workgroups((total + 7) / 8 * 8, [&](uint32_t first, dim3 grid) {
    a.first = first;
    switch (c.head_dim) { MOE_TREE(64) MOE_TREE(128) MOE_TREE(256) MOE_TREE(512) }
  });
#undef MOE_TREE
#undef MOE_TREE_ROWS
  if (e != hipSuccess || !cut) return e;
#define MOE_JOIN(D) \
  case D: hipLaunchKernelGGL((attn_tree_join_kernel<D>), grid, dim3(256), 0, st, a); break;
  const int64_t groups = ((int64_t)c.heads_kv * a.rows * (c.head_dim / 4) + 255) / 256;   // of a sequence
  return launch_workgroups(c.batch * groups, [&](uint32_t first, dim3 grid) {
    a.first = first;
    switch (c.head_dim) { MOE_JOIN(64) MOE_JOIN(128) MOE_JOIN(256) MOE_JOIN(512) }
  });
#undef MOE_JOIN
}

}  // namespace moe
