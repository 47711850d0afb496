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
//
// Which calls: more than 64 rows to a key-value head.  In a row (calls on one state, whose keys the caches
// partly hold), 32 sequences of 1000 to 4096 keys, 26 nodes, 32 heads of 128 on 8 take 94 us here and 149 in
// the kernel for few rows, 8 of 6000 to 8192 keys and 64 nodes 83 and 224 (FP8 83 and 303), 4 of 2000 to 4096,
// 40 nodes of 64 elements 25 and 49, 16 of 2000 to 4096, 16 nodes of 32 heads on one 512-element head 97 and 142.
//
// Bound by memory up to about 100 rows (the keys once: 32 sequences, 26 nodes 6.3 TB/s
// inside the loop), by the matrix units and what stands between their products
// beyond: among other calls 64 nodes of 8 sequences of 3000 to 8192, FP8 take 73 us (479 TFLOP/s), 16 nodes of
// 64 heads on one 512-element head, 16 sequences of 2048 to 4096 155 us (506 TFLOP/s).  (Figures of
// variants below are such cases in a row, both sides of one run.)  A part of a sequence costs a workgroup 9 us before its
// first step (its place in the work, pages, masks, first tiles: each waits for
// the one before) and 2 behind its last; the partial results, 100 MB in the last
// case, are joined in 9 to 18 us.
#include <type_traits>

#include "attn_decode_kernels.h"
#include "attn_tiles.h"

namespace moe {

namespace {

// The work of all sequences, laid end to end in tiles of 64 keys, is cut into
// equal pieces, one per workgroup (of a head and row group); nothing is cut
// where pieces is 0.  A sequence counts START tiles more than it has, before its
// first: what a part of a sequence costs next to its tiles (its rows of q,
// masks and first tiles, its partial result), so that a piece with the start of
// a sequence has as many tiles less.
struct Work {
  uint32_t per;            // length of a piece
  uint32_t at, end;        // of this one, and
  int w;                   // its number
  uint32_t begin;          // where sequence b begins, and
  int b, len;              // its number, p.seq_lens[b]
};
template <int START>
__device__ __forceinline__ bool find_work(const DecodeArgs& p, int w, Work& out) {
  const int lane = threadIdx.x & 63;
  out.w = w;
  if (p.pieces == 0) {
    out.w = 0;
    out.per = 1u << 30;
    out.at = out.begin = 0;
    out.b = w;
    out.len = entry(p.seq_lens, w);
    out.end = 1;           // the sequence alone
    return true;
  }
  uint32_t total = 0;      // the host has checked that it stays below 2^31
  int raw = 0, mine = 0, incl = 0;
  auto look = [&](int b0) {
    raw = b0 + lane < p.batch ? p.seq_lens[b0 + lane] : 0;
    mine = b0 + lane < p.batch ? range_of<true>(p, raw).tiles + START : 0;
    incl = wave_scan(mine);
  };
  for (int b0 = 0; b0 < p.batch; b0 += 64) {
    look(b0);
    total += __builtin_amdgcn_readlane(incl, 63);
  }
  out.per = __builtin_amdgcn_readfirstlane((total + p.pieces - 1) / p.pieces);
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
      out.begin = base + __builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(mine, l);
      return true;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}
// The piece's part of the sequence that `k` stands at, and k at the next one.
template <int START>
__device__ __forceinline__ Part next_part(const DecodeArgs& p, Work& k) {
  Part x;
  x.b = k.b;
  x.rng = range_of<true>(p, k.len);
  x.slot = k.w + k.b;      // every step along the work raises one of the two
  const uint32_t start = p.pieces ? k.begin + START : 0, past = start + x.rng.tiles;
  const uint32_t from = max(k.at, start), to = p.pieces ? min(k.end, past) : past;
  x.splits = __builtin_amdgcn_readfirstlane((int)((past - 1) / k.per - start / k.per) + 1);
  x.starts = from == start && from < to;
  x.first = (int)(from - start) << p.tile_shift;
  x.last = from < to ? (int)min((int64_t)max(x.rng.end, 0), (int64_t)(to - start) << p.tile_shift) : -1;
  k.begin = past;
  k.at = past;
  ++k.b;
  if (k.at < k.end) k.len = entry(p.seq_lens, k.b);
  return x;
}

// The kernel's arguments, loaded where they are asked for: held from the kernel's start
// they would be most of the scalar registers, and the loop's own would not find a place.
typedef const __attribute__((address_space(4))) DecodeArgs* Args;
__device__ __forceinline__ Args arguments() {
  Args a = (Args)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(a));
  return a;
}

// Where 16-key tiles of the walk lie, 64 of them, a tile per lane, and the pages of the
// next 64: a step takes its tiles' places from lanes.
template <bool FP8>
struct WalkTiles {
  Range rng;
  int b, h, base;
  int next;                // page, -1: none
  uint32_t lo, hi;         // byte offset of the tile's first row in k and v
  uint32_t slo, shi;       // FP8: its row among the scales
  uint64_t there;          // tiles whose page is
  __device__ __forceinline__ int64_t key_of_lane(int tile) const {
    const int64_t key = 16 * ((int64_t)tile + (threadIdx.x & 63));
    return key >= rng.front ? key + rng.gap : key;
  }
  __device__ __forceinline__ int page(Args p, int tile) const {
    const int64_t key = key_of_lane(tile);
    if (key >= rng.len) return -1;
    const int id = (p->table + (int64_t)b * p->table_width)[key >> p->page_shift];
    return id >= 0 && id < p->pages ? id : -1;
  }
  __device__ __forceinline__ void place(Args p, int id) {
    const int in_page = (int)(key_of_lane(base) & ((1 << p->page_shift) - 1));
    const int64_t at = max(id, 0);
    const int64_t off = at * p->sp + h * p->sh + in_page * p->st;
    lo = (uint32_t)off;
    hi = (uint32_t)(off >> 32);
    if constexpr (FP8) {
      const int64_t srow = ((at * p->hkv + h) << p->page_shift) + in_page;
      slo = (uint32_t)srow;
      shi = (uint32_t)(srow >> 32);
    }
    there = __ballot(id >= 0);
  }
  __device__ __forceinline__ WalkTiles(const Range& r, int seq, int head, int tile)
      : rng(r), b(seq), h(head), base(tile) {
    const Args p = arguments();
    const int id = page(p, base);
    next = page(p, base + 64);
    place(p, id);
  }
  // steps are asked for in order, and none lies in two groups
  __device__ __forceinline__ void advance(int tile) {
    if (tile < base + 64) return;
    const Args p = arguments();
    base += 64;
    place(p, next);
    next = page(p, base + 64);
  }
  __device__ __forceinline__ static int64_t lane_of(uint32_t hi, uint32_t lo, int i) {
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane(hi, i) << 32 |
                     (uint32_t)__builtin_amdgcn_readlane(lo, i));
  }
};

// Where a wave's loads of a step lie, the same for all lanes: N of the step's
// TILES 16-key tiles, every TILES / N th from tile `sub` on.
template <int TILES, int N, bool FP8>
struct Place {
  int64_t off[N];        // bytes of the tile's first row in k and v
  int64_t srow[N];       // FP8: its row among the scales
  uint32_t ok;           // tiles of the step whose page is there
  __device__ __forceinline__ void find(WalkTiles<FP8>& tiles, int at0, int sub) {
    tiles.advance(at0 >> 4);
    const int t0 = (at0 >> 4) - tiles.base;
    ok = (uint32_t)(tiles.there >> t0) & ((1u << TILES) - 1);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int tile = t0 + TILES / N * i + sub;
      off[i] = tiles.lane_of(tiles.hi, tiles.lo, tile);
      if constexpr (FP8) srow[i] = tiles.lane_of(tiles.shi, tiles.slo, tile);
    }
  }
};

// ONE: one tensor serves as keys and values, and is loaded once (512-element
// heads, whose tiles have one permutation for both reads).
template <int D, bool FP8, bool ONE, int RG>
__global__ __launch_bounds__(64 * RG * (D == 512 ? 2 : 1), 2) void attn_tree_rows_kernel(DecodeArgs p) {
  constexpr int SPLIT = D == 512 ? 2 : 1;
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
  // tiles of K (and of V); steps that are asked for ahead of the one that is
  // computed: bf16 into LDS, as many as two workgroups on a CU have room for, FP8 into registers.
  // (32 keys a step and five tiles take as long as 64 and two.  512-element heads two steps ahead
  // spilled 30 registers: 202 us instead of 168 at 16 nodes of 64 heads.)
  constexpr int KB = ONE ? 3 : FP8 || SPLIT == 2 ? 2 : 2 * (RG / 4) * (D == 64 ? 2 : 1);
  constexpr int DIST = SPLIT == 2 ? 1 : !FP8 ? KB - 1 : D < 256 ? 2 : 1;
  constexpr int SETS = FP8 ? DIST : 1;
  constexpr int TB = BN * D * 2;             // bytes of one tile
  constexpr int V0 = ONE ? 0 : KB * TB;      // the tiles of V
  constexpr int X0 = (ONE ? KB : 2 * KB) * TB;   // the waves' parts of S
  constexpr int XB = SPLIT > 1 ? RG * SPLIT * NK * 4096 : 0;
  constexpr uint32_t ALL = (1u << (BN / 16)) - 1;
  static_assert(!ONE || SPLIT == 2, "ONE: 512-element heads");
  __shared__ __align__(16) char lds[X0 + XB];
  const int tid = threadIdx.x;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave = wv / SPLIT, part = wv % SPLIT;   // row group, slice of the columns
  // Large heads work what depends on the lane out anew each time, from the one
  // register that holds it: kept over the loop it would take ones that they do not have.
  const int lane_once = tid & 63;
  auto here = [&]() {
    int x = lane_once;
    if constexpr (D >= 256) asm volatile("" : "+v"(x));
    return x;
  };

  // Workgroups go to the 8 XCDs in turn: those on the same keys stay together on one
  const uint32_t wg = p.first + blockIdx.x;
  const uint32_t per_xcd = (p.total + 7) / 8;
  const uint32_t at = (wg & 7) * per_xcd + (wg >> 3);
  if ((wg >> 3) >= per_xcd || at >= p.total) return;
  const int per_piece = p.hkv * p.rgroups;
  const int w = __builtin_amdgcn_readfirstlane(at / per_piece), rest = at - w * per_piece;
  const int h = __builtin_amdgcn_readfirstlane(rest / p.rgroups);
  const int rg = __builtin_amdgcn_readfirstlane(rest - h * p.rgroups);
  Work work;
  // 13 us where a tile takes 2.6, 11 where it takes 5; 3 and 8 tiles were slower by 1 to 3%
  constexpr int START = D == 512 ? 2 : 5;
  if (!find_work<START>(p, w, work)) return;

  // this lane's row: whether it is one, its token and head
  struct Row {
    bool live;
    int tok, head;
  };
  auto my_row = [&](Args a) {
    const int row = rg * BM + wave * 32 + (here() & 31);
    Row r;
    r.live = row < a->rows;
    r.tok = r.live ? row / a->group : 0;
    r.head = r.live ? h * a->group + row - r.tok * a->group : 0;
    return r;
  };
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  const int st = (int)p.st;
  // Staging: chunk i of a thread lies in row r0 + RS i of the tile, whose wave's
  // rows are in one 16-key tile of the walk.  Its place in the row is permuted
  // on the global side, since the load writes LDS in lane order.
  constexpr int WR = 64 / C;                  // rows of a wave's load
  auto row_of = [&](int i) { return wv * WR + (int)((here() & 63u) / C) + RS * i; };
  auto chunk = [&](int t, int r) {
    return (int)((here() & 63u) % C) ^ (t ? v_swz<D>(r) : k_swz<D>(r));
  };

  while (work.at < work.end) {
  const Part pt = next_part<START>(p, work);
  if (pt.last < 0) continue;                  // nothing but what a start counts
  Range rng = pt.rng;                         // the same in all lanes, and in scalar registers
  for (int* x : {&rng.lo, &rng.len, &rng.tiles, &rng.ctx, &rng.front, &rng.gap, &rng.end})
    *x = __builtin_amdgcn_readfirstlane(*x);
  const int first = __builtin_amdgcn_readfirstlane(pt.first);
  const int last = __builtin_amdgcn_readfirstlane(pt.last);
  const int steps = last > first ? (last - first + BN - 1) / BN : 0;
  WalkTiles<FP8> tiles(rng, pt.b, h, first >> 4);

  bf16x8 qf[NF];
  int my_tok;
  bool my_live;
  {
    const Args a = arguments();
    const Row r = my_row(a);
    my_tok = r.tok;
    my_live = r.live;
    const uint16_t* q = a->q + ((int64_t)pt.b * a->q_len + r.tok) * a->q_st + r.head * a->q_sh;
    const uint32_t flip = a->q_flip;
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      u32x4 x = {0, 0, 0, 0};
      if (r.live) x = *reinterpret_cast<const u32x4*>(q + 16 * (part * NF + j) + 8 * (here() >> 5));
      qf[j] = __builtin_bit_cast(bf16x8, x ^ flip);
    }
  }
  f32x16 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m = kNoMax, l = 0.f, l2 = 0.f;   // two sums: shorter chains

  // A load of all waves takes RS rows: NP of the step's 16-key tiles, every SKIPth, are
  // this wave's, and LPT loads go to each.
  constexpr int TILES = BN / 16, SKIP = RS > 16 ? RS / 16 : 1, NP = TILES / SKIP, LPT = LD / NP;
  typedef Place<TILES, NP, FP8> StepPlace;
  const int sub = wv * WR / 16;
  Seen seen = seen_of(p, rng, pt.b, my_tok, my_live);
  seen.row_sinks = seen.sinks;                // rows that keep nothing are set to zero at the end

  u32x2 codes[SETS][FP8 ? NT : 1][FP8 ? LD : 1];      // FP8: on their way
  uint32_t scale[SETS][FP8 ? NT : 1][FP8 ? LD : 1];   // and their scale bytes
  // places of the walk whose keys are all kept: [0, head) and [tail, end), by 32s
  const int head_end = seen.sinks & ~31, tail_end = (rng.ctx & ~31) - rng.gap;
  auto tail_of = [&](int lo) { return (int)min((int64_t)lo + 31, (int64_t)INT_MAX - 31) / 32 * 32 - rng.gap; };
  const int any_tail = tail_of(seen.lo), all_tail = tail_of(seen.all_lo);
  auto covers = [&](int at0, int tail) {
    return (at0 >= tail && at0 + BN <= tail_end) || at0 + BN <= head_end;
  };
  // asks for a step's tile of tensor t (0: K, 1: V); whether it is on its way into LDS
  auto fetch = [&](int t, int buf, int at0, const StepPlace& pl, int set) __attribute__((always_inline)) {
    const char* data = t ? p.v : p.k;
    const uint8_t* scales = t ? p.vs : p.ks;
    auto& reg = codes[set];
    auto& rsc = scale[set];
    const int to = (t ? V0 : 0) + buf * TB + wv * 1024;
    const bool whole = pl.ok == ALL && covers(at0, any_tail);
    if (!FP8 && whole) {
#pragma unroll
      for (int i = 0; i < LD; ++i) {
        const int r = row_of(i);
        load_lds16(lds0 + to + i * TH * 16, data + pl.off[i / LPT],
                   (uint32_t)((r & 15) * st + 16 * chunk(t, r)));
      }
      return true;
    }
    // keys that no row keeps, and those of pages that are not there, are zeros
#pragma unroll D == 512 && !FP8 ? 1 : LD
    for (int i = 0; i < LD; ++i) {
      const int r = row_of(i), c = chunk(t, r);
      const char* base = data + pl.off[i / LPT];
      const int tile = TILES / NP * (i / LPT) + sub;
      const bool read = whole || ((pl.ok >> tile & 1) != 0 &&
                                  any_keeps(seen, rng, rng.key_of(at0 + 16 * tile) + (r & 15)));
      if constexpr (FP8) {
        const int64_t sr = pl.srow[i / LPT];
        reg[t][i] = u32x2{0, 0};
        rsc[t][i] = 127;
        if (read) {
          reg[t][i] = *reinterpret_cast<const u32x2*>(base + (uint32_t)((r & 15) * st + 8 * c));
          rsc[t][i] = scales[sr * NG + (uint32_t)((r & 15) * NG + c / 16)];
        }
      } else {
        u32x4 x = {0, 0, 0, 0};
        if (read) x = *reinterpret_cast<const u32x4*>(base + (uint32_t)((r & 15) * st + 16 * c));
        *reinterpret_cast<u32x4*>(lds + to + i * TH * 16 + here() * 16) = x;
      }
    }
    return false;
  };
  auto put = [&](int t, int buf, int set) __attribute__((always_inline)) {   // FP8: codes as bf16 into LDS
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < LD; ++i) {
        const float s = scale_of(scale[set][t][i]);
        const u32x2 a = fp8x4_to_bf16(codes[set][t][i][0], s), b = fp8x4_to_bf16(codes[set][t][i][1], s);
        *reinterpret_cast<u32x4*>(lds + (t ? V0 : 0) + buf * TB + wv * 1024 + i * TH * 16 + here() * 16) =
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
  auto k_lane = [&]() {
    const int x = here();
    return k_at<D>(x & 31, x >> 5);
  };
  auto v_lane = [&]() {
    const int x = here();
    return v_at<D>(4 * (x >> 5) + ((x & 15) >> 2), ((x >> 4) & 1) * 2 + ((x & 3) >> 1)) + (x & 1) * 8;
  };
  // masks a step's scores; `ok`: which of its 16-key tiles are there
  auto mask = [&](f32x16(&sc)[NK], int at0, uint32_t ok) {
    if ((ok & ALL) == ALL && covers(at0, all_tail)) return;
#pragma unroll
    for (int t = 0; t < NK; ++t) {
      const int base = rng.key_of(at0 + 32 * t) + 4 * (here() >> 5);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const bool there = ok >> (2 * t + (i >> 3)) & 1;
        const bool kept = there & row_keeps(seen, rng, base + 8 * (i >> 2) + (i & 3));
        sc[t][i] = kept ? sc[t][i] : -INFINITY;
      }
    }
  };
  u32x4 pw[2 * NK];
  // the maximum and the weights of a step's scores
  auto weigh = [&](f32x16(&sc)[NK]) {
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
#pragma unroll
    for (int e = 0; e < NE; e += 2) {
      const float a = exp2_fast(fmaf(sc[e / 16][e % 16], p.scale2, -m));
      const float b = exp2_fast(fmaf(sc[e / 16][e % 16 + 1], p.scale2, -m));
      l += a;
      l2 += b;
      pw[e / 8][e / 2 % 4] = pack_bf16(a, b);
    }
  };
  auto q_arrived = [&]() {
#pragma unroll
    for (int j = 0; j < NF; ++j) arrived(__builtin_bit_cast(u32x4, qf[j]));
  };

  if constexpr (SPLIT == 1) {
    // Bits of the steps from the one that is computed on: tiles whose page is there, and steps that
    // are wholly on their way into LDS.
    uint32_t there = 0, on_way = 0;
    StepPlace pl;
    auto ask = [&](int ahead, int buf, int at0, int set) __attribute__((always_inline)) {
      pl.find(tiles, at0, sub);
      there |= pl.ok << (TILES * ahead);
      const bool k = fetch(0, buf, at0, pl, set), v = fetch(1, buf, at0, pl, set);
      on_way |= (uint32_t)(k && v) << ahead;
    };
#pragma unroll
    for (int i = 0; i < DIST; ++i)
      if (i < steps) ask(i, FP8 ? 0 : i, first + i * BN, FP8 ? i : 0);
    if (steps > 0) {
      put(0, 0, 0);
      put(1, 0, 0);
    }
    q_arrived();
    step_barrier<0>();
    int buf = 0, free = KB - 1;               // the tile that is read, and that of the step before it
    // FP8's eight groups with up to 128 rows: waves without rows keep out of the others' way (26 nodes
    // of 32 sequences, 104 rows of 128 elements: 93 us, with their products 117)
    const bool busy = !FP8 || rg * BM + wave * 32 < p.rows;
    auto step = [&](int it, int set) __attribute__((always_inline)) {
      const int at0 = first + it * BN;
      if (it + DIST < steps) ask(DIST, free, at0 + DIST * BN, set);
      if (busy) {
      int ka = buf * TB + k_lane(), va = V0 + buf * TB + v_lane();
      asm volatile("" : "+v"(ka), "+v"(va));
      f32x16 sc[NK];
#pragma unroll
      for (int t = 0; t < NK; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) sc[t][i] = 0.f;
      // LDS reads run AHEAD products before their use, in an order fixed by hand; products go
      // before the SIMD's other wave's weights (64 nodes of 8 sequences, FP8 67 us, without 69)
      constexpr int AHEAD = D == 256 ? 2 : 4;
      auto read = [&](int i) { return i < QK ? read_k(ka, i) : read_v(va, i - QK); };
      bf16x8 f[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) f[i] = read(i);
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int i = 0; i < QK; ++i) {
        sc[i % NK] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i % AHEAD], qf[i / NK], sc[i % NK], 0, 0, 0);
        f[i % AHEAD] = read(i + AHEAD);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
      mask(sc, at0, there);
      weigh(sc);
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int i = 0; i < PV; ++i) {
        o[i % ND] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            f[(QK + i) % AHEAD], __builtin_bit_cast(bf16x8, pw[i / ND]), o[i % ND], 0, 0, 0);
        if (i + AHEAD < PV) f[(QK + i) % AHEAD] = read(QK + i + AHEAD);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
      }
      if (it + 1 < steps) {
        put(0, buf ^ 1, (set + 1) % SETS);
        put(1, buf ^ 1, (set + 1) % SETS);
      }
      free = buf;
      buf = buf + 1 == KB ? 0 : buf + 1;
      there >>= TILES;
      on_way >>= 1;
      // the next step's tiles are there, those of the steps after it may be on their way
      constexpr uint32_t LATER = ((1u << DIST) - 1) & ~1u;
      if (!FP8 && DIST > 1 && (on_way & LATER) == LATER) step_barrier<(DIST - 1) * 2 * LD>();
      else step_barrier<0>();
    };
    if constexpr (SETS > 1) {
      for (int it = 0; it < steps; it += SETS)
#pragma unroll
        for (int j = 0; j < SETS; ++j)
          if (it + j < steps) step(it + j, j);
    } else {
      for (int it = 0; it < steps; ++it) step(it, 0);
    }
  } else {
    // As in attn_prefill_kernel.h: half of a step is matrix products (its
    // scores, and with V of the step before), half vector instructions.  The
    // second four waves, which share the SIMDs of the first, are half a step
    // late, so that products run beside weights.  Tiles of K take turns in kb,
    // kb_next .., the tile of V is vb; with ONE that is K's of the step before.
    constexpr int AHEAD = ONE && !FP8 ? 3 : 2;   // 3 is what the registers hold; 164 us and 168 with 2
    float* xs = reinterpret_cast<float*>(lds + X0);
    f32x16 sc[NK];
    int kb = 0, vb = 0;   // tiles of K and V that are read
    StepPlace pl;         // of the step whose K was asked for last
    pl.ok = 0;
    if (steps > 0) {
      pl.find(tiles, first, sub);
      fetch(0, 0, first, pl, 0);
      put(0, 0, 0);
    }
    q_arrived();
    step_barrier<0>();
    uint32_t ok_before = 0, ok = pl.ok;
    auto products = [&](auto begins) __attribute__((always_inline)) {
      constexpr bool LAG = !decltype(begins)::value;
      int ka = kb * TB + k_lane(), va = V0 + vb * TB + v_lane();
      asm volatile("" : "+v"(ka), "+v"(va));
      auto read = [&](int i) { return i < QK ? read_k(ka, i) : read_v(va, i - QK); };
      constexpr int N = LAG ? QK + PV : QK;
      // before the weights of the SIMD's other wave: 16 nodes of 64 heads on one head 151 us, without 164
      __builtin_amdgcn_s_setprio(1);
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
      const int at4 = here() * 4;
#pragma unroll
      for (int t = 0; t < NK; ++t)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<f32x4*>(xs + ((wv * NK + t) * 4 + i / 4) * 256 + at4) =
              f32x4{sc[t][i], sc[t][i + 1], sc[t][i + 2], sc[t][i + 3]};
#pragma unroll
      for (int i = QK; i < N; ++i) {
        o[(i - QK) % ND] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            f[i % AHEAD], __builtin_bit_cast(bf16x8, pw[(i - QK) / ND]), o[(i - QK) % ND], 0, 0, 0);
        if (i + AHEAD < N) f[i % AHEAD] = read(i + AHEAD);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
    };
    auto weights = [&](int at0, uint32_t there) __attribute__((always_inline)) {
      const int at4 = here() * 4;
#pragma unroll
      for (int t = 0; t < NK; ++t)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const f32x4 y =
              *reinterpret_cast<const f32x4*>(xs + (((wv ^ 1) * NK + t) * 4 + i / 4) * 256 + at4);
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[t][i + e] += y[e];
        }
      mask(sc, at0, there);
      weigh(sc);
    };
    // one step of early or late waves: both pass the same two barriers
    auto step = [&](int it, auto begins, auto late) __attribute__((always_inline)) {
      constexpr bool LATE = decltype(late)::value;
      const int at0 = first + it * BN;
      const int kb_next = kb + 1 == KB ? 0 : kb + 1;
      const int vb_next = ONE ? kb : vb ^ 1;
      const bool more = it + 1 < steps;
      auto load = [&]() __attribute__((always_inline)) {
        if constexpr (!ONE) fetch(1, vb_next, at0, pl, 0);
        if (more) {
          pl.find(tiles, at0 + BN, sub);
          fetch(0, kb_next, at0 + BN, pl, 0);
        }
      };
      auto store = [&]() __attribute__((always_inline)) {
        if (more) put(0, kb_next, 0);
        if constexpr (!ONE) put(1, vb_next, 0);
      };
      // FP8 codes are on their way beside the weights alone: a register that the products had to
      // take back from memory would wait for them
      if constexpr (!FP8 || LATE) load();
      if constexpr (!LATE) products(begins);
      else if constexpr (!decltype(begins)::value) weights(at0 - BN, ok_before);
      if constexpr (LATE) store();
      lds_barrier();
      if constexpr (FP8 && !LATE) load();
      if constexpr (LATE) products(begins); else weights(at0, ok);
      if constexpr (!LATE) store();
      kb = kb_next;
      vb = vb_next;
      ok_before = ok;
      ok = pl.ok;
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
        weights(first + (steps - 1) * BN, ok_before);
      }
      const int va = V0 + vb * TB + v_lane();
#pragma unroll
      for (int i = 0; i < PV; ++i)
        o[i % ND] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            read_v(va, i), __builtin_bit_cast(bf16x8, pw[i / ND]), o[i % ND], 0, 0, 0);
    }
    lds_barrier();                            // all have read the last tiles
  }

  l += l2;
  l += __shfl_xor(l, 32);
  const Args a = arguments();
  const Row r = my_row(a);
  const int hh = here() >> 5;
  if (pt.starts && h == 0 && rg == 0 && tid == 0) a->meta[pt.b] = make_int2(pt.slot, pt.splits);
  if (rg * BM + wave * 32 >= a->rows) continue;   // no row of the wave is one
  if (seen.row_lo == INT_MAX) {               // a row without a place keeps nothing, whatever its q
    m = kNoMax;
    l = 0.f;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  }
  if (pt.splits == 1) {
    if (!r.live) continue;
    const int64_t qrow = (int64_t)pt.b * a->q_len + r.tok;
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    uint16_t* dst = a->out + qrow * a->o_st + r.head * a->o_sh;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<u32x2*>(dst + 32 * (part * ND + d) + 2 * i + 4 * hh) =
            u32x2{pack_bf16(o[d][i] * inv, o[d][i + 1] * inv),
                  pack_bf16(o[d][i + 2] * inv, o[d][i + 3] * inv)};
    if (a->lse && hh == 0 && part == 0)
      a->lse[qrow * a->hq + r.head] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
  } else {
    // in the order of the registers, so that a wave stores whole lines: groups of 32 rows, quads of
    // columns, (lane / 32, row)
    const int64_t group = ((int64_t)pt.slot * a->hkv + h) * a->rgroups * RG + rg * RG + wave;
    f32x4* dst = reinterpret_cast<f32x4*>(a->part_o) + group * (8 * D) + here();
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        dst[64 * (4 * (part * ND + d) + i / 4)] = f32x4{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
    if (hh == 0 && part == 0) {
      a->part_m[group * 32 + here()] = m;
      a->part_l[group * 32 + here()] = l;
    }
  }
  }
}

// Joins the parts of sequences that are cut.  A workgroup takes 32 rows and 64 columns:
// a lane has a row's quads as the parts hold them, and the rows go out through LDS.
template <int D>
__global__ __launch_bounds__(256) void attn_tree_join_kernel(DecodeArgs p) {
  constexpr int COLS = 64, SLICES = D / COLS;
  __shared__ u32x2 rows[32][COLS / 4 + 1];
  const int groups = (p.rows + 31) / 32, held = p.rgroups * p.row_groups;   // held: with those that are no rows
  const uint32_t wg = p.first + blockIdx.x;
  const int slice = wg % SLICES;
  const uint32_t rest = wg / SLICES;
  const uint32_t bh = rest / groups;
  const int group = rest - bh * groups;
  const int b = bh / p.hkv, h = bh - b * p.hkv;
  const int2 mt = p.meta[b];
  if (mt.y <= 1) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t g0 = ((int64_t)mt.x * p.hkv + h) * held + group, step = (int64_t)p.hkv * held;
  // two quads a lane: wave, and wave + 4, of the slice's 8 pairs of 4 columns
  const f32x4* src = reinterpret_cast<const f32x4*>(p.part_o) + g0 * (8 * D) + 64 * (8 * slice + wave) + lane;
  f32x4 o[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  float l = 0.f, m = kNoMax;
#pragma unroll 4
  for (int i = 0; i < mt.y; ++i) {
    const int64_t at = (g0 + i * step) * 32 + (lane & 31);
    const float mi = p.part_m[at], li = p.part_l[at];
    const f32x4 x = src[i * step * (8 * D)], y = src[i * step * (8 * D) + 64 * 4];
    const float mn = fmaxf(m, mi);
    const float a = exp2_fast(m - mn), c = exp2_fast(mi - mn);
    m = mn;
    l = l * a + li * c;
    o[0] = o[0] * a + x * c;
    o[1] = o[1] * a + y * c;
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    o[i] *= inv;
    rows[lane & 31][2 * (wave + 4 * i) + (lane >> 5)] =
        u32x2{pack_bf16(o[i][0], o[i][1]), pack_bf16(o[i][2], o[i][3])};
  }
  auto place = [&](int r, int& tok, int& head) {
    const int row = group * 32 + r;
    tok = row / p.group;
    head = h * p.group + row - tok * p.group;
    return row < p.rows;
  };
  int tok, head;
  if (p.lse && slice == 0 && threadIdx.x < 32 && place(lane, tok, head))
    p.lse[((int64_t)b * p.q_len + tok) * p.hq + head] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
  __syncthreads();
  const int r = threadIdx.x / 8, c = threadIdx.x % 8;    // 16 bytes of a row
  if (!place(r, tok, head)) return;
  const u32x2 x = rows[r][2 * c], y = rows[r][2 * c + 1];
  *reinterpret_cast<u32x4*>(p.out + ((int64_t)b * p.q_len + tok) * p.o_st + head * p.o_sh +
                            COLS * slice + 8 * c) = u32x4{x[0], x[1], y[0], y[1]};
}

}  // namespace

bool tree_rows_apply(const moe_attn_config& c) { return c.q_len * (c.heads_q / c.heads_kv) > 64; }

namespace {

// The work of all sequences, end to end, is cut into equal pieces, so that one
// round of workgroups takes them.  With four rounds of whole sequences nothing is
// cut: workgroups that end early take the next ones (288 sequences of 200 to 2048 keys
// on 8 heads of 128: 317 us, cut 322).
//
// Eight groups of 32 rows in a workgroup read keys once where four would read them twice and
// turn FP8 into bf16 twice: 64 nodes of 12 sequences of 3000 to 6000, 4 heads on each of 8, 128 elements
// 85 us (bf16 90) and 95 with four (95), 64 elements 61 (62) and 67 (63).  Up to 128 rows four hold
// them all, but with 256 elements in FP8 a thread of four groups holds twice the codes of one
// of eight and spills them: 32 nodes of 16 sequences 174 us with eight groups, 337 with four (bf16 182 and 157).
// FP8 heads of 64 and 128 elements take eight too: a memory fault was reported the first time that four groups
// ran on FP8 heads of 64.  Executed on the CPU, the code of that kernel stays in bounds, waits for all it
// reads and gives the right numbers, so that the fault has no explanation, and the kernel is not there any more.
// With up to 128 rows half of the waves then have none, and load and convert only: 26 nodes of 32 sequences,
// 104 rows of 128 elements 93 us (bf16, four groups 95).
struct TreePlan {
  int rows, rg, rgroups, pieces;   // rg: groups of 32 rows in a workgroup
  int64_t slots;
};
TreePlan tree_plan(const moe_attn_config& c, bool f8) {
  TreePlan t;
  t.rows = c.q_len * (c.heads_q / c.heads_kv);
  t.rg = c.head_dim < 512 && (t.rows > 128 || f8) ? 8 : 4;
  t.rgroups = (t.rows + 32 * t.rg - 1) / (32 * t.rg);
  const int64_t per = (int64_t)c.heads_kv * t.rgroups;
  // workgroups that the GPU holds at once: two on a CU, of eight waves one
  const int at_once = t.rg == 8 || c.head_dim == 512 ? 256 : 512;
  t.pieces = c.batch * per >= 4 * at_once ? 0 : (int)std::max<int64_t>(1, at_once / per);
  t.slots = (int64_t)t.pieces + c.batch;
  return t;
}

}  // namespace

size_t tree_rows_ws_bytes(const moe_attn_config& c) {
  size_t rows = 0;                 // of the caches' types the one that takes more
  for (bool f8 : {false, true}) {
    const TreePlan t = tree_plan(c, f8);
    if (t.pieces) rows = std::max(rows, (size_t)t.slots * c.heads_kv * t.rgroups * t.rg * 32);
  }
  return up256(rows * c.head_dim * 4) + 2 * up256(rows * 4) + up256((size_t)c.batch * 8) + 256;
}

hipError_t launch_tree_rows(const moe_attn_config& c, int sinks, const moe_rows& q,
                            const moe_kv_cache& kv, const int32_t* table, int table_width,
                            const int32_t* lens, const uint64_t* masks, const moe_rows& out,
                            float* lse, void* ws, hipStream_t st) {
  const bool one = kv.k == kv.v && (kv.format != MOE_KV_FP8 || kv.k_scale == kv.v_scale);
  const bool f8 = kv.format == MOE_KV_FP8;
  const TreePlan t = tree_plan(c, f8);
  DecodeArgs a = decode_args(c, q, kv, table, table_width, lens, out, lse);
  a.masks = masks; a.sinks = sinks;
  a.rows = t.rows; a.rgroups = t.rgroups; a.row_groups = t.rg;
  a.q_flip = c.scale < 0.f ? 0x80008000u : 0u;
  a.scale2 = (c.scale < 0.f ? -c.scale : c.scale) * kLog2e;
  a.tile_shift = 6;
  char* w = static_cast<char*>(ws);
  const bool cut = t.pieces > 0 &&
                   !whole_sequences(longest_walk<true>(c, a) * c.head_dim * (f8 ? 1 : 2) * (one ? 1 : 2),
                                    (int64_t)c.batch * c.heads_kv * t.rgroups, true);
  if (cut) {
    const size_t rows = (size_t)t.slots * c.heads_kv * t.rgroups * t.rg * 32;
    a.part_o = reinterpret_cast<float*>(w); w += up256(rows * c.head_dim * 4);
    a.part_m = reinterpret_cast<float*>(w); w += up256(rows * 4);
    a.part_l = reinterpret_cast<float*>(w); w += up256(rows * 4);
  }
  a.meta = reinterpret_cast<int2*>(w);
  a.pieces = cut ? t.pieces : 0;
  const int64_t total = (int64_t)(cut ? t.pieces : c.batch) * c.heads_kv * t.rgroups;
  a.total = (uint32_t)total;
#define MOE_TREE_ROWS(D, F, O, G)                                                              \
  hipLaunchKernelGGL((attn_tree_rows_kernel<D, F, O, G>), grid, dim3(64 * G * (D == 512 ? 2 : 1)), 0, st, a)
#define MOE_TREE(D)                                                                            \
  case D:                                                                                      \
    if (f8) MOE_TREE_ROWS(D, true, false, 8);                                                  \
    else if (t.rg == 8) MOE_TREE_ROWS(D, false, false, 8);                                     \
    else MOE_TREE_ROWS(D, false, false, 4);                                                    \
    break;
  const hipError_t e = launch_workgroups((total + 7) / 8 * 8, [&](uint32_t first, dim3 grid) {
    a.first = first;
    switch (c.head_dim) {
      MOE_TREE(64) MOE_TREE(128) MOE_TREE(256)
      case 512:
        if (f8) { if (one) MOE_TREE_ROWS(512, true, true, 4); else MOE_TREE_ROWS(512, true, false, 4); }
        else { if (one) MOE_TREE_ROWS(512, false, true, 4); else MOE_TREE_ROWS(512, false, false, 4); }
        break;
    }
  });
#undef MOE_TREE
#undef MOE_TREE_ROWS
  if (e != hipSuccess || !cut) return e;
#define MOE_JOIN(D) \
  case D: hipLaunchKernelGGL((attn_tree_join_kernel<D>), grid, dim3(256), 0, st, a); break;
  const int64_t each = (int64_t)c.heads_kv * ((a.rows + 31) / 32) * (c.head_dim / 64);   // of a sequence
  return launch_workgroups(c.batch * each, [&](uint32_t first, dim3 grid) {
    a.first = first;
    switch (c.head_dim) { MOE_JOIN(64) MOE_JOIN(128) MOE_JOIN(256) MOE_JOIN(512) }
  });
#undef MOE_JOIN
}

}  // namespace moe
