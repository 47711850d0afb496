// Rows and pages of the paged cache moved on the device
// (include/moe_serving.h: moe_kv_compact, moe_kv_copy_pages).  Nothing is
// computed: bound by the bytes, read once and written once.
//
// Measured: up to 32 accepted rows of each of 512 sequences, 8 FP8 heads of 128 12.3 us (32 MB,
// 2.6 TB/s: counts, lengths, path, pages and rows wait for one another), of three
// sequences 4.1 us, the launch; 240 pages of 256 KB, of which every 15 have one source, 16 to 19 us (122 MB).
#include <algorithm>

#include "attn_internal.h"

namespace moe {

namespace {

struct MoveArgs {
  char* data[2];           // k, and v where it is a tensor of its own
  uint8_t* scale[2];       // their scales, null for none
  int kinds, scales;
  int64_t sp, sh, st;      // bytes
  int64_t pages;
  int heads, page_shift;
  int chunk_shift;         // 16-byte chunks of a row: 2^chunk_shift
  int groups;              // scale bytes of a row
  uint32_t first;          // the launch's first workgroup
};

MoveArgs move_args(const moe_kv_cache& c) {
  MoveArgs a{};
  const int eb = c.format == MOE_KV_FP8 ? 1 : 2;
  a.data[0] = static_cast<char*>(c.k);
  a.data[1] = static_cast<char*>(c.v);
  a.kinds = c.k == c.v ? 1 : 2;
  if (eb == 1) {
    a.scale[0] = c.k_scale;
    a.scale[1] = c.v_scale;
    a.scales = c.k_scale == c.v_scale ? 1 : 2;
  }
  a.sp = c.stride_page * eb; a.sh = c.stride_head * eb; a.st = c.stride_token * eb;
  a.pages = c.pages;
  a.heads = c.heads;
  a.page_shift = __builtin_ctz((unsigned)c.page_size);
  a.chunk_shift = __builtin_ctz((unsigned)(c.head_dim * eb / 16));
  a.groups = c.head_dim < 128 ? 1 : c.head_dim / 128;
  return a;
}

struct CompactArgs {
  MoveArgs m;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* path;
  const int32_t* counts;
  int nodes, width;
  int units, parts;        // heads of k and v a workgroup takes, workgroups of a sequence
};

// A workgroup takes `units` heads of k or v (or both) of a sequence.  In one turn its threads hold
// all moved rows of as many of them as 8 chunks of 16 bytes a thread have room for
// (one of 64 rows of 1 KB) before the first is written, so that a row may be
// source and destination at once.  Rows are counted to the next power of two,
// so that a chunk's place needs no division.
// 512 sequences of up to 32 rows, 8 FP8 heads of 128: 13.1 us; with a workgroup for every
// head and tensor, each of which walks lengths, path and table again, 24.5.
constexpr int kMoveThreads = 512;
__global__ __launch_bounds__(kMoveThreads) void kv_compact_kernel(CompactArgs p) {
  __shared__ int64_t from[64], to[64];       // byte offsets of the rows in k or v, head 0; -1: stays
  __shared__ int64_t sfrom[64], sto[64];     // rows of head 0's scales
  const uint32_t wg = p.m.first + blockIdx.x;
  const int b = wg / p.parts, part = wg - b * p.parts;
  const int tid = threadIdx.x;
  const int n = min(max(p.counts[b], 0), p.nodes);
  const int64_t len = max(p.lens[b], 0), cap = (int64_t)p.width << p.m.page_shift;
  if (tid < 64) {
    const int node = tid < p.nodes ? p.path[(int64_t)b * p.nodes + tid] : -1;
    int64_t f = -1, t = -1, sf = 0, s = 0;
    const int64_t src = len + node, dst = len + tid;
    const int mask = (1 << p.m.page_shift) - 1;
    if (tid < n && node >= 0 && node < p.nodes && node != tid && src < cap && dst < cap) {
      const int32_t* row = p.table + (int64_t)b * p.width;
      const int64_t ps = row[src >> p.m.page_shift], pd = row[dst >> p.m.page_shift];
      if (ps >= 0 && ps < p.m.pages && pd >= 0 && pd < p.m.pages) {
        f = ps * p.m.sp + (src & mask) * p.m.st;
        t = pd * p.m.sp + (dst & mask) * p.m.st;
        sf = ((ps * p.m.heads) << p.m.page_shift) + (src & mask);
        s = ((pd * p.m.heads) << p.m.page_shift) + (dst & mask);
      }
    }
    from[tid] = f;
    to[tid] = t;
    sfrom[tid] = sf;
    sto[tid] = s;
  }
  __syncthreads();
  if (n == 0) return;
  const int cs = p.m.chunk_shift, ns = n > 1 ? 32 - __builtin_clz(n - 1) : 0;
  const int first = part * p.units, last = min(first + p.units, p.m.heads * p.m.kinds);
  const int turn = 4096 >> (cs + ns);        // units in a turn
  const int g = p.m.groups;
  const bool both = p.m.kinds == 1 && p.m.scales == 2;   // one tensor with two arrays of scales
  for (int u0 = first; u0 < last; u0 += turn) {
    const int units = min(turn, last - u0), total = units << (cs + ns);
    u32x4 x[8];
    char* at_of[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = tid + kMoveThreads * i, r = (at >> cs) & ((1 << ns) - 1), u = u0 + (at >> (cs + ns));
      at_of[i] = nullptr;
      if (at < total && r < n && from[r] >= 0) {
        const int kind = p.m.kinds == 2 ? u & 1 : 0, h = p.m.kinds == 2 ? u >> 1 : u;
        char* head = p.m.data[kind] + h * p.m.sh + 16 * (at & ((1 << cs) - 1));
        x[i] = *reinterpret_cast<const u32x4*>(head + from[r]);
        at_of[i] = head + to[r];
      }
    }
    // scales: a row's groups of every unit, `sub` of them a thread
    auto scale_of = [&](int i, int& r, int64_t& step, uint8_t*& sc, uint8_t*& sc2) {
      const int at = tid + kMoveThreads * i;          // group, row, unit
      const int c = at % g, rest = at / g;
      r = rest & ((1 << ns) - 1);
      const int u = u0 + (rest >> ns);
      if (!p.m.scale[0] || u >= u0 + units || r >= n || from[r] < 0) return false;
      const int kind = p.m.kinds == 2 ? u & 1 : 0, h = p.m.kinds == 2 ? u >> 1 : u;
      if (p.m.scales == 1 && kind) return false;
      sc = p.m.scale[p.m.scales == 2 ? kind : 0];
      sc2 = both ? p.m.scale[1] : nullptr;
      step = ((int64_t)h << p.m.page_shift) * g + c;
      return true;
    };
    // units * rows * groups is at most 4096 / (chunks of a row / groups): 2 bytes a thread
    uint8_t s0[2], s1[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int r;
      int64_t step;
      uint8_t *sc, *sc2;
      if (scale_of(i, r, step, sc, sc2)) {
        s0[i] = sc[sfrom[r] * g + step];
        if (sc2) s1[i] = sc2[sfrom[r] * g + step];
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at_of[i]) *reinterpret_cast<u32x4*>(at_of[i]) = x[i];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int r;
      int64_t step;
      uint8_t *sc, *sc2;
      if (scale_of(i, r, step, sc, sc2)) {
        sc[sto[r] * g + step] = s0[i];
        if (sc2) sc2[sto[r] * g + step] = s1[i];
      }
    }
  }
}

struct CopyArgs {
  MoveArgs m;
  const int32_t* src;
  const int32_t* dst;
  int64_t chunks;          // of a page of k or v
  int64_t schunks;         // of a page's scales, which are contiguous
  int parts, sparts;       // workgroups for each of them
  int per;                 // workgroups per pair
};

// 16-byte chunks a thread moves (the 240 pages above: with eight 31 us, non-temporal 22)
constexpr int kCopyChunks = 4;

__global__ __launch_bounds__(256) void kv_copy_pages_kernel(CopyArgs p) {
  const uint32_t wg = p.m.first + blockIdx.x;
  const uint32_t pair = wg / p.per;
  int part = wg - pair * p.per;
  const int64_t s = p.src[pair], d = p.dst[pair];
  if (s < 0 || s >= p.m.pages || d < 0 || d >= p.m.pages || s == d) return;
  const bool scales = part >= p.parts * p.m.kinds;
  if (scales) part -= p.parts * p.m.kinds;
  const int each = scales ? p.sparts : p.parts;
  const int kind = part / each;
  part -= kind * each;
  const int64_t total = scales ? p.schunks : p.chunks;
  const int64_t at0 = (int64_t)part * 256 * kCopyChunks + threadIdx.x;
  u32x4 x[kCopyChunks];
  if (scales) {
    uint8_t* base = p.m.scale[kind];
#pragma unroll
    for (int i = 0; i < kCopyChunks; ++i) {
      const int64_t at = at0 + 256 * i;
      if (at < total) x[i] = *reinterpret_cast<const u32x4*>(base + (s * total + at) * 16);
    }
#pragma unroll
    for (int i = 0; i < kCopyChunks; ++i) {
      const int64_t at = at0 + 256 * i;
      if (at < total) *reinterpret_cast<u32x4*>(base + (d * total + at) * 16) = x[i];
    }
    return;
  }
  char* base = p.m.data[kind];
  auto place = [&](int64_t at) {           // chunk of a page: its head, row, place in the row
    const int64_t row = at >> p.m.chunk_shift;
    return (row >> p.m.page_shift) * p.m.sh + (row & ((1 << p.m.page_shift) - 1)) * p.m.st +
           16 * (at & ((1 << p.m.chunk_shift) - 1));
  };
#pragma unroll
  for (int i = 0; i < kCopyChunks; ++i) {
    const int64_t at = at0 + 256 * i;
    if (at < total) x[i] = *reinterpret_cast<const u32x4*>(base + s * p.m.sp + place(at));
  }
#pragma unroll
  for (int i = 0; i < kCopyChunks; ++i) {
    const int64_t at = at0 + 256 * i;
    if (at < total) *reinterpret_cast<u32x4*>(base + d * p.m.sp + place(at)) = x[i];
  }
}

}  // namespace

hipError_t launch_kv_compact(const moe_kv_cache& c, int batch, int nodes, const int32_t* table,
                             int width, const int32_t* lens, const int32_t* path,
                             const int32_t* counts, hipStream_t st) {
  if (batch == 0 || width == 0 || c.pages == 0) return hipSuccess;
  CompactArgs a{};
  a.m = move_args(c);
  a.table = table; a.lens = lens; a.path = path; a.counts = counts;
  a.nodes = nodes; a.width = width;
  // a workgroup of its own for every head while there are no more than two a CU, which a CU holds
  // at once (512 sequences of 16 heads of k and v: 13.1 us; 14.7 with twice as many, 20.2 with four times)
  const int units = c.heads * a.m.kinds;
  a.units = (int)std::min<int64_t>(units, std::max<int64_t>(1, (int64_t)batch * units / 512));
  a.parts = (units + a.units - 1) / a.units;
  return launch_workgroups((int64_t)batch * a.parts, [&](uint32_t first, dim3 grid) {
    a.m.first = first;
    hipLaunchKernelGGL(kv_compact_kernel, grid, dim3(kMoveThreads), 0, st, a);
  });
}

hipError_t launch_kv_copy_pages(const moe_kv_cache& c, int64_t n, const int32_t* src,
                                const int32_t* dst, hipStream_t st) {
  if (n == 0 || c.pages == 0) return hipSuccess;
  CopyArgs a{};
  a.m = move_args(c);
  a.src = src; a.dst = dst;
  const int64_t each = 256 * kCopyChunks;
  a.chunks = ((int64_t)c.heads * c.page_size) << a.m.chunk_shift;
  a.parts = (int)((a.chunks + each - 1) / each);
  if (a.m.scales) {
    a.schunks = (int64_t)c.heads * c.page_size * a.m.groups / 16;   // pages have 16 rows and more
    a.sparts = (int)((a.schunks + each - 1) / each);
  }
  a.per = a.parts * a.m.kinds + a.sparts * a.m.scales;
  // pairs go out in launches of which each has fewer than 2^32 workgroups in all
  const int64_t most = (int64_t(1) << 31) / a.per;
  for (int64_t at = 0; at < n; at += most) {
    const int64_t now = n - at < most ? n - at : most;
    a.src = src + at;
    a.dst = dst + at;
    const hipError_t e = launch_workgroups(now * a.per, [&](uint32_t first, dim3 grid) {
      a.m.first = first;
      hipLaunchKernelGGL(kv_copy_pages_kernel, grid, dim3(256), 0, st, a);
    });
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
