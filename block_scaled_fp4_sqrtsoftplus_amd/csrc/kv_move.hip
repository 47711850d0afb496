// Rows and pages of the paged cache moved on the device
// (include/moe_serving.h: moe_kv_compact, moe_kv_copy_pages).  Nothing is
// computed: bound by the bytes, read once and written once.
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
};

// One workgroup per sequence and head, and for k and v.  Its threads hold all
// of the moved rows (up to 64 of 1 KB: 16 chunks of 16 bytes a thread) before
// the first is written, so that a row may be source and destination at once.
__global__ __launch_bounds__(256) void kv_compact_kernel(CompactArgs p) {
  __shared__ int64_t from[64], to[64];       // byte offsets of the rows in k or v; -1: stays
  __shared__ int64_t sfrom[64], sto[64];     // rows of the scales
  const uint32_t wg = p.m.first + blockIdx.x;
  const int kind = p.m.kinds == 2 ? wg & 1 : 0;
  const uint32_t rest = p.m.kinds == 2 ? wg >> 1 : wg;
  const int b = rest / p.m.heads, h = rest - b * p.m.heads;
  const int n = min(max(p.counts[b], 0), p.nodes);
  if (n == 0) return;
  const int tid = threadIdx.x;
  if (tid < 64) {
    int64_t f = -1, t = -1, sf = 0, s = 0;
    if (tid < n) {
      const int node = p.path[(int64_t)b * p.nodes + tid];
      const int64_t len = max(p.lens[b], 0), cap = (int64_t)p.width << p.m.page_shift;
      const int64_t src = len + node, dst = len + tid;
      const int mask = (1 << p.m.page_shift) - 1;
      if (node >= 0 && node < p.nodes && node != tid && src < cap && dst < cap) {
        const int32_t* row = p.table + (int64_t)b * p.width;
        const int64_t ps = row[src >> p.m.page_shift], pd = row[dst >> p.m.page_shift];
        if (ps >= 0 && ps < p.m.pages && pd >= 0 && pd < p.m.pages) {
          f = ps * p.m.sp + h * p.m.sh + (src & mask) * p.m.st;
          t = pd * p.m.sp + h * p.m.sh + (dst & mask) * p.m.st;
          sf = ((ps * p.m.heads + h) << p.m.page_shift) + (src & mask);
          s = ((pd * p.m.heads + h) << p.m.page_shift) + (dst & mask);
        }
      }
    }
    from[tid] = f;
    to[tid] = t;
    sfrom[tid] = sf;
    sto[tid] = s;
  }
  __syncthreads();
  char* data = p.m.data[kind];
  const int cs = p.m.chunk_shift, total = n << cs;
  u32x4 x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int at = tid + 256 * i;
    if (at < total && from[at >> cs] >= 0)
      x[i] = *reinterpret_cast<const u32x4*>(data + from[at >> cs] + 16 * (at & ((1 << cs) - 1)));
  }
  // scales: up to 64 rows of 4 bytes, one a thread; one tensor may have two arrays
  const int g = p.m.groups;
  const int r = tid / g, c = tid - r * g;
  const bool scaled = p.m.scale[0] && (p.m.scales == 2 || kind == 0) && r < n && from[r] >= 0;
  const bool both = p.m.kinds == 1 && p.m.scales == 2;
  uint8_t* sc = p.m.scale[p.m.scales == 2 ? kind : 0];
  uint8_t s0 = 0, s1 = 0;
  if (scaled) {
    s0 = sc[sfrom[r] * g + c];
    if (both) s1 = p.m.scale[1][sfrom[r] * g + c];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int at = tid + 256 * i;
    if (at < total && from[at >> cs] >= 0)
      *reinterpret_cast<u32x4*>(data + to[at >> cs] + 16 * (at & ((1 << cs) - 1))) = x[i];
  }
  if (scaled) {
    sc[sto[r] * g + c] = s0;
    if (both) p.m.scale[1][sto[r] * g + c] = s1;
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

constexpr int kCopyChunks = 8;   // 16-byte chunks a thread moves

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
  return launch_workgroups((int64_t)batch * c.heads * a.m.kinds, [&](uint32_t first, dim3 grid) {
    a.m.first = first;
    hipLaunchKernelGGL(kv_compact_kernel, grid, dim3(256), 0, st, a);
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
