// The pool of cache pages (include/moe_serving.h: moe_pool_grow,
// moe_pool_fork, moe_pool_trim): block table, lengths and reference counts
// on the device.
//
// All results are whole numbers and do not depend on the order of the atomic
// additions: a page is free exactly when its count is 0, and free pages are
// handed out by their number.  Bound by the launches and by latencies; of
// memory the counts are read once, and the table entries that change.  256
// sequences that grow by 9 tokens on shared pages, 2560 pages in all: grow 8.5 us, trim 3.9, fork 5.8.
#include <algorithm>
#include <climits>

#include "attn_internal.h"

namespace moe {

namespace {

constexpr int kThreads = 1024;
constexpr int kChunk = 8 * kThreads;     // pages a workgroup looks through

struct GrowArgs {
  int32_t* refs;
  int32_t* table;
  int32_t* lens;
  int64_t pages;
  int batch, width, page_shift;
  int64_t tokens;
  const int32_t* cu;
  int64_t* slots;
  int32_t* positions;
  int32_t* src;
  int32_t* dst;
  int32_t* missing;
  // workspace
  int32_t* totals;         // pages wanted, pages free
  int32_t* free_in;        // [chunks] free pages of each
  int32_t* old;            // [batch] lengths before
  int32_t* base;           // [batch] how many pages the sequences before want
  int32_t* copies;         // [batch] whether the partly filled page is copied
  int32_t* growers;        // [pages] how many sequences grow on a shared page
  int32_t* keeper;         // [pages] the smallest keep_key of theirs
  int32_t* list;           // [pages] the free pages in order
};

__device__ __forceinline__ int clamp_cu(const GrowArgs& p, int b) {
  return (int)min((int64_t)max(p.cu[b], 0), p.tokens);
}

// The sum of x over the workgroup's threads before this one, and over all.
__device__ __forceinline__ int block_scan(int x, int& all, int* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int incl = wave_scan(x);
  __syncthreads();
  if (lane == 63) lds[wave] = incl;
  __syncthreads();
  int before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) {
    const int v = lds[w];
    if (w < wave) before += v;
    all += v;
  }
  return before + incl - x;
}

// The 8 counts of a thread's pages in a chunk: bit i of the result says that page 8 t + i is free.
__device__ __forceinline__ uint32_t free_bits(const GrowArgs& p, int64_t page0) {
  uint32_t bits = 0;
  if (page0 + 8 <= p.pages) {
    const int4 a = *reinterpret_cast<const int4*>(p.refs + page0);
    const int4 b = *reinterpret_cast<const int4*>(p.refs + page0 + 4);
    bits = (a.x == 0) | (a.y == 0) << 1 | (a.z == 0) << 2 | (a.w == 0) << 3 | (b.x == 0) << 4 |
           (b.y == 0) << 5 | (b.z == 0) << 6 | (b.w == 0) << 7;
  } else {
    for (int i = 0; i < 8; ++i)
      if (page0 + i < p.pages && p.refs[page0 + i] == 0) bits |= 1u << i;
  }
  return bits;
}

// What one sequence asks for.
struct Want {
  int len, longer;         // tokens before and after
  int first, past;         // table entries that get a fresh page
  int shared;              // the partly filled page it grows on, if others hold it too, or -1
};
__device__ __forceinline__ Want want_of(const GrowArgs& p, int b) {
  Want w;
  const int cap = p.width << p.page_shift, mask = (1 << p.page_shift) - 1;
  w.len = min(max(p.lens[b], 0), cap);
  const int n = max(clamp_cu(p, b + 1) - clamp_cu(p, b), 0);
  w.longer = (int)min((int64_t)w.len + n, (int64_t)cap);
  w.first = (w.len + mask) >> p.page_shift;
  w.past = (w.longer + mask) >> p.page_shift;
  w.shared = -1;
  if (w.longer > w.len && (w.len & mask)) {
    const int page = p.table[(int64_t)b * p.width + (w.len >> p.page_shift)];
    if (page >= 0 && page < p.pages && p.refs[page] > 1) w.shared = page;
  }
  return w;
}

// Where all holders of a page grow, the one with the smallest key keeps it: the one with the most
// tokens on it, of equals the first.  What it writes there is behind the tokens of all others, so
// that they lose nothing, also where there is no page left for their copies.
__device__ __forceinline__ int keep_key(const GrowArgs& p, const Want& w, int b) {
  const int mask = (1 << p.page_shift) - 1;
  return (mask - (w.len & mask)) << 16 | b;      // 12 bits and 16
}

// Workgroup 0: how many pages each sequence wants, and whether it copies the page it grows on.
// The others: how many pages of a chunk are free.
__global__ __launch_bounds__(kThreads) void pool_plan_kernel(GrowArgs p) {
  __shared__ int lds[kThreads / 64];
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    const int c = blockIdx.x - 1;
    int all;
    block_scan(__popc(free_bits(p, (int64_t)c * kChunk + 8 * tid)), all, lds);
    if (tid == 0) p.free_in[c] = all;
    return;
  }
  // growers of each shared page, counted after all of them have cleared its places
  bool any = false;
  for (int b = tid; b < p.batch; b += kThreads) {
    const int s = want_of(p, b).shared;
    if (s < 0) continue;
    any = true;
    atomicExch(&p.growers[s], 0);
    atomicExch(&p.keeper[s], INT_MAX);
  }
  if (__syncthreads_or(any)) {
    __threadfence();
    __syncthreads();
    for (int b = tid; b < p.batch; b += kThreads) {
      const Want w = want_of(p, b);
      if (w.shared < 0) continue;
      atomicAdd(&p.growers[w.shared], 1);
      atomicMin(&p.keeper[w.shared], keep_key(p, w, b));
    }
    __threadfence();
    __syncthreads();
  }
  int base = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
    const int b = b0 + tid;
    int need = 0;
    Want w{};
    bool copy = false;
    if (b < p.batch) {
      w = want_of(p, b);
      if (w.shared >= 0) {
        const int n = atomicAdd(&p.growers[w.shared], 0), key = atomicAdd(&p.keeper[w.shared], 0);
        copy = !(n == p.refs[w.shared] && key == keep_key(p, w, b));
      }
      need = w.past - w.first + copy;
    }
    int all;
    const int before = block_scan(need, all, lds);
    if (b < p.batch) {
      p.old[b] = w.len;
      p.base[b] = base + before;
      p.copies[b] = copy;
    }
    base += all;
  }
  if (tid == 0) p.totals[0] = base;
}

// The free pages in order, as many as are wanted.
__global__ __launch_bounds__(kThreads) void pool_list_kernel(GrowArgs p) {
  __shared__ int lds[kThreads / 64];
  const int tid = threadIdx.x, c = blockIdx.x;
  int before = 0;
  for (int i = tid; i < c; i += kThreads) before += p.free_in[i];
  int all;
  block_scan(before, all, lds);
  const int wanted = p.totals[0];
  const int64_t page0 = (int64_t)c * kChunk + 8 * tid;
  const uint32_t bits = free_bits(p, page0);
  int own;
  int at = all + block_scan(__popc(bits), own, lds);
  if (c == (int)gridDim.x - 1 && tid == 0) p.totals[1] = all + own;
  for (int i = 0; i < 8; ++i)
    if (bits >> i & 1) {
      if (at < wanted) p.list[at] = (int)(page0 + i);
      ++at;
    }
}

// Workgroups below `seq_groups`: a wave per sequence writes its entries, counts and length.
// The others: a thread per token writes its slot and position.
__global__ __launch_bounds__(256) void pool_fill_kernel(GrowArgs p, uint32_t seq_groups) {
  const int mask = (1 << p.page_shift) - 1;
  const int found = p.pages > 0 ? p.totals[1] : 0;
  auto fresh = [&](int rank) { return rank < found ? p.list[rank] : -1; };
  if (blockIdx.x < seq_groups) {
    const int lane = threadIdx.x & 63, b = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.missing = max(p.totals[0] - found, 0);
    if (b >= p.batch) return;
    const int len = p.old[b], copy = p.copies[b];
    const int n = max(clamp_cu(p, b + 1) - clamp_cu(p, b), 0);
    const int longer = (int)min((int64_t)len + n, (int64_t)p.width << p.page_shift);
    const int first = (len + mask) >> p.page_shift, past = (longer + mask) >> p.page_shift;
    int32_t* row = p.table + (int64_t)b * p.width;
    for (int c = first + lane; c < past; c += 64) {
      const int page = fresh(p.base[b] + copy + c - first);
      row[c] = page;
      if (page >= 0) p.refs[page] = 1;
    }
    if (lane == 0) {
      int s = -1, d = -1;
      if (copy && (d = fresh(p.base[b])) >= 0) {
        s = row[len >> p.page_shift];
        row[len >> p.page_shift] = d;
        p.refs[d] = 1;
        atomicSub(&p.refs[s], 1);
      }
      p.src[b] = s;
      p.dst[b] = d;
      p.lens[b] = copy && d < 0 ? len : longer;   // without its copy it stays as it is
    }
    return;
  }
  const int64_t t = (int64_t)(blockIdx.x - seq_groups) * 256 + threadIdx.x;
  if (t >= p.tokens) return;
  // the last sequence that starts at t or before
  int lo = 0, hi = p.batch;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.cu[mid + 1] > t) hi = mid; else lo = mid + 1;
  }
  int64_t slot = -1;
  int pos = 0;
  if (lo < p.batch && t >= clamp_cu(p, lo)) {
    const int len = p.old[lo], copy = p.copies[lo];
    const int64_t at = (int64_t)len + (t - clamp_cu(p, lo));
    pos = (int)min(at, (int64_t)INT_MAX);
    if (at < (int64_t)p.width << p.page_shift) {
      const int c = (int)(at >> p.page_shift), first = (len + mask) >> p.page_shift;
      int page;
      if (c >= first) page = fresh(p.base[lo] + copy + c - first);
      else if (copy) page = fresh(p.base[lo]);
      else page = p.table[(int64_t)lo * p.width + c];
      if (page >= 0 && page < p.pages) slot = ((int64_t)page << p.page_shift) + (at & mask);
    }
  }
  p.slots[t] = slot;
  p.positions[t] = pos;
}

// All of it in one workgroup, for pools and calls of the sizes below: three launches and
// their latencies become one (6 sequences and 4000 pages: 8 us instead of 20.5).
constexpr int kSmallBatch = kThreads, kSmallPages = 64 * kThreads, kSmallTokens = 32 * kThreads;
constexpr int kSmallWanted = 8192;       // pages a call may want
constexpr int kSlots = 2 * kSmallBatch;  // places for shared pages

__global__ __launch_bounds__(kThreads) void pool_grow_kernel(GrowArgs p) {
  __shared__ int lds[kThreads / 64];
  __shared__ int cu[kSmallBatch + 1], old[kSmallBatch], base[kSmallBatch];
  __shared__ uint8_t copies[kSmallBatch];
  __shared__ int slot_page[kSlots], growers[kSlots], keeper[kSlots];
  __shared__ int list[kSmallWanted];
  const int tid = threadIdx.x, mask = (1 << p.page_shift) - 1;
  for (int b = tid; b <= p.batch; b += kThreads) cu[b] = p.cu[b];
  for (int i = tid; i < kSlots; i += kThreads) {
    slot_page[i] = -1;
    growers[i] = 0;
    keeper[i] = INT_MAX;
  }
  // free pages: a thread's are next to each other, in eights
  const int per = (int)((p.pages + kThreads - 1) / kThreads + 7) / 8;   // at most 8
  uint64_t bits = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t page0 = ((int64_t)tid * per + i) * 8;
    if (i < per && page0 < p.pages) bits |= (uint64_t)free_bits(p, page0) << (8 * i);
  }
  Want w{};
  w.shared = -1;
  if (tid < p.batch) w = want_of(p, tid);
  const int holders = w.shared >= 0 ? p.refs[w.shared] : 0;
  __syncthreads();
  // sequences that grow on one shared page meet in its place; there are twice as many places as sequences
  int at = 0;
  if (w.shared >= 0) {
    at = (int)((uint32_t)w.shared * 2654435761u >> 21) & (kSlots - 1);
    for (;;) {
      const int was = atomicCAS(&slot_page[at], -1, w.shared);
      if (was == -1 || was == w.shared) break;
      at = (at + 1) & (kSlots - 1);
    }
    atomicAdd(&growers[at], 1);
    atomicMin(&keeper[at], keep_key(p, w, tid));
  }
  __syncthreads();
  const bool copy =
      w.shared >= 0 && !(growers[at] == holders && keeper[at] == keep_key(p, w, tid));
  int wanted, found;
  const int mine = block_scan(tid < p.batch ? w.past - w.first + copy : 0, wanted, lds);
  int rank = block_scan(__popcll(bits), found, lds);
  const int64_t page0 = (int64_t)tid * per * 8;
  // (offsets that fall may want more than the host has counted, and get no more than this)
  found = min(found, kSmallWanted);
  while (bits && rank < min(wanted, kSmallWanted)) {
    list[rank++] = (int)page0 + __builtin_ctzll(bits);
    bits &= bits - 1;
  }
  if (tid < p.batch) {
    old[tid] = w.len;
    base[tid] = mine;
    copies[tid] = copy;
  }
  __syncthreads();
  auto fresh = [&](int i) { return i < found ? list[i] : -1; };
  // slots and positions, before the entries they are read from change
  for (int64_t t = tid; t < p.tokens; t += kThreads) {
    int lo = 0, hi = p.batch;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid + 1] > t) hi = mid; else lo = mid + 1;
    }
    int64_t slot = -1;
    int pos = 0;
    const int start = lo < p.batch ? (int)min((int64_t)max(cu[lo], 0), p.tokens) : 0;
    if (lo < p.batch && t >= start) {
      const int64_t to = (int64_t)old[lo] + (t - start);
      pos = (int)min(to, (int64_t)INT_MAX);
      if (to < (int64_t)p.width << p.page_shift) {
        const int c = (int)(to >> p.page_shift), first = (old[lo] + mask) >> p.page_shift;
        int page;
        if (c >= first) page = fresh(base[lo] + copies[lo] + c - first);
        else if (copies[lo]) page = fresh(base[lo]);
        else page = p.table[(int64_t)lo * p.width + c];
        if (page >= 0 && page < p.pages) slot = ((int64_t)page << p.page_shift) + (to & mask);
      }
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
  }
  if (tid == 0) *p.missing = max(wanted - found, 0);
  if (tid < p.batch) {
    int32_t* row = p.table + (int64_t)tid * p.width;
    int s = -1, d = -1;
    if (copy && (d = fresh(mine)) >= 0) {
      s = w.shared;
      row[w.len >> p.page_shift] = d;
      p.refs[d] = 1;
      atomicSub(&p.refs[s], 1);
    }
    p.src[tid] = s;
    p.dst[tid] = d;
    p.lens[tid] = copy && d < 0 ? w.len : w.longer;   // without its copy it stays as it is
  }
  // new entries: found by the page they are the next of
  for (int i = tid; i < wanted; i += kThreads) {
    int lo = 0, hi = p.batch;              // the last sequence that wants its first page at i or before
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (base[mid] > i) hi = mid; else lo = mid + 1;
    }
    --lo;
    const int c = i - base[lo] - copies[lo];
    if (c < 0) continue;                   // the copy
    const int page = fresh(i);
    p.table[(int64_t)lo * p.width + ((old[lo] + mask) >> p.page_shift) + c] = page;
    if (page >= 0) p.refs[page] = 1;
  }
}

struct PoolArgs {
  int32_t* refs;
  int32_t* table;
  int32_t* lens;
  int64_t pages;
  int batch, width, page_shift;
};

__device__ __forceinline__ void count(const PoolArgs& p, int page, int by) {
  if (page >= 0 && page < p.pages) atomicAdd(&p.refs[page], by);
}

// A workgroup owns `cols` columns of the table for all sequences: it has read all of
// their entries before it writes one.  The last workgroup does the lengths.  PER: entries a thread holds.
template <int PER>
__global__ __launch_bounds__(kThreads) void pool_fork_kernel(PoolArgs p, const int32_t* parents,
                                                             int cols) {
  const int tid = threadIdx.x;
  const bool lengths = blockIdx.x == gridDim.x - 1;
  const int c0 = blockIdx.x * cols;
  const int n = lengths ? 1 : min(cols, p.width - c0);
  const int total = p.batch * n;
  int32_t* to = lengths ? p.lens : p.table + c0;
  const int stride = lengths ? 1 : p.width;
  const int none = lengths ? 0 : -1;
  int x[PER], old[PER];
  bool moves[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = tid + kThreads * i;
    moves[i] = false;
    if (at >= total) continue;
    const int b = at / n, c = at - b * n, up = parents[b];
    moves[i] = up != b;
    if (!moves[i]) continue;
    x[i] = up >= 0 && up < p.batch ? to[(int64_t)up * stride + c] : none;
    old[i] = to[(int64_t)b * stride + c];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (!moves[i]) continue;
    const int at = tid + kThreads * i, b = at / n, c = at - b * n;
    if (!lengths && x[i] != old[i]) {
      count(p, x[i], 1);
      count(p, old[i], -1);
    }
    to[(int64_t)b * stride + c] = x[i];
  }
}

// A workgroup per sequence.
__global__ __launch_bounds__(256) void pool_trim_kernel(PoolArgs p, const int32_t* lens, int window,
                                                        int sinks) {
  const int b = blockIdx.x;
  int len = max(p.lens[b], 0);
  if (lens) len = min(len, max(lens[b], 0));
  int32_t* row = p.table + (int64_t)b * p.width;
  for (int c = threadIdx.x; c < p.width; c += 256) {
    const int64_t first = (int64_t)c << p.page_shift, past = first + (int64_t(1) << p.page_shift);
    const bool seen = first < len && !(window > 0 && first >= sinks && past <= (int64_t)len - window + 1);
    if (seen) continue;
    const int page = row[c];
    if (page == -1) continue;
    count(p, page, -1);
    row[c] = -1;
  }
  __syncthreads();                        // every thread has read the length
  if (threadIdx.x == 0) p.lens[b] = len;
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }
int64_t chunks_of(const moe_page_pool& p) { return (p.pages + kChunk - 1) / kChunk; }

PoolArgs pool_args(const moe_page_pool& p) {
  return PoolArgs{p.refs, p.table, p.lens, p.pages, p.batch, p.width,
                  __builtin_ctz((unsigned)p.page_size)};
}

}  // namespace

size_t pool_ws_bytes(const moe_page_pool& p) {
  return 256 + up256(chunks_of(p) * 4) + 3 * up256((size_t)p.batch * 4) + 3 * up256(p.pages * 4);
}

hipError_t launch_pool_grow(const moe_page_pool& pool, int64_t tokens, const int32_t* cu,
                            int64_t* slots, int32_t* positions, int32_t* src, int32_t* dst,
                            int32_t* missing, void* ws, hipStream_t st) {
  GrowArgs a{};
  a.refs = pool.refs; a.table = pool.table; a.lens = pool.lens; a.pages = pool.pages;
  a.batch = pool.batch; a.width = pool.width;
  a.page_shift = __builtin_ctz((unsigned)pool.page_size);
  a.tokens = tokens; a.cu = cu; a.slots = slots; a.positions = positions;
  a.src = src; a.dst = dst; a.missing = missing;
  char* w = static_cast<char*>(ws);
  const int64_t chunks = chunks_of(pool);
  auto take = [&](size_t n) {
    int32_t* at = reinterpret_cast<int32_t*>(w);
    w += up256(n * 4);
    return at;
  };
  a.totals = take(2);
  a.free_in = take(chunks);
  a.old = take(pool.batch); a.base = take(pool.batch); a.copies = take(pool.batch);
  a.growers = take(pool.pages); a.keeper = take(pool.pages); a.list = take(pool.pages);
  if (pool.batch <= kSmallBatch && pool.pages <= kSmallPages && tokens <= kSmallTokens &&
      2 * (int64_t)pool.batch + tokens / pool.page_size <= kSmallWanted) {
    hipLaunchKernelGGL(pool_grow_kernel, dim3(1), dim3(kThreads), 0, st, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(pool_plan_kernel, dim3((unsigned)chunks + 1), dim3(kThreads), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (chunks > 0) {
    hipLaunchKernelGGL(pool_list_kernel, dim3((unsigned)chunks), dim3(kThreads), 0, st, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const uint32_t seq_groups = std::max(1, (pool.batch + 3) / 4);
  const int64_t groups = seq_groups + (tokens + 255) / 256;
  hipLaunchKernelGGL(pool_fill_kernel, dim3((unsigned)groups), dim3(256), 0, st, a, seq_groups);
  return hipGetLastError();
}

hipError_t launch_pool_fork(const moe_page_pool& pool, const int32_t* parents, hipStream_t st) {
  if (pool.batch == 0) return hipSuccess;
  const PoolArgs a = pool_args(pool);
  // columns a workgroup owns: one for large batches, whose entries are its threads' registers
  // (256 sequences: 5.8 us with an entry a thread, 11.6 with four).  A column is one workgroup's, since
  // all of it has to be read before any of it is written and a call has no memory of its own for the old
  // entries; past 16384 sequences a thread holds up to 64 entries, more than its registers (570
  // are spilled): 64 columns of 16384 sequences 47 us, of 65536 288.
  const int cols = std::clamp(kThreads / pool.batch, 1, 64);
  const unsigned groups = (unsigned)((pool.width + cols - 1) / cols) + 1;
  const int64_t most = (int64_t)pool.batch * cols;
  if (most <= kThreads)
    hipLaunchKernelGGL((pool_fork_kernel<1>), dim3(groups), dim3(kThreads), 0, st, a, parents, cols);
  else if (most <= 4 * kThreads)
    hipLaunchKernelGGL((pool_fork_kernel<4>), dim3(groups), dim3(kThreads), 0, st, a, parents, cols);
  else if (most <= 16 * kThreads)
    hipLaunchKernelGGL((pool_fork_kernel<16>), dim3(groups), dim3(kThreads), 0, st, a, parents, cols);
  else
    hipLaunchKernelGGL((pool_fork_kernel<64>), dim3(groups), dim3(kThreads), 0, st, a, parents, cols);
  return hipGetLastError();
}

hipError_t launch_pool_trim(const moe_page_pool& pool, const int32_t* lens, int window, int sinks,
                            hipStream_t st) {
  if (pool.batch == 0) return hipSuccess;
  hipLaunchKernelGGL(pool_trim_kernel, dim3((unsigned)pool.batch), dim3(256), 0, st,
                     pool_args(pool), lens, window, sinks);
  return hipGetLastError();
}

}  // namespace moe
