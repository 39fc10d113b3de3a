// The life of a pool's pages: copies, forks, room for growth, release and compaction.
//
// refs[p] counts the page-table entries that hold page p; a page with refs 0 is free. New pages
// are handed out lowest first, in item order, so a call's result depends on its inputs alone
// (the counts are integer atomics, whose order does not change the result).
//
//  * page_count_kernel, page_list_kernel: which pages are free, and for compaction which live
//    ones lie above the border, as lists in the workspace. Each CTA takes a chunk of pages and
//    adds up the counts of the chunks before its own; one more CTA ranks the items' needs.
//  * fork_kernel, extend_kernel, free_kernel, compact_kernel: the page table and the counts,
//    with the rows to copy.
//  * copy_kernel: listed pages.
// The kernels of a call start early and wait for the one before them: where no page is copied,
// launches and the latency of a few dependent loads bound a call (free, fork and extend of 8
// children: 26 us in all). Copies are bound by HBM: a CTA copies the rows of one (page, layer,
// channel), four 16-byte loads a thread in flight, many CTAs to an SM (compaction of 9000 pages,
// 3.98 GB read and written: 647 us, 6.2 TB/s; 500 MLA pages, 498 MB: 85 us, 5.8 TB/s; 384 copies
// of a fork: 133 us of which 113 are their writes at the rate of a plain copy).
#include "kamera_dev.cuh"
#include "kamera_ptx.cuh"

namespace kamera {

namespace {

constexpr int kThr = 256;
constexpr int kPer = 4;              // pages per thread
constexpr int kChunk = kThr * kPer;  // pages per chunk
// Up to so many chunks, each listing CTA counts them all itself, which saves a launch (extend and
// free of 64 requests: 13 us instead of 14 at 1024 pages; 16 instead of 14 at 16384).
constexpr int kOwnCount = 4;

struct Work {  // the workspace
  long long *rank;    // [n] free pages needed before each item
  long long *scalar;  // n_free, n_moves
  int *counts;        // [chunks] free pages of each chunk
  int *list;          // free pages, ascending (compaction: those below the border)
  int *above;         // compaction: live pages from the border on, descending
  int *pos;           // compaction: a live page's index in `above`
};

__host__ __device__ inline int page_chunks(long long pages) {
  return (int)((pages + kChunk - 1) / kChunk);
}

__host__ __device__ inline Work work_of(void *ws, int n, long long pages) {
  Work w;
  w.rank = static_cast<long long *>(ws);
  w.scalar = w.rank + n;
  w.counts = reinterpret_cast<int *>(w.scalar + 2);
  w.list = w.counts + page_chunks(pages);
  w.above = w.list + pages;
  w.pos = w.above + pages;
  return w;
}

// Inclusive scan over the CTA's values; every thread also gets the total.
template <class T>
__device__ __forceinline__ T block_scan(T x, T *total) {
  __shared__ T part[kThr / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // earlier readers of part are done
  if (lane == 31) part[warp] = x;
  __syncthreads();
  T before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kThr / 32; ++w) {
    if (w < warp) before += part[w];
    sum += part[w];
  }
  *total = sum;
  return x + before;
}

template <class T>
__device__ __forceinline__ T block_sum(T x) {
  T total;
  block_scan(x, &total);
  return total;
}

__device__ __forceinline__ int page_of(const PageArgs &a, int req, long long index) {
  return a.table[(long long)req * a.pool.pt_stride + index];
}
__device__ __forceinline__ bool in_pool(const PageArgs &a, int page) {
  return page >= 0 && page < a.num_pages;
}
__device__ __forceinline__ long long pages_for(const PageArgs &a, int tokens) {
  return ((long long)tokens + a.lay.page_size - 1) / a.lay.page_size;
}

// A thread's counts; -1 past the pool.
__device__ __forceinline__ void load_refs(const PageArgs &a, long long p0, int *r) {
#pragma unroll
  for (int e = 0; e < kPer; ++e) r[e] = p0 + e < a.num_pages ? a.refs[p0 + e] : -1;
}

__global__ void __launch_bounds__(kThr) page_count_kernel(const __grid_constant__ PageArgs a) {
  ptx::launch_dependents();
  ptx::wait_for_previous();
  const Work w = work_of(a.ws, a.n, a.num_pages);
  int r[kPer];
  load_refs(a, (long long)blockIdx.x * kChunk + kPer * threadIdx.x, r);
  int n = 0;
#pragma unroll
  for (int e = 0; e < kPer; ++e) n += r[e] == 0;
  n = block_sum(n);
  if (threadIdx.x == 0) w.counts[blockIdx.x] = n;
}

// Whether an item keeps its rules.
__device__ __forceinline__ bool fork_ok(const PageArgs &a, const kamera_fork_item &f) {
  return f.parent >= 0 && f.parent < a.pool.num_reqs && f.child >= 0 &&
         f.child < a.pool.num_reqs && f.child != f.parent && f.num_tokens >= 0 &&
         f.num_tokens <= (long long)a.pool.pt_stride * a.lay.page_size;
}
__device__ __forceinline__ bool span_ok(const PageArgs &a, const kamera_page_span &s) {
  return s.req >= 0 && s.req < a.pool.num_reqs && s.from_tok >= 0 && s.to_tok >= s.from_tok &&
         s.to_tok <= (long long)a.pool.pt_stride * a.lay.page_size;
}

// Free pages that item i needs (0 for an item that breaks its rules).
__device__ __forceinline__ long long item_need(const PageArgs &a, int i) {
  if (a.forks) {
    const kamera_fork_item f = a.forks[i];
    return fork_ok(a, f) && f.num_tokens % a.lay.page_size != 0;
  }
  const kamera_page_span s = a.spans[i];
  return span_ok(a, s) ? pages_for(a, s.to_tok) - pages_for(a, s.from_tok) : 0;
}

__global__ void __launch_bounds__(kThr) page_list_kernel(const __grid_constant__ PageArgs a) {
  const Work w = work_of(a.ws, a.n, a.num_pages);
  const int tid = threadIdx.x, chunks = page_chunks(a.num_pages);
  const bool compact = !a.forks && !a.spans;
  ptx::launch_dependents();
  ptx::wait_for_previous();
  if (blockIdx.x == chunks) {  // the items' ranks
    long long base = 0;
    for (int i0 = 0; i0 < a.n; i0 += kThr) {
      const int i = i0 + tid;
      const long long need = i < a.n ? item_need(a, i) : 0;
      long long total;
      const long long incl = block_scan(need, &total);
      if (i < a.n) w.rank[i] = base + incl - need;
      base += total;
    }
    return;
  }
  long long before = 0, all = 0;  // free pages in the chunks before this one, and in all
  if (chunks <= kOwnCount) {
    const int first = blockIdx.x * kChunk;
#pragma unroll 8
    for (int p = tid; p < (int)a.num_pages; p += kThr) {
      const int n = a.refs[p] == 0;
      all += n;
      if (p < first) before += n;
    }
  } else {
    for (int c = tid; c < chunks; c += kThr) {
      const int n = w.counts[c];
      all += n;
      if (c < blockIdx.x) before += n;
    }
  }
  before = block_sum(before);
  all = block_sum(all);
  const long long p0 = (long long)blockIdx.x * kChunk + kPer * tid;
  const long long live = a.num_pages - all;  // the border of compaction
  int r[kPer], n = 0, total;
  load_refs(a, p0, r);
#pragma unroll
  for (int e = 0; e < kPer; ++e) n += r[e] == 0;
  long long at = before + block_scan(n, &total) - n;  // free pages below this thread's
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const long long p = p0 + e;
    if (p >= a.num_pages) break;
    if (compact && p == live) w.scalar[1] = at;  // as many live pages lie above the border
    if (r[e] == 0) {
      if (!compact || p < live) w.list[at] = (int)p;
      ++at;
    } else if (compact && p >= live) {
      const int after = (int)((a.num_pages - 1 - p) - (all - at));  // live pages above this one
      w.above[after] = (int)p;
      w.pos[p] = after;
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    w.scalar[0] = all;
    if (compact) {
      if (all == 0) w.scalar[1] = 0;
      *a.num_live = (int)live;
    }
  }
}

// `bytes` (a multiple of 16) from src to dst by the CTA.
__device__ __forceinline__ void copy_bytes(__nv_bfloat16 *dst, const __nv_bfloat16 *src,
                                           int bytes) {
  const uint4 *s = reinterpret_cast<const uint4 *>(src);
  uint4 *d = reinterpret_cast<uint4 *>(dst);
  const int n = bytes >> 4;
  constexpr int kB = 4;
  for (int e0 = threadIdx.x; e0 < n; e0 += kThr * kB) {
    uint4 v[kB];
#pragma unroll
    for (int j = 0; j < kB; ++j)
      if (e0 + j * kThr < n) v[j] = s[e0 + j * kThr];
#pragma unroll
    for (int j = 0; j < kB; ++j)
      if (e0 + j * kThr < n) d[e0 + j * kThr] = v[j];
  }
}

// The first `rows` rows of page src to page dst in one layer of one channel (K or V).
__device__ __forceinline__ void copy_rows(const PageArgs &a, int lc, long long src, long long dst,
                                          int rows) {
  const int ch = lc % a.lay.n_ch, layer = lc / a.lay.n_ch;
  const int row = ch == 0 ? a.lay.row_k : a.lay.row_v;
  __nv_bfloat16 *p = (ch == 0 ? a.pool.k : a.pool.v) + (long long)layer * a.pool.num_slots * row;
  const long long page = (long long)a.lay.page_size * row;
  for (int r0 = 0; r0 < rows; r0 += 4096) {  // 4096 rows: at most 128 MB, an int of bytes
    const int n = min(4096, rows - r0);
    copy_bytes(p + dst * page + (long long)r0 * row, p + src * page + (long long)r0 * row,
               n * row * 2);
  }
}

// Item x; slice y = (layer, channel). Slice 0 also writes the child's entries and the counts.
__global__ void __launch_bounds__(kThr) fork_kernel(const __grid_constant__ PageArgs a) {
  ptx::launch_dependents();
  ptx::wait_for_previous();
  const Work w = work_of(a.ws, a.n, a.num_pages);
  const kamera_fork_item f = a.forks[blockIdx.x];
  const int tid = threadIdx.x;
  const bool lead = blockIdx.y == 0;
  if (!fork_ok(a, f)) {
    if (lead && tid == 0) atomicOr(a.status, KAMERA_DEVICE_BAD_ITEM);
    return;
  }
  const int full = f.num_tokens / a.lay.page_size, rest = f.num_tokens - full * a.lay.page_size;
  int page = -1;
  if (rest) {
    const long long rank = w.rank[blockIdx.x];
    if (rank >= w.scalar[0]) {
      if (lead && tid == 0) atomicOr(a.status, KAMERA_DEVICE_NO_PAGES);
      return;
    }
    page = w.list[rank];
  }
  if (lead) {
    int32_t *child = a.table + (long long)f.child * a.pool.pt_stride;
    for (int i = tid; i < full; i += kThr) {
      const int p = page_of(a, f.parent, i);
      child[i] = p;
      if (in_pool(a, p))
        atomicAdd(a.refs + p, 1);
      else
        atomicOr(a.status, KAMERA_DEVICE_SLOT_OOB);
    }
    if (rest && tid == 0) {
      child[full] = page;
      a.refs[page] = 1;
    }
  }
  if (!rest) return;
  const int src = page_of(a, f.parent, full);
  if (!in_pool(a, src)) {
    if (lead && tid == 0) atomicOr(a.status, KAMERA_DEVICE_SLOT_OOB);
    return;
  }
  for (int lc = blockIdx.y; lc < a.lay.L * a.lay.n_ch; lc += gridDim.y)
    copy_rows(a, lc, src, page, rest);
}

__global__ void __launch_bounds__(kThr) extend_kernel(const __grid_constant__ PageArgs a) {
  ptx::launch_dependents();
  ptx::wait_for_previous();
  const Work w = work_of(a.ws, a.n, a.num_pages);
  const kamera_page_span s = a.spans[blockIdx.x];
  if (!span_ok(a, s)) {
    if (threadIdx.x == 0) atomicOr(a.status, KAMERA_DEVICE_BAD_ITEM);
    return;
  }
  const long long p0 = pages_for(a, s.from_tok), n = pages_for(a, s.to_tok) - p0;
  const long long rank = w.rank[blockIdx.x];
  if (n > 0 && rank + n > w.scalar[0]) {
    if (threadIdx.x == 0) atomicOr(a.status, KAMERA_DEVICE_NO_PAGES);
    return;
  }
  int32_t *row = a.table + (long long)s.req * a.pool.pt_stride + p0;
  for (long long i = threadIdx.x; i < n; i += kThr) {
    const int page = w.list[rank + i];
    row[i] = page;
    a.refs[page] = 1;
  }
}

__global__ void __launch_bounds__(kThr) free_kernel(const __grid_constant__ PageArgs a) {
  ptx::launch_dependents();
  ptx::wait_for_previous();
  const kamera_page_span s = a.spans[blockIdx.x];
  if (!span_ok(a, s)) {
    if (threadIdx.x == 0) atomicOr(a.status, KAMERA_DEVICE_BAD_ITEM);
    return;
  }
  const long long p0 = pages_for(a, s.from_tok), p1 = pages_for(a, s.to_tok);
  int32_t *row = a.table + (long long)s.req * a.pool.pt_stride;
  for (long long i = p0 + threadIdx.x; i < p1; i += kThr) {
    const int page = atomicExch(row + i, -1);  // an entry named twice is released once
    if (!in_pool(a, page)) {
      atomicOr(a.status, KAMERA_DEVICE_SLOT_OOB);
    } else if (atomicSub(a.refs + page, 1) <= 0) {  // nothing held it: the count stays
      atomicAdd(a.refs + page, 1);
      atomicOr(a.status, KAMERA_DEVICE_BAD_ITEM);
    }
  }
}

// Move k takes the k-th live page above the border to the k-th free page below it. The CTAs
// walk (move, layer, channel) units; the table and the counts are spread over the grid.
__global__ void __launch_bounds__(kThr) compact_kernel(const __grid_constant__ PageArgs a) {
  ptx::launch_dependents();
  ptx::wait_for_previous();
  const Work w = work_of(a.ws, a.n, a.num_pages);
  const long long moves = w.scalar[1], live = a.num_pages - w.scalar[0];
  const long long gtid = (long long)blockIdx.x * kThr + threadIdx.x;
  const long long gthr = (long long)gridDim.x * kThr;
  for (long long k = gtid; k < moves; k += gthr) {
    const int src = w.above[moves - 1 - k], dst = w.list[k];
    a.refs[dst] = a.refs[src];
    a.refs[src] = 0;
  }
  const long long entries = (long long)a.pool.num_reqs * a.pool.pt_stride;
  for (long long e = gtid; e < entries; e += gthr) {
    const int p = a.table[e];
    if (p < live || p >= a.num_pages) continue;
    const int i = w.pos[p];  // not written for a page that nothing holds
    if (i >= 0 && i < moves && w.above[i] == p) a.table[e] = w.list[moves - 1 - i];
  }
  const int nlc = a.lay.L * a.lay.n_ch;
  for (long long u = blockIdx.x; u < moves * nlc; u += gridDim.x) {
    const long long k = u / nlc;
    copy_rows(a, (int)(u - k * nlc), w.above[moves - 1 - k], w.list[k], a.lay.page_size);
  }
}

__global__ void __launch_bounds__(kThr) copy_kernel(const __grid_constant__ PageArgs a) {
  ptx::launch_dependents();
  ptx::wait_for_previous();
  const int nlc = a.lay.L * a.lay.n_ch;
  for (long long u = blockIdx.x; u < (long long)a.n * nlc; u += gridDim.x) {
    const long long k = u / nlc;
    const int src = a.src[k], dst = a.dst[k];
    if (!in_pool(a, src) || !in_pool(a, dst)) {
      if (threadIdx.x == 0) atomicOr(a.status, KAMERA_DEVICE_SLOT_OOB);
      continue;
    }
    copy_rows(a, (int)(u - k * nlc), src, dst, a.lay.page_size);
  }
}

cudaError_t list_pages(const PageArgs &a, bool ranks, cudaStream_t s) {
  const int chunks = page_chunks(a.num_pages);
  if (chunks > kOwnCount) {
    const cudaError_t e = launch_early(page_count_kernel, dim3(chunks), kThr, 0, s, a);
    if (e != cudaSuccess) return e;
  }
  return launch_early(page_list_kernel, dim3(chunks + (ranks ? 1 : 0)), kThr, 0, s, a);
}

constexpr int kGrid = 152 * 8;  // CTAs that walk copy units: eight on each SM

}  // namespace

size_t page_workspace(long long num_pages, int n) {
  return (size_t)(n + 2) * 8 + ((size_t)page_chunks(num_pages) + 3 * (size_t)num_pages) * 4;
}

cudaError_t launch_fork(const PageArgs &a, cudaStream_t s) {
  const cudaError_t e = list_pages(a, true, s);
  if (e != cudaSuccess) return e;
  const int nlc = a.lay.L * a.lay.n_ch;
  return launch_early(fork_kernel, dim3((unsigned)a.n, (unsigned)(nlc < 65535 ? nlc : 65535)), kThr,
                      0, s, a);
}

cudaError_t launch_extend(const PageArgs &a, cudaStream_t s) {
  const cudaError_t e = list_pages(a, true, s);
  if (e != cudaSuccess) return e;
  return launch_early(extend_kernel, dim3((unsigned)a.n), kThr, 0, s, a);
}

cudaError_t launch_free(const PageArgs &a, cudaStream_t s) {
  return launch_early(free_kernel, dim3((unsigned)a.n), kThr, 0, s, a);
}

cudaError_t launch_compact(const PageArgs &a, cudaStream_t s) {
  const cudaError_t e = list_pages(a, false, s);
  if (e != cudaSuccess) return e;
  return launch_early(compact_kernel, dim3(kGrid), kThr, 0, s, a);
}

cudaError_t launch_copy_pages(const PageArgs &a, cudaStream_t s) {
  const long long units = (long long)a.n * a.lay.L * a.lay.n_ch;
  return launch_early(copy_kernel, dim3((unsigned)(units < kGrid ? units : kGrid)), kThr, 0, s, a);
}

}  // namespace kamera
