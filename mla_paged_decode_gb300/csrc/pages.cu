// Page operations on the paged latent cache: copy, fork, allocate, free,
// compact.  A pool is described by its block table [R, W] (-1: no page), the
// requests' lengths [R] and one reference count per page (0: free).
//
// Every choice is a function of the inputs alone: new pages are the lowest
// free ids, handed out in the order of the forks (or requests), and a
// compaction pairs the k-th live page past the dense range with the k-th hole
// inside it.  Counts change through integer atomics, whose order does not
// matter.
//
// Finding free pages is a two-level count: a chunk of 1024 pages per CTA
// counts its free pages with ballots and lists them, and the kernel that
// hands pages out turns a rank into a page by a scan over the chunk counts.
// What moves is page rows, so that these calls are bound by HBM (2 bytes of
// traffic per byte moved) when pages move and by launch latency otherwise.
#include "common.cuh"
#include "pages.cuh"

namespace mla {

namespace {

constexpr int kScanThreads = 256;
constexpr int kCopyThreads = 288;
constexpr int kSliceBytes = kCopyThreads * 16 * 4;  // a quarter of a bf16 page, half of an e4m3 one
static_assert(kPage * kDqk % kSliceBytes == 0, "pages are whole slices");

// Waits for the stream's previous kernel (every kernel here is launched as
// its programmatic dependent; releasing the next one early changed nothing).
__device__ __forceinline__ void wait_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void flag(int32_t *error_word, int bit) {
  if (error_word) atomicOr(error_word, bit);
}

// Pages that hold n >= 0 tokens (n + 63 would wrap for the largest lengths and sinks).
__device__ __forceinline__ int pages_of(int n) { return n / kPage + (n % kPage ? 1 : 0); }

// Copies `bytes` (a multiple of 16) from src to dst with all threads of the
// CTA, four 16-byte loads of a thread in flight.
__device__ __forceinline__ void copy_bytes(unsigned char *dst, const unsigned char *src, int bytes) {
  const int n = bytes / 16, step = int(blockDim.x);
  const uint4 *s = reinterpret_cast<const uint4 *>(src);
  uint4 *d = reinterpret_cast<uint4 *>(dst);
  for (int i0 = threadIdx.x; i0 < n; i0 += 4 * step) {
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i0 + u * step < n) v[u] = __ldcs(s + i0 + u * step);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i0 + u * step < n) __stcs(d + i0 + u * step, v[u]);
  }
}

// Sum over the CTA (every thread gets it); `scratch` holds blockDim.x / 32 of T.
template <typename T>
__device__ __forceinline__ T block_sum(T x, T *scratch) {
  if constexpr (sizeof(T) == 4) x = __reduce_add_sync(0xffffffffu, x);
  else
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  const int nw = int(blockDim.x + 31) / 32;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
  __syncthreads();
  T total = 0;
  for (int w = 0; w < nw; ++w) total += scratch[w];
  return total;
}

// What fork k needs: its parent's length and, when the last page is partial,
// that page (a copy of it goes to a new one).
struct Fork {
  int parent, child, len, page;  // page: the partial page, -1 when there is none
  bool ok;                       // indices and length in range
  bool bad_page;                 // the partial page's entry is out of range
};

__device__ __forceinline__ Fork read_fork(const PagesTable &t, const int32_t *parents,
                                          const int32_t *children, int k) {
  Fork f{parents[k], children[k], 0, -1, false, false};
  if (f.parent < 0 || f.parent >= t.rows || f.child < 0 || f.child >= t.rows) return f;
  f.len = t.seq_lens[f.parent];
  if (f.len < 0 || (long long)f.len > (long long)t.width * kPage) return f;
  f.ok = true;
  if (f.len % kPage) {
    f.page = t.block_table[size_t(f.parent) * t.width + f.len / kPage];
    f.bad_page = f.page < 0 || f.page >= t.num_pages;
    if (f.bad_page) f.page = -1;
  }
  return f;
}

// The first CTAs take a chunk each: the number of its free pages, and their
// ids in ascending order.  For a fork, further CTAs count the forks that need
// a page, kForkBlock at a time.
constexpr int kForkBlock = kScanThreads;

__global__ void __launch_bounds__(kScanThreads)
    pages_scan_kernel(PagesTable t, PagesWorkspace ws, const int32_t *parents, const int32_t *children, int n_forks) {
  wait_previous();
  __shared__ int s_warp[kScanThreads / 32];
  const int32_t *ref_counts = t.ref_counts;
  const int num_pages = t.num_pages;
  if (int(blockIdx.x) >= pages_chunks(num_pages)) {
    const int blk = int(blockIdx.x) - pages_chunks(num_pages), k = blk * kForkBlock + int(threadIdx.x);
    const int total = block_sum(k < n_forks && read_fork(t, parents, children, k).page >= 0 ? 1 : 0, s_warp);
    if (threadIdx.x == 0) ws.fork_count[blk] = total;
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = blockIdx.x * kPagesChunk + warp * 128;
  uint32_t mask[4];
  int n = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int id = first + 32 * j + lane;
    mask[j] = __ballot_sync(0xffffffffu, id < num_pages && ref_counts[id] == 0);
    n += __popc(mask[j]);
  }
  if (lane == 0) s_warp[warp] = n;
  __syncthreads();
  int at = 0, total = 0;
  for (int w = 0; w < kScanThreads / 32; ++w) {
    if (w < warp) at += s_warp[w];
    total += s_warp[w];
  }
  if (threadIdx.x == 0) ws.chunk_free[blockIdx.x] = total;
  int32_t *list = ws.free_list + size_t(blockIdx.x) * kPagesChunk;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if ((mask[j] >> lane) & 1u) list[at + __popc(mask[j] & ((1u << lane) - 1u))] = first + 32 * j + lane;
    at += __popc(mask[j]);
  }
}

// The page of rank `rank` among the free ones (-1 past their number), for one
// warp: lanes scan the chunk counts 32 at a time.
__device__ __forceinline__ int free_page_of_rank(const PagesWorkspace &ws, int num_chunks, int rank) {
  const int lane = threadIdx.x & 31;
  int base = 0;
  for (int c0 = 0; c0 < num_chunks; c0 += 32) {
    const int mine = c0 + lane < num_chunks ? ws.chunk_free[c0 + lane] : 0;
    int incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const int total = __shfl_sync(0xffffffffu, incl, 31);
    if (rank < base + total) {
      const uint32_t past = __ballot_sync(0xffffffffu, rank < base + incl);
      const int l = __ffs(past) - 1;
      const int excl = __shfl_sync(0xffffffffu, base + incl - mine, l);
      return ws.free_list[size_t(c0 + l) * kPagesChunk + (rank - excl)];
    }
    base += total;
  }
  return -1;
}

// ------------------------------------------------------------------ copy

__global__ void __launch_bounds__(kCopyThreads)
    pages_copy_kernel(const unsigned char *src_pool, unsigned char *dst_pool, const int32_t *src,
                      const int32_t *dst, int src_pages, int dst_pages, int page_bytes, int32_t *error_word) {
  wait_previous();
  const int s = src[blockIdx.x], d = dst[blockIdx.x];
  if (s < 0 || s >= src_pages || d < 0 || d >= dst_pages) {
    if (threadIdx.x == 0 && blockIdx.y == 0) flag(error_word, kErrPagesEntry);
    return;
  }
  const size_t off = size_t(blockIdx.y) * kSliceBytes;
  copy_bytes(dst_pool + size_t(d) * page_bytes + off, src_pool + size_t(s) * page_bytes + off, kSliceBytes);
}

// ------------------------------------------------------------------ fork

constexpr int kManyForks = 256;

// One CTA per fork and share of its page's slices: the rank of the fork's new
// page is the number of earlier forks with a partial page (the counts of the
// blocks before, and those before it in its own).  The first share also
// writes the child's row, its length and the counts.
__global__ void __launch_bounds__(kCopyThreads)
    pages_fork_kernel(PagesTable t, unsigned char *pool, int row_bytes, const int32_t *parents,
                      const int32_t *children, PagesWorkspace ws, int num_chunks, int32_t *error_word) {
  wait_previous();
  __shared__ int s_scratch[kCopyThreads / 32];
  __shared__ int s_new;
  const int k = blockIdx.x;
  const Fork f = read_fork(t, parents, children, k);
  const int used = f.page >= 0 ? (f.len % kPage) * row_bytes : 0;  // bytes of the partial page
  if (blockIdx.y > 0 && int(blockIdx.y) * kSliceBytes >= used) return;
  if (f.page >= 0) {
    const int blk = k / kForkBlock;
    int before = 0;
    for (int i = threadIdx.x; i < blk; i += blockDim.x) before += ws.fork_count[i];
    const int j = blk * kForkBlock + int(threadIdx.x);
    if (j < k) before += read_fork(t, parents, children, j).page >= 0 ? 1 : 0;
    before = block_sum(before, s_scratch);
    if (threadIdx.x < 32) {
      const int pg = free_page_of_rank(ws, num_chunks, before);
      if (threadIdx.x == 0) s_new = pg;
    }
    __syncthreads();
  }
  const int fresh = f.page >= 0 ? s_new : -1;
  const bool full_pool = f.page >= 0 && fresh < 0;
  if (blockIdx.y == 0) {
    if (threadIdx.x == 0) {
      if (!f.ok || f.bad_page) flag(error_word, kErrPagesEntry);
      if (full_pool) flag(error_word, kErrPagesFull);
    }
    if (f.ok) {
      const int held = full_pool ? 0 : f.len / kPage;
      const int32_t *from = t.block_table + size_t(f.parent) * t.width;
      int32_t *to = t.block_table + size_t(f.child) * t.width;
      for (int i = threadIdx.x; i < t.width; i += blockDim.x) {
        int e = i < held ? from[i] : -1;
        if (e < -1 || e >= t.num_pages) {
          flag(error_word, kErrPagesEntry);
          e = -1;
        }
        if (e >= 0) atomicAdd(t.ref_counts + e, 1);
        to[i] = i == held && fresh >= 0 ? fresh : e;
      }
      if (threadIdx.x == 0) {
        t.seq_lens[f.child] = full_pool ? 0 : f.len;
        if (fresh >= 0) t.ref_counts[fresh] = 1;
      }
    }
  }
  if (fresh >= 0) {
    const size_t page_bytes = size_t(kPage) * row_bytes;
    for (int off = int(blockIdx.y) * kSliceBytes; off < used; off += int(gridDim.y) * kSliceBytes)
      copy_bytes(pool + fresh * page_bytes + off, pool + f.page * page_bytes + off, min(kSliceBytes, used - off));
  }
}

// ------------------------------------------------------------------ allocate

// Pages that request b gains from old_lens[b] to new_lens[b] tokens (0 for a
// length out of range, which *bad reports, or one that does not grow).
__device__ __forceinline__ int pages_gained(const PagesTable &t, const int32_t *new_lens, int b, bool *bad) {
  const int L = t.seq_lens[b], N = new_lens[b];
  *bad = L < 0 || N < 0 || (long long)L > (long long)t.width * kPage ||
         (long long)N > (long long)t.width * kPage;
  return *bad ? 0 : max(0, pages_of(N) - pages_of(L));
}

constexpr int kAllocThreads = 128;

__global__ void __launch_bounds__(kAllocThreads)
    pages_alloc_kernel(PagesTable t, const int32_t *new_lens, PagesWorkspace ws, int num_chunks,
                       int32_t *error_word) {
  wait_previous();
  __shared__ long long s_scratch[kAllocThreads / 32];
  const int b = blockIdx.x;
  bool bad;
  const int need = pages_gained(t, new_lens, b, &bad);
  if (bad && threadIdx.x == 0) flag(error_word, kErrPagesEntry);
  if (need == 0) return;
  // what the requests before this one ask for may pass 2^31 pages, fit or not
  long long before = 0, total = 0;
  for (int j = threadIdx.x; j < b; j += blockDim.x) {
    bool skip;
    before += pages_gained(t, new_lens, j, &skip);
  }
  before = block_sum(before, s_scratch);
  for (int c = threadIdx.x; c < num_chunks; c += blockDim.x) total += ws.chunk_free[c];
  total = block_sum(total, s_scratch);
  if (before + need > total) {  // this request does not fit: it gains nothing
    if (threadIdx.x == 0) flag(error_word, kErrPagesFull);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = pages_of(t.seq_lens[b]);
  int32_t *row = t.block_table + size_t(b) * t.width;
  for (int i = warp; i < need; i += kAllocThreads / 32) {
    const int pg = free_page_of_rank(ws, num_chunks, int(before) + i);
    if (lane != 0) continue;
    if (row[first + i] != -1) {  // a page is already there: leave it
      flag(error_word, kErrPagesEntry);
      continue;
    }
    row[first + i] = pg;
    t.ref_counts[pg] = 1;
  }
}

// ------------------------------------------------------------------ free

constexpr int kFreeThreads = 128;

// One CTA per request: the pages past its new length, and those that no
// query at position new_len or later sees through (window, sinks).
__global__ void __launch_bounds__(kFreeThreads)
    pages_free_kernel(PagesTable t, const int32_t *new_lens, int window, int sinks, int32_t *error_word) {
  wait_previous();
  const int b = blockIdx.x;
  const int L = t.seq_lens[b], N = new_lens[b];
  if (N < 0 || N > L || (long long)L > (long long)t.width * kPage) {
    if (threadIdx.x == 0) flag(error_word, kErrPagesEntry);
    return;
  }
  const int keep = pages_of(N);
  // out of view: pages [lo, hi)
  const int lo = pages_of(sinks);
  const int hi = window > 0 && N >= window ? (N - window + 1) / kPage : 0;
  int32_t *row = t.block_table + size_t(b) * t.width;
  for (int i = threadIdx.x; i < t.width; i += blockDim.x) {
    if (i < keep && !(i >= lo && i < hi)) continue;
    const int e = row[i];
    if (e == -1) continue;
    row[i] = -1;
    if (e < 0 || e >= t.num_pages) {
      flag(error_word, kErrPagesEntry);
      continue;
    }
    if (atomicSub(t.ref_counts + e, 1) <= 0) {  // was free already
      atomicAdd(t.ref_counts + e, 1);
      flag(error_word, kErrPagesEntry);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) t.seq_lens[b] = N;
}

// ------------------------------------------------------------------ compact

// Small pools skip the scan: every plan CTA counts all pages itself (one
// chunk: 9.4 us a free and compact instead of 10.4; 14 chunks: 7 us slower).
constexpr int kDirectChunks = 2;

// With n live pages: a free id below n is a hole, a live id from n up a
// mover; there are m of each.  Writes the holes in order to free_list, the
// movers by their rank among the live pages to `movers` (ranks n - m .. n),
// every live page's rank to `rank` (-1 for a free one), {n, m} to `totals`, and to `remap` (when
// given) what does not move: a live page below n, and -1 for a free one.
__global__ void __launch_bounds__(kScanThreads)
    pages_compact_plan_kernel(const int32_t *ref_counts, int num_pages, PagesWorkspace ws, int num_chunks,
                              int32_t *remap) {
  wait_previous();
  __shared__ int s_scratch[kScanThreads / 32];
  __shared__ int s_warp[kScanThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int before = 0, total = 0;
  if (num_chunks <= kDirectChunks) {  // no scan ran: count the pages here
    for (int i = threadIdx.x; i < num_pages; i += blockDim.x) {
      const int x = ref_counts[i] == 0 ? 1 : 0;
      total += x;
      if (i < int(blockIdx.x) * kPagesChunk) before += x;
    }
  } else {
    for (int c = threadIdx.x; c < num_chunks; c += blockDim.x) {
      const int x = ws.chunk_free[c];
      total += x;
      if (c < int(blockIdx.x)) before += x;
    }
  }
  before = block_sum(before, s_scratch);
  total = block_sum(total, s_scratch);
  const int live = num_pages - total;
  const int first = blockIdx.x * kPagesChunk + warp * 128;
  uint32_t mask[4];
  int n = 0, below = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int id = first + 32 * j + lane;
    const bool is_free = id < num_pages && ref_counts[id] == 0;
    mask[j] = __ballot_sync(0xffffffffu, is_free);
    n += __popc(mask[j]);
    below += is_free && id < live ? 1 : 0;
  }
  if (lane == 0) s_warp[warp] = n;
  below = block_sum(below, s_scratch);
  // the CTA whose chunk holds id `live` (the last one when every page is
  // live) knows the holes: the free pages below it
  const int owner = min(live / kPagesChunk, num_chunks - 1);
  if (int(blockIdx.x) == owner && threadIdx.x == 0) {
    ws.totals[0] = live;
    ws.totals[1] = before + below;
  }
  int at = before;  // free pages before this warp's next 32 ids
  for (int w = 0; w < warp; ++w) at += s_warp[w];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int id = first + 32 * j + lane;
    const int free_before = at + __popc(mask[j] & ((1u << lane) - 1u));
    if (id < num_pages) {
      if ((mask[j] >> lane) & 1u) {
        if (id < live) ws.holes[free_before] = id;
        ws.rank[id] = -1;
        if (remap) remap[id] = -1;
      } else {
        ws.rank[id] = id - free_before;
        if (id >= live) ws.movers[id - free_before] = id;
        else if (remap) remap[id] = id;
      }
    }
    at += __popc(mask[j]);
  }
}

// Persistent: page moves in slices, then table entries, then counts and the
// movers' remap; nothing a CTA writes is read by another.
__global__ void __launch_bounds__(kCopyThreads)
    pages_compact_kernel(PagesTable t, unsigned char *pool, int page_bytes, int32_t *remap,
                         PagesWorkspace ws, int32_t *error_word) {
  wait_previous();
  const int live = ws.totals[0], m = ws.totals[1];
  const int slices = page_bytes / kSliceBytes;
  const long long moves = (long long)m * slices;
  for (long long i = blockIdx.x; i < moves; i += gridDim.x) {
    const int h = int(i / slices), s = int(i - (long long)h * slices);
    const size_t off = size_t(s) * kSliceBytes;
    copy_bytes(pool + size_t(ws.holes[h]) * page_bytes + off,
               pool + size_t(ws.movers[live - m + h]) * page_bytes + off, kSliceBytes);
  }
  const long long stride = (long long)gridDim.x * blockDim.x;
  const long long me = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long entries = (long long)t.rows * t.width;
  for (long long i = me; i < entries; i += stride) {
    const int e = t.block_table[i];
    if (e == -1) continue;
    // (asked below `live` too, where something may move into a free page)
    const int rank = e < 0 || e >= t.num_pages ? -1 : ws.rank[e];
    if (rank < 0) {  // no page, or a free one
      flag(error_word, kErrPagesEntry);
      continue;
    }
    if (e >= live) t.block_table[i] = ws.holes[rank - (live - m)];  // (a live page below stays)
  }
  for (long long h = me; h < m; h += stride) {
    const int from = ws.movers[live - m + h], to = ws.holes[h];
    t.ref_counts[to] = t.ref_counts[from];
    t.ref_counts[from] = 0;
    if (remap) remap[from] = to;
  }
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), dim3 grid, int threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t scan(const PagesTable &t, const PagesWorkspace &ws, const int32_t *parents, const int32_t *children,
                 int n, cudaStream_t stream) {
  return launch(pages_scan_kernel, dim3(pages_chunks(t.num_pages) + (n + kForkBlock - 1) / kForkBlock),
                kScanThreads, stream, t, ws, parents, children, n);
}
cudaError_t scan(const PagesTable &t, const PagesWorkspace &ws, cudaStream_t stream) {
  return scan(t, ws, nullptr, nullptr, 0, stream);
}

}  // namespace

cudaError_t launch_pages_copy(const void *src_pool, void *dst_pool, const int32_t *src, const int32_t *dst,
                              int n, int src_pages, int dst_pages, int row_bytes, int32_t *error_word,
                              cudaStream_t stream) {
  const int page_bytes = kPage * row_bytes;
  return launch(pages_copy_kernel, dim3(n, page_bytes / kSliceBytes), kCopyThreads, stream,
                static_cast<const unsigned char *>(src_pool), static_cast<unsigned char *>(dst_pool), src,
                dst, src_pages, dst_pages, page_bytes, error_word);
}

cudaError_t launch_pages_fork(const PagesTable &t, void *pool, int row_bytes, const int32_t *parents,
                              const int32_t *children, int n, const PagesWorkspace &ws, int32_t *error_word,
                              cudaStream_t stream) {
  cudaError_t e = scan(t, ws, parents, children, n, stream);
  if (e != cudaSuccess) return e;
  // few forks: a CTA per slice, so that a page is copied by four; many: one
  // CTA walks a page's slices and pays for the fork's lookups once
  const int shares = n <= kManyForks ? kPage * row_bytes / kSliceBytes : 1;
  return launch(pages_fork_kernel, dim3(n, shares), kCopyThreads, stream, t,
                static_cast<unsigned char *>(pool), row_bytes, parents, children, ws,
                pages_chunks(t.num_pages), error_word);
}

cudaError_t launch_pages_alloc(const PagesTable &t, const int32_t *new_lens, const PagesWorkspace &ws,
                               int32_t *error_word, cudaStream_t stream) {
  cudaError_t e = scan(t, ws, stream);
  if (e != cudaSuccess) return e;
  return launch(pages_alloc_kernel, dim3(t.rows), kAllocThreads, stream, t, new_lens, ws,
                pages_chunks(t.num_pages), error_word);
}

cudaError_t launch_pages_free(const PagesTable &t, const int32_t *new_lens, int window, int sinks,
                              int32_t *error_word, cudaStream_t stream) {
  return launch(pages_free_kernel, dim3(t.rows), kFreeThreads, stream, t, new_lens, window, sinks,
                error_word);
}

cudaError_t launch_pages_compact(const PagesTable &t, void *pool, int row_bytes, int32_t *remap, int grid,
                                 const PagesWorkspace &ws, int32_t *error_word, cudaStream_t stream) {
  const int chunks = pages_chunks(t.num_pages);
  cudaError_t e = chunks <= kDirectChunks ? cudaSuccess : scan(t, ws, stream);
  if (e == cudaSuccess)
    e = launch(pages_compact_plan_kernel, dim3(chunks), kScanThreads, stream,
               static_cast<const int32_t *>(t.ref_counts), t.num_pages, ws, chunks, remap);
  if (e == cudaSuccess)
    e = launch(pages_compact_kernel, dim3(grid), kCopyThreads, stream, t, static_cast<unsigned char *>(pool),
               kPage * row_bytes, remap, ws, error_word);
  return e;
}

}  // namespace mla
