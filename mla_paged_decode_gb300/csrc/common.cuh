// Shared definitions of the MLA paged-decode kernels (sm_103a).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

namespace mla {

constexpr int kDqk = 576;        // 512 latent + 64 rope
constexpr int kDv = 512;         // latent = value
constexpr int kPage = 64;        // tokens per cache page
constexpr int kTile = 64;        // partition-local tokens per KV tile
constexpr int kSlotHeads = 64;   // heads per split-partial slot in the workspace
// Schedule cost of a request piece's boundary (its Q, the pipeline refill,
// the epilogue), in tiles: an e4m3 piece also splits its Q into two terms,
// and its tiles are shorter, so its boundary weighs more tiles (each value
// the measured best of 4, 8 and 12 on that dtype's workloads).
constexpr int kPieceCost = 4;
constexpr int kPieceCostE4m3 = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Device error word bits (workspace header).
constexpr int kErrBadPage = 1;
constexpr int kErrBadLen = 2;
constexpr int kErrTimeout = 4;   // a bounded wait inside the kernel gave up

// Workspace layout (all offsets multiples of 256 bytes):
//   [0, 256)                 header: int32 error word
//   info                     int4[num_virtual_requests]: {first CTA, splits, its slot}
//   slot lse                 fp32[2 * grid][kSlotHeads]   (base-2 lse of a split)
//   slot out                 fp32[2 * grid][kSlotHeads][512] (normalised split output)
struct WorkspaceLayout {
  size_t info, slot_lse, slot_out, total;
};

__host__ __device__ constexpr size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

__host__ __device__ constexpr WorkspaceLayout workspace_layout(int num_virtual, int grid) {
  return WorkspaceLayout{
      256, align256(256 + 16 * size_t(num_virtual)),
      align256(align256(256 + 16 * size_t(num_virtual)) +
               sizeof(float) * size_t(2 * grid) * kSlotHeads),
      align256(align256(align256(256 + 16 * size_t(num_virtual)) +
                        sizeof(float) * size_t(2 * grid) * kSlotHeads) +
               sizeof(float) * size_t(2 * grid) * kSlotHeads * kDv)};
}

struct DecodeParams {
  const __nv_bfloat16 *q;     // [B, 1, H, 576]
  const void *kv;             // [num_pages, 64, 576] bf16 or e4m3
  const int32_t *block_table; // [B, max_pages]
  const int32_t *seq_lens;    // [B]
  __nv_bfloat16 *out;         // [B, 1, H, 512]
  float *lse;                 // [B, 1, H]
  unsigned char *ws;          // workspace base
  WorkspaceLayout wl;
  int batch, heads, head_groups, heads_per_group;
  int num_pages, max_pages;
  int part_id, num_parts;
  // All partitions in one launch (tensor-core kernel only): output row bv of
  // `batch` = num_parts * req_batch rows is request bv % req_batch of
  // partition bv / req_batch; out / lse are then [P, B, ...].  Otherwise
  // fused = 0 and req_batch = batch.
  int fused = 0, req_batch = 0;
  // fused only: the partitions' LSE combine, written by the merge kernel
  // ([B, rows, 512] bf16 and, optionally, [B, rows] fp32 in the lse base)
  __nv_bfloat16 *comb_out = nullptr;
  float *comb_lse = nullptr;
  // Query tokens per request (tensor-core kernel only; 1 elsewhere): the
  // `heads` rows of a request are then q_len x q_heads, row i * q_heads + h
  // for query token i, and token i of T sees the global tokens t < L - T + i + 1.
  int q_len = 1, q_heads = 0;
  // Owner mask (tensor-core kernel only): when own_parts > num_parts the call
  // computes partition own_part of own_parts through the gather of partition
  // part_id = own_part mod num_parts of num_parts (num_parts divides both 8
  // and own_parts), and the softmax drops every gathered token whose global
  // index is not own_part mod own_parts.  Otherwise own_parts = 0.
  int own_parts = 0, own_part = 0;
  // Strided gather (tensor-core kernel, P in {3, 5, 6, 7}):
  // partition r's rows of page lp are y0 + kP (y0 = (r - 64 lp)
  // mod P), landed by TMA with a traversal stride of P in atoms of 8 rows,
  // `apg` atoms per page.  The tile walk then runs over slots: page lp holds
  // slots [8 apg lp, 8 apg (lp + 1)), slot 8 apg lp + k is row y0 + kP when
  // that row is below 64 (else the slot is empty), and a request's length in
  // slots ends just past its last owned token.  Otherwise strided = 0.
  int strided = 0, apg = 0;
  int s_q63 = 0, s_r63 = 0, s_c64 = 0;  // strided: 63 / P, 63 mod P, 64 mod P
  // Views (tensor-core kernel, MULTI >= 3; see ViewReq): 0 none, kViewWindow
  // (window, sinks) or kViewShared (groups of requests with shared pages;
  // `prefix_blocks` bounds the 64-row blocks of all groups).
  int view = 0;
  int window = 0, sinks = 0;
  const int32_t *group_starts = nullptr;  // [num_groups + 1]
  const int32_t *shared_pages = nullptr;  // [num_groups]
  int2 *group_table = nullptr;            // [num_groups], in the workspace (see fill_group_table)
  int num_groups = 0, prefix_blocks = 0;
  // Chunks (kViewChunk; pair kernel): request b's query tokens are tokens
  // chunk_starts[b] .. chunk_starts[b + 1] of the `chunk_tokens` tokens of Q, q_heads
  // rows each, and the last of its seq_lens[b] cached ones.
  const int32_t *chunk_starts = nullptr;  // [batch + 1]
  int chunk_tokens = 0;
  // Shared pages, or windows, attended by the pair kernel (csrc/decode_pair.cu) in
  // pair_blocks blocks of 128 rows on `pairs` CTA pairs; prefix_blocks is then 0.
  // The last pair_tails of them are the requests' own pages (0: left to the
  // other kernel).
  int pair_blocks = 0, pair_tails = 0, pairs = 0;
  int kv_e4m3;
  float kv_scale;             // 1 for bf16
  float score_scale_log2;     // sm_scale * log2(e): scores kept in the base-2 domain
  int lse_base2;              // output lse in base 2 (else natural)
};

// ---------------------------------------------------------------- host: per-device set-up

// Raises one kernel's dynamic shared-memory limit on each device the first
// time it is launched there.  Thread-safe: host threads that launch on the
// same device for the first time at once take a lock, and later launches
// read only an atomic flag.  One static instance per kernel.
struct SmemLimitOnce {
  std::atomic<uint64_t> done{0};  // bit d: set on device d
  std::mutex mu;
  template <typename Kernel>
  cudaError_t ensure(Kernel kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    const uint64_t bit = 1ull << dev;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    std::lock_guard<std::mutex> lk(mu);
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

// ---------------------------------------------------------------- partition rule

// Tokens owned by partition r of P out of a global length L: t < L, t mod P == r.
__host__ __device__ __forceinline__ int local_len(int L, int P, int r) {
  return L / P + (r < L % P ? 1 : 0);
}

// Virtual request v -> its output row b and head group g: group-major,
// v = g * batch + b.  The split schedule cuts the concatenated tile sequence
// of all virtual requests into equal cost ranges, one per CTA; in this order
// the head groups of a request (or the query-token groups of a request with
// several query tokens) sit at the same offset of head_groups equal stretches
// of that sequence, so CTAs c, c + G / head_groups, ... walk the same pages
// at the same time and the later reads of a page find it in L2: the cache
// is read from HBM once for all rows of a request.
__host__ __device__ __forceinline__ int vreq_row(const DecodeParams &p, int v) { return v % p.batch; }
__host__ __device__ __forceinline__ int vreq_group(const DecodeParams &p, int v) { return v / p.batch; }
__host__ __device__ __forceinline__ int vreq_index(const DecodeParams &p, int b, int g) {
  return g * p.batch + b;
}

// Output row bv -> the input request it reads (q, block table, length) and
// the partition it attends for.
__device__ __forceinline__ int req_of(const DecodeParams &p, int bv) {
  return p.fused ? bv % p.req_batch : bv;
}
__device__ __forceinline__ int part_of(const DecodeParams &p, int bv) {
  return p.fused ? bv / p.req_batch : p.part_id;
}

// Pages of the longest request: lengths and their sums with a page stay below 2^31,
// however wide the block table is.
constexpr int kMaxRequestPages = (1 << 25) - 1;

// Clamp a global length to what the block table can hold; flag a bad one.
__device__ __forceinline__ int checked_len(const DecodeParams &p, int b, int *err) {
  int L = p.seq_lens[b];
  int cap = min(p.max_pages, kMaxRequestPages) * kPage;
  if (L < 0 || L > cap) {
    if (err) atomicOr(err, kErrBadLen);
    L = L < 0 ? 0 : cap;
  }
  return L;
}

// Global tokens visible to row `row` of a request of length L, and to the
// rows of head group g (its last row sees the most).
__device__ __forceinline__ int row_len(const DecodeParams &p, int L, int row) {
  return p.q_len <= 1 ? L : max(0, L - p.q_len + row / p.q_heads + 1);
}
__device__ __forceinline__ int group_len(const DecodeParams &p, int L, int g) {
  return p.q_len <= 1 ? L : row_len(p, L, min(p.heads, (g + 1) * p.heads_per_group) - 1);
}

// Strided gather: the first row partition `part` owns in logical page lp,
// and the slots of a request of length L (see DecodeParams::strided).
__host__ __device__ __forceinline__ int strided_y0(int part, int P, int lp) {
  return ((part - (kPage % P) * (lp % P)) % P + P) % P;
}
__host__ __device__ __forceinline__ int strided_slots(int L, int P, int r, int apg) {
  const int n = local_len(L, P, r);
  if (n == 0) return 0;
  const int t_last = r + P * (n - 1);
  const int lp = t_last / kPage;
  const int y0 = strided_y0(r, P, lp);
  return 8 * apg * lp + (t_last - kPage * lp - y0) / P + 1;
}
// The slots of consecutive tiles that hold a row (below 64 within its page),
// walked atom by atom without a division: page lp + 1 starts at
// y0 - (64 mod P) (mod P), and a page with start y0 holds 63 / P + 1 rows of
// the partition, one fewer when y0 > 63 mod P.
struct StridedMask {
  int ap, y0;  // the next atom: its index within its page, its page's first row
  __device__ void start(const DecodeParams &p, int part, long long t) {
    const int a = int(8 * t), lp = a / p.apg;
    ap = a - lp * p.apg;
    y0 = strided_y0(part, p.num_parts, lp);
  }
  // bit i set when slot i of the next tile holds a row; moves to the tile after
  __device__ __forceinline__ unsigned long long next(const DecodeParams &p) {
    unsigned long long m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int rows = p.s_q63 + 1 - (y0 > p.s_r63 ? 1 : 0);
      const int v = min(8, max(0, rows - 8 * ap));
      m |= ((1ull << v) - 1ull) << (8 * k);
      if (++ap == p.apg) {
        ap = 0;
        y0 -= p.s_c64;
        if (y0 < 0) y0 += p.num_parts;
      }
    }
    return m;
  }
};

// ---------------------------------------------------------------- views
//
// A view is what a 64-row block of queries attends to: `tiles` pages of one
// block-table row, first the `nsink` pages from page 0, then those from page
// `first` on, up to token `end`.
//
// Window: virtual request v is head group v / B of request v mod B.  The
// block sees its sinks and the pages from the first token of its first
// query's window to its last query.
//
// Shared: the first prefix_blocks virtual requests are 64-row blocks of the
// groups' rows over the shared pages, the others (request, head group) pairs
// over the request's own pages.  Group g's blocks have ids block_base(g) and
// up: rows / 64 rounded down at its first row, plus g, which leaves every
// group at least the ids it needs (ceil(m / 64) <= floor((a + m) / 64) -
// floor(a / 64) + 1); ids between are empty.
//
// Chunk: 128-row blocks of the requests' query tokens (ragged) over the tokens up to
// the block's last query.  Request b's blocks have ids floor(its first row / 128) + b
// and up, as the groups' blocks above.
constexpr int kViewWindow = 1, kViewShared = 2, kViewChunk = 3;

struct ViewReq {
  int tiles = 0;
  int row0 = 0, rows = 0;  // first row of q / out / lse, rows of the block
  int req = 0;             // block-table row
  int first = 0, nsink = 0;
  int end = 0;             // tokens from here on are not seen by any row
  int lead = 0;            // window: tokens below are not seen, sinks aside
  bool unsure = false;     // shared pages: the group's table is needed (see shared_view)
  __device__ __forceinline__ int page(long long t) const {
    return t < nsink ? int(t) : int(t) - nsink + first;
  }
  // rows of page t of the view that some row sees, as bits
  __device__ __forceinline__ unsigned long long seen_rows(const DecodeParams &p, int t) const {
    const int base = page(t) * kPage;
    auto below = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull; };
    const unsigned long long sunk = below(p.sinks - base);
    return t < nsink ? sunk : (below(end - base) & ~below(lead - base)) | (sunk & below(end - base));
  }
  // tokens of tile t that some row sees, counted from the tile's start
  __device__ __forceinline__ int seen(const DecodeParams &p, long long t) const {
    const int base = page(t) * kPage;
    return t < nsink ? min(kPage, p.sinks - base) : min(kPage, end - base);
  }
};

__device__ __forceinline__ int group_start(const DecodeParams &p, int g) {
  return min(max(p.group_starts[g], 0), p.batch);
}
template <int R = 64>
__device__ __forceinline__ int block_base(const DecodeParams &p, int g) {
  return int((long long)group_start(p, g) * p.heads / R) + g;
}
__device__ __forceinline__ int group_shared_pages(const DecodeParams &p, int g) {
  return min(max(p.shared_pages[g], 0), min(p.max_pages, kMaxRequestPages));
}
// The last group that starts at or before request b.
__device__ __forceinline__ int group_of_request(const DecodeParams &p, int b) {
  int lo = 0, hi = p.num_groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.group_starts[mid] <= b) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The pages that the requests of each group attend to together, and the request whose
// row names them: {pages, request}.  Commonly the first request of a group reaches
// all its shared pages, and no table is needed.  Where it does not (it has ended, or
// is shorter), they are read from a request that reaches them all, or else from the
// longest, and then only the pages that it fills count as shared: its last page is
// left to the requests' own, where rows that nobody sees may hold anything.
//
// Every CTA that meets such a group fills the table for itself, a warp a group, and
// makes its schedule anew; all of them write the same words.  (A search by each view
// instead, with a group's first half ended: 1,024 requests x 16 heads 509 us against
// 134 with none ended, 512 x 128 10,190 against 377, as most views of a long batch
// searched through half of it; and its loop in every role cost the other calls up
// to 9 %.)
static __device__ __noinline__ void fill_group_table(const DecodeParams &p) {
  const int lane = threadIdx.x & 31;
  for (int g = int(threadIdx.x) >> 5; g < p.num_groups; g += int(blockDim.x) >> 5) {
    const int b0 = group_start(p, g), b1 = group_start(p, g + 1), pages = group_shared_pages(p, g);
    int len = 0, who = b0;
    for (int b = b0; b < b1; b += 128) {
      int L[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) L[u] = b + lane + 32 * u < b1 ? checked_len(p, b + lane + 32 * u, nullptr) : 0;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (L[u] > len) len = L[u], who = b + lane + 32 * u;
      if (__any_sync(0xffffffffu, len >= pages * kPage)) break;
    }
    for (int o = 16; o; o >>= 1) {  // the longest; the first of equals
      const int l = __shfl_xor_sync(0xffffffffu, len, o), b = __shfl_xor_sync(0xffffffffu, who, o);
      if (l > len || (l == len && b < who)) len = l, who = b;
    }
    if (lane == 0) p.group_table[g] = make_int2(min(pages, len / kPage), who);
  }
}

// Blocks of R rows of a batch with shared pages: block v < `blocks` of a group's rows
// over its shared pages, or (OWN) block v - blocks of the requests' rows over their
// own pages.  `groups`: the table, or null where it is not needed; the view then says
// (`unsure`) if it is.
template <int R, bool OWN>
__device__ __forceinline__ ViewReq shared_view(const DecodeParams &p, int v, int blocks, const int2 *groups) {
  ViewReq r;
  const bool own = OWN && v >= blocks;
  const int u = v - blocks, b = own ? u % p.batch : 0, L = own ? checked_len(p, b, nullptr) : 0;
  if (own && L == 0) return r;  // (roles walk over runs of ended requests one by one)
  int lo = 0, hi = p.num_groups - 1;  // the last group that starts at or before the block, or request b
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (own ? p.group_starts[mid] <= b : block_base<R>(p, mid) <= v) lo = mid;
    else hi = mid - 1;
  }
  const int b0 = group_start(p, lo), b1 = group_start(p, lo + 1);
  int2 shared = make_int2(0, b0);
  if (groups) shared = groups[lo];
  else shared.x = group_shared_pages(p, lo);
  if (own) {
    const int g = u / p.batch;
    r.row0 = b * p.heads + R * g;
    r.rows = min(R, p.heads - R * g);
    r.end = row_len(p, L, min(p.heads, R * (g + 1)) - 1);
    r.req = b;
    r.first = shared.x;
    r.tiles = max(0, (r.end + kPage - 1) / kPage - shared.x);
    r.unsure = !groups && L < shared.x * kPage;
  } else {
    const int k = v - block_base<R>(p, lo), rows = (b1 - b0) * p.heads;
    if (k < 0 || R * k >= rows) return r;
    r.row0 = b0 * p.heads + R * k;
    r.rows = min(R, rows - R * k);
    r.req = shared.y;
    r.tiles = shared.x;
    r.end = shared.x * kPage;
    r.unsure = !groups && checked_len(p, b0, nullptr) < r.end;
  }
  return r;
}

// Block u / B of R rows of request u mod B, through its window and its sinks.
template <int R = 64>
__device__ __forceinline__ ViewReq window_block(const DecodeParams &p, int u) {
  ViewReq r;
  const int b = u % p.batch, g = u / p.batch;
  r.req = b;
  r.row0 = b * p.heads + R * g;
  r.rows = min(R, p.heads - R * g);
  const int L = checked_len(p, b, nullptr);
  r.end = row_len(p, L, min(p.heads, R * (g + 1)) - 1);
  if (r.end == 0) return r;
  // the block's first query sits at position L - T + R g / q_heads
  r.lead = max(0, L - p.q_len + (R * g) / p.q_heads + 1 - p.window);
  r.first = r.lead / kPage;
  r.nsink = min((p.sinks + kPage - 1) / kPage, r.first);
  r.tiles = r.nsink + (r.end + kPage - 1) / kPage - r.first;
  return r;
}

// First query token of request b of a chunked batch; the tokens from chunk_start(batch)
// on are nobody's.
__device__ __forceinline__ int chunk_start(const DecodeParams &p, int b) {
  return min(max(p.chunk_starts[b], 0), p.chunk_tokens);
}
template <int R>
__device__ __forceinline__ int chunk_base(const DecodeParams &p, int b) {
  return int((long long)chunk_start(p, b) * p.q_heads / R) + b;
}
// Block v of R rows of a chunked batch, of request lo.  (Starts that fall are cut to none
// or to rows of other requests, never to rows outside Q.)
template <int R>
__device__ __forceinline__ ViewReq chunk_block_of(const DecodeParams &p, int v, int lo) {
  ViewReq r;
  r.req = lo;
  const int s0 = chunk_start(p, lo), n = chunk_start(p, lo + 1) - s0;
  const long long k = v - chunk_base<R>(p, lo), rows = (long long)n * p.q_heads;
  if (k < 0 || R * k >= rows) return r;
  r.row0 = int((long long)s0 * p.q_heads + R * k);
  r.rows = int(min((long long)R, rows - R * k));
  r.end = max(0, checked_len(p, lo, nullptr) - n + (int(R * k) + r.rows - 1) / p.q_heads + 1);
  r.tiles = (r.end + kPage - 1) / kPage;
  return r;
}

// The last request whose blocks start at or before block v, and the block.
template <int R>
__device__ __forceinline__ int chunk_request(const DecodeParams &p, int v) {
  int lo = 0, hi = p.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (chunk_base<R>(p, mid) <= v) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
template <int R>
__device__ __forceinline__ ViewReq chunk_block(const DecodeParams &p, int v) {
  return chunk_block_of<R>(p, v, chunk_request<R>(p, v));
}

// What the roles of a CTA start from: the first piece's view, and the groups' table or
// null (in shared memory: held in registers it made the softmax of an e4m3 cache spill).
struct ViewStart {
  ViewReq view;
  const int2 *groups;
};

// MULTI: 3 windows, 4 shared pages.
template <int MULTI>
__device__ __forceinline__ ViewReq view_req(const DecodeParams &p, int v, const int2 *groups) {
  if constexpr (MULTI == 3) return window_block(p, v);
  else return shared_view<64, true>(p, v, p.prefix_blocks, groups);
}

// What row `row` (of all rows) of a block sees: tokens below `hi`, and of
// those the ones from `lo` on or below the sinks.
struct RowView {
  int lo, hi;
};
template <bool WINDOW>
__device__ __forceinline__ RowView row_view(const DecodeParams &p, const ViewReq &r, int row) {
  const int b = min(row / p.heads, p.batch - 1);
  const int pos = checked_len(p, b, nullptr) - p.q_len + (row - b * p.heads) / p.q_heads;
  return RowView{WINDOW ? max(0, pos + 1 - p.window) : 0, min(max(0, pos + 1), r.end)};
}

// The same of a row of a chunk's block.
__device__ __forceinline__ RowView chunk_row_view(const DecodeParams &p, const ViewReq &r, int row) {
  const int s0 = chunk_start(p, r.req), n = chunk_start(p, r.req + 1) - s0;
  const int token = int((row - (long long)s0 * p.q_heads) / p.q_heads);
  return RowView{0, min(max(0, checked_len(p, r.req, nullptr) - n + token + 1), r.end)};
}

// Owned tokens of virtual request v (its group's widest row).
// MULTI: rows may differ in the tokens they see (several query tokens, or an
// owner mask); MULTI == 2: the strided gather, whose lengths count slots.  A
// compile-time switch, so that each kernel keeps only its own length rule.
template <int MULTI = 0>
__device__ __forceinline__ int request_len(const DecodeParams &p, int v, int *err) {
  int bv = vreq_row(p, v);
  int L = checked_len(p, req_of(p, bv), err);
  if (MULTI) L = group_len(p, L, vreq_group(p, v));
  // under an owner mask, a request the real partition owns no token of is
  // empty (the neutral pair), however many the gathered partition holds
  if (MULTI && p.own_parts > p.num_parts && local_len(L, p.own_parts, p.own_part) == 0) return 0;
  // strided gather (MULTI == 2): the length in slots
  if (MULTI == 2) return strided_slots(L, p.num_parts, part_of(p, bv), p.apg);
  return local_len(L, p.num_parts, part_of(p, bv));
}

// Kernels whose rows may differ in the tokens they see: several query
// tokens per request, or an owner mask.
__host__ __device__ __forceinline__ bool multi_rows(const DecodeParams &p) {
  return p.q_len > 1 || p.own_parts > p.num_parts || p.strided;
}

// Owner mask of the gathered partition's tiles.  Local token j of partition
// part_id of num_parts is global token part_id + j * num_parts; with
// Q = own_parts / num_parts it belongs to own_part when j = c mod Q,
// c = own_part / num_parts.  bits(t): bit i set when local token 64t + i is
// owned.
struct OwnerMask {
  unsigned long long comb;  // bits 0, Q, 2Q, ... below 64
  int q, c;
  __device__ __forceinline__ unsigned long long bits(long long t) const {
    return comb << int(((long long)c - (64 * t) % q + q) % q);
  }
};

__device__ inline OwnerMask owner_mask_of(const DecodeParams &p) {
  OwnerMask o;
  o.q = p.own_parts / p.num_parts;
  o.c = p.own_part / p.num_parts;
  o.comb = 0;
  for (int j = 0; j < 64; j += o.q) o.comb |= 1ull << j;
  return o;
}

template <int MULTI = 0>
__device__ __forceinline__ int request_tiles(const DecodeParams &p, int v) {
  return (request_len<MULTI>(p, v, nullptr) + kTile - 1) / kTile;
}

// ---------------------------------------------------------------- split schedule
//
// Cost-weighted stream-K split of the concatenated tile sequence of all
// virtual requests v = g * batch + b (tiles_v = ceil(local_len / 64)).
// Every request with tiles costs tiles_v + PC: the extra units stand for the
// per-piece work (Q load, pipeline refill, epilogue), so a CTA whose range
// crosses a request boundary gets fewer tiles.  Request v occupies cost units
// [P_v, P_v + tiles_v) followed by a gap of PC; C = total cost.  PC is a
// compile-time constant of each kernel variant (kPieceCost, or kPieceCostE4m3
// for the e4m3 tensor-core variants): read from the launch parameters instead
// it measured slower.
// G_eff = min(gridDim.x, C) CTAs; CTA c owns the tiles whose cost lies in
// [c*C/G_eff, (c+1)*C/G_eff).  A request crossing a boundary is split; each
// split writes a normalised fp32 partial into slot 2c (the CTA's first
// request) or 2c+1 (its last); the request's first CTA records {itself,
// split count, its slot} and a second kernel merges the splits.

// Virtual requests of a launch.
template <int MULTI = 0>
__device__ __forceinline__ int virtual_requests(const DecodeParams &p) {
  return p.batch * p.head_groups + (MULTI == 4 ? p.prefix_blocks : 0);
}

struct CtaRange {
  long long start, end;   // cost range of this CTA
  long long total;        // C
  int g_eff;              // CTAs that own cost units
  int v_begin;            // first virtual request with tiles in range
  long long p_begin;      // cost start of v_begin
};

__device__ __forceinline__ long long sched_start(long long c, long long C, int g_eff) {
  return c * C / g_eff;
}

// Largest c with sched_start(c) <= x.
__device__ __forceinline__ int sched_owner(long long x, long long C, int g_eff) {
  return int(((x + 1) * g_eff - 1) / C);
}

// The same two with a 32-bit division where the product allows it (a 64-bit one
// costs hundreds of cycles; views and the pair kernel start and end pieces often).
__device__ __forceinline__ long long sched_start_short(long long c, long long C, int g_eff) {
  const long long x = c * C;
  return x >> 32 ? x / g_eff : (long long)(uint32_t(x) / uint32_t(g_eff));
}
__device__ __forceinline__ int sched_owner_short(long long x, long long C, int g_eff) {
  const long long y = (x + 1) * g_eff - 1;
  return y >> 32 || C >> 32 ? int(y / C) : int(uint32_t(y) / uint32_t(C));
}

__device__ __forceinline__ long long request_cost(int tiles, int piece_cost) {
  return tiles > 0 ? tiles + piece_cost : 0;
}

// Block-wide: computes worker `idx`'s range of V requests over `workers`
// workers.  All threads must call it.  `scratch` needs blockDim.x / 32 + 1
// long longs of shared memory.  ONCE: with at most a request per thread,
// tiles_of runs once and a single scan finds the range.
template <int PC, bool ONCE, typename Tiles>
__device__ __forceinline__ void schedule_range(int V, int idx, int workers, Tiles tiles_of, CtaRange *r,
                                               long long *scratch) {
  const int tid = threadIdx.x, nw = blockDim.x / 32, lane = tid & 31, warp = tid >> 5;
  if constexpr (ONCE) {
    if (V <= int(blockDim.x)) {  // a request per thread: one scan gives the total and every start
      const int tiles = tid < V ? tiles_of(tid) : 0;
      const long long cst = request_cost(tiles, PC);
      long long incl = cst;
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) scratch[warp] = incl;
      if (tid == 0) r->v_begin = V;
      __syncthreads();
      long long before = 0, C = 0;
      for (int w = 0; w < nw; ++w) {
        if (w < warp) before += scratch[w];
        C += scratch[w];
      }
      const int g_eff = int(C < (long long)workers ? C : (long long)workers);
      const bool has = g_eff > 0 && idx < g_eff;
      const long long start = has ? sched_start_short(idx, C, g_eff) : 0;
      const long long excl = before + incl - cst;
      if (tid == 0) {
        r->total = C;
        r->g_eff = g_eff;
        r->start = start;
        r->end = has ? sched_start_short(idx + 1, C, g_eff) : 0;
      }
      if (has && tiles > 0 && excl + tiles > start && excl - PC <= start) {
        r->v_begin = tid;
        r->p_begin = excl;
      }
      __syncthreads();
      return;
    }
  }
  // pass 1: total cost
  long long mine = 0;
  for (int v = tid; v < V; v += blockDim.x) mine += request_cost(tiles_of(v), PC);
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) scratch[warp] = mine;
  __syncthreads();
  if (tid == 0) {
    long long C = 0;
    for (int w = 0; w < nw; ++w) C += scratch[w];
    r->total = C;
    r->g_eff = int(C < (long long)workers ? C : (long long)workers);
    r->v_begin = V;
    r->p_begin = 0;
    if (r->g_eff > 0 && idx < r->g_eff) {
      r->start = sched_start(idx, C, r->g_eff);
      r->end = sched_start(idx + 1, C, r->g_eff);
    } else {
      r->start = r->end = 0;
    }
  }
  __syncthreads();
  const long long start = r->start, end = r->end;
  if (start >= end) return;
  // pass 2: the first request whose tiles end after `start` (chunked block
  // scan of the costs); its predecessor ends at P_v - PC
  long long base = 0;
  for (int v0 = 0; v0 < V; v0 += blockDim.x) {
    int v = v0 + tid;
    const int tiles = v < V ? tiles_of(v) : 0;
    const long long cst = request_cost(tiles, PC);
    long long incl = cst;
    for (int o = 1; o < 32; o <<= 1) {
      long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    long long wbase = 0, chunk = 0;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) wbase += scratch[w];
      chunk += scratch[w];
    }
    const long long excl = base + wbase + incl - cst;
    if (tiles > 0 && excl + tiles > start && excl - PC <= start) {
      r->v_begin = v;
      r->p_begin = excl;
    }
    base += chunk;
    __syncthreads();
    if (r->v_begin < V) break;  // uniform: read after the barrier
  }
  __syncthreads();
}

// The same for shared pages, tiles_of(v, groups, &unsure); fills the groups' table when one of
// them is unsure without it.  Returns the table or null, the same for all threads.
template <int PC, typename Tiles>
__device__ __forceinline__ const int2 *schedule_views(const DecodeParams &p, int V, int idx, int workers,
                                                      Tiles tiles_of, CtaRange *r, long long *scratch) {
  const int2 *groups = nullptr;
#pragma unroll 1
  for (;;) {
    bool unsure = false;
    schedule_range<PC, true>(V, idx, workers, [&](int v) { return tiles_of(v, groups, &unsure); }, r, scratch);
    if (groups || !__syncthreads_or(unsure)) return groups;
    fill_group_table(p);
    __syncthreads();
    groups = p.group_table;
  }
}

// This CTA's range of a launch whose workers are its CTAs.
template <int MULTI = 0, int PC = kPieceCost>
__device__ inline void cta_schedule(const DecodeParams &p, CtaRange *r, long long *scratch) {
  schedule_range<PC, false>(virtual_requests<MULTI>(p), int(blockIdx.x), int(gridDim.x),
                            [&](int v) { return request_tiles<MULTI>(p, v); }, r, scratch);
}

// ---------------------------------------------------------------- conversions

__device__ __forceinline__ float bf16_bits_to_float(uint16_t b) {
  return __uint_as_float(uint32_t(b) << 16);
}

// The larger of two, NaN when either is (fmaxf drops a NaN).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two OCP e4m3 bytes -> two exact f16 values (hardware conversion).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t two) {
  uint32_t r;
  asm("{ cvt.rn.f16x2.e4m3x2 %0, %1; }" : "=r"(r) : "h"(two));
  return r;
}

// Two floats -> two OCP e4m3 bytes, round to nearest even, saturated to the
// finite range (hardware conversion): `lo` in the low byte.
__device__ __forceinline__ uint16_t float2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("{ cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2; }" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two floats -> two OCP e5m2 bytes (hardware conversion, RNE, saturated):
// `lo` in the low byte.
__device__ __forceinline__ uint16_t float2_to_e5m2x2(float lo, float hi) {
  uint16_t r;
  asm("{ cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2; }" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e5m2 bytes -> two exact floats (through the hardware f16 conversion).
__device__ __forceinline__ float2 e5m2x2_to_float2(uint16_t two) {
  uint32_t h;
  asm("{ cvt.rn.f16x2.e5m2x2 %0, %1; }" : "=r"(h) : "h"(two));
  __half2 hh = *reinterpret_cast<__half2 *>(&h);
  return __half22float2(hh);
}

// The largest |x| of eight bf16 values, as two 16-bit lanes of bits without the
// sign (which are ordered like the magnitudes).
__device__ __forceinline__ uint32_t largest_bf16x8(uint4 v) {
  return __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
}

// 2^k with which q enters as two e4m3 terms: the largest |q|, as bf16 bits `mx`, comes
// to lie in [2^7, 2^8).  An Inf or NaN keeps k = 0.
__device__ __forceinline__ float q_scale(uint32_t mx) {
  const int k = mx < 0x7f80u ? min(126, max(-126, 134 - int(mx >> 7))) : 0;
  return __int_as_float((127 + k) << 23);
}
// The same for a scale that one row has to itself: a row with an Inf or a NaN
// turns into NaN (saturated to e4m3's range, an Inf would read as a number).
__device__ __forceinline__ float row_q_scale(uint32_t mx) {
  return mx < 0x7f80u ? q_scale(mx) : __int_as_float(0x7fffffff);
}
// 2^-k (of NaN: any finite number, as the scores are NaN already).
__device__ __forceinline__ float inverse_q_scale(float scale) {
  return scale == scale ? __int_as_float((254 << 23) - __float_as_int(scale)) : 1.f;
}

// 2^k of whole rows of Q that a warp holds, lane + 32 u their chunk (8 of 576 dims) in
// v[u]: nine loads are four rows.
template <int N>
__device__ __forceinline__ void row_q_scales(const uint4 (&v)[N], int lane, float (&scale)[N * 32 / 72]) {
  static_assert(N % 9 == 0, "whole rows");
  uint32_t mx[N * 32 / 72] = {};
#pragma unroll
  for (int u = 0; u < N; ++u) {
    // load u meets row 32 u / 72 and, from lane `next` on, the one after it
    const int row = 32 * u / 72, next = (row + 1) * 72 - 32 * u;
    const uint32_t x = largest_bf16x8(v[u]);
    if (next >= 32) {
      mx[row] = __vmaxu2(mx[row], x);
    } else {
      mx[row] = __vmaxu2(mx[row], lane < next ? x : 0u);
      mx[row + 1] = lane < next ? 0u : x;
    }
  }
#pragma unroll
  for (int w = 0; w < N * 32 / 72; ++w)
    scale[w] = row_q_scale(__reduce_max_sync(0xffffffffu, max(mx[w] & 0xffffu, mx[w] >> 16)));
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t two) {
  uint32_t h = e4m3x2_to_f16x2(two);
  __half2 hh = *reinterpret_cast<__half2 *>(&h);
  return __half22float2(hh);
}

}  // namespace mla
