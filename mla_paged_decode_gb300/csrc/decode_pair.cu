// Attention of blocks of 128 rows on CTA pairs: the rows of a group (all heads
// and query tokens of its requests) over the pages they share, the rows of a
// request over its own pages, or through its window and sinks, or the rows of a
// chunk of new tokens over all tokens up to their own.
//
// The product is [rows x 576] x [576 x tokens] and [rows x tokens] x [tokens x
// 512]: 2176 flops per row and cached token, compute bound from about 150 rows
// on.  O for 128 rows is 128 x 512 fp32, all of an SM's TMEM, so a pair of
// CTAs holds one block of 128 rows, 64 each (cta_group::2, M = 128): O takes
// 256 columns and two S buffers of 256 tokens the other 256, and each SM's
// shared memory supplies half of the B operand, so that the tensor cores see
// N = 256 (6 KB of operands per 64 cycles; one CTA at M = N = 64 reads 4 KB per
// 32 and starves).  In this shape each SM holds its 64 rows in all 128 TMEM
// lanes: lanes 0..63 columns 0 .. N/2 - 1, lanes 64..127 the others.
//
// Per tile of 256 tokens (4 pages), CTA r of the pair loads
//   K: pages 2r, 2r + 1, nine units of 64 dims x 128 tokens (its half of N);
//   V: dims 256r .. 256r + 255 of all four pages, eight units of 32 tokens
//      (its half of N of the two PV products),
// 17 units of 16 KB through one ring of seven; a page is read twice, from L2.
// (e4m3 caches: five units of 128 dims and four of a page, Q and P as two fp8
// terms each, with the arithmetic of the decode kernel's views.)
//
// Roles (384 threads): warp 0 producer, warp 1 score MMAs and TMEM, warp 2 PV
// MMAs (both in the even CTA only), warps 4..11 softmax and epilogue.  Thread
// (lane l of TMEM, half g) handles the 64 tokens of page 2 (l / 64) + g for row
// l mod 64: four threads share a row, and exchange their maxima through shared
// memory once a tile.  O is rescaled only when a row's maximum grew by more
// than 2^8, as in the decode kernel.  Per tile i: S_i -> softmax -> P_i -> PV_i,
// while S_{i+1} runs.  P has one buffer, handed over page by page (p_full,
// p_free): P_{i+1} of a page is written while PV_i works on the next ones, and
// PV_{i+1} follows PV_i without a gap.
//
// Work is split as in the decode kernel: the tiles of all blocks in one line,
// cut into equal ranges, one per pair; pieces leave fp32 partials, but for
// windows and chunks' blocks that one pair holds whole.  Q and the epilogue are a piece's boundary.
#include "common.cuh"
#include "pair_maps.cuh"
#include "sm100.cuh"
#include "splits.cuh"

namespace mla {
using namespace sm100;

namespace pair {
constexpr int kThreads = 384;
// kinds of the kernel: shared pages alone (all of whose rows are seen), windows,
// shared pages and then the requests' own, chunks
constexpr int kWhole = 0, kWindow = 1, kTails = 2, kChunk = 3;
// kinds whose blocks write their rows themselves, unless they are cut
constexpr bool writes_rows(int kind) { return kind == kWindow || kind == kChunk; }
constexpr int kRows = 64;                       // per CTA
constexpr int kPairRows = 128;                  // per pair
constexpr int kTilePages = 4;
constexpr int kUnitBytes = 16384;
constexpr int kMaxRing = 7;
constexpr int kPBytes = kTilePages * kRows * 128;
// bf16: Q as [dim block of 64][64 rows][128 B], P as [page][64 rows][128 B], both
// swizzled.  e4m3: Q as two terms of [block of 128 dims][64 rows][128 B],
// swizzled; P as [page][term][8-row group][16-token chunk][8 rows][16 B].
constexpr int kQTerm = 5 * kRows * 128;   // e4m3
constexpr int kPTerm = kRows * kPage;     // e4m3
template <bool F8>
struct Cfg {
  static constexpr int kRing = F8 ? 6 : 7;
  static constexpr int kKUnits = F8 ? 5 : 9, kVUnits = F8 ? 4 : 8;
  static constexpr int kQBytes = F8 ? 2 * kQTerm : 9 * kRows * 128;
  static constexpr int kOffP = kQBytes;
  static constexpr int kOffRing = kOffP + kPBytes;
  static constexpr int kOffMisc = kOffRing + kRing * kUnitBytes;
};
// A piece's boundary (Q, the first scores, the epilogue) in tiles.  It weighs most
// where short tails stand beside long blocks of shared pages: with 2 tiles (e4m3)
// the pairs at the end got so many tails that 128 rows x 64 requests over 128
// shared pages took 153 us, with 3 133, with 4 127, with 6 123; 512 rows x 32, 400
// pages and tails of 1500 tokens 624 with 3, 596 with 4, 589 with 6; bf16, 128
// pages: 1 184, 3 145, 4 148, 6 148; 512 x 32, 16 pages + 700: 3 90, 4 87, 6 94.
template <bool F8, int KIND>
constexpr int kPieceTiles = KIND == kTails ? 4 : F8 ? 2 : 1;
constexpr int kOffQ = 0;
constexpr uint32_t kColO = 0, kColS = 256;      // S buffer b: 128 columns from 256 + 128 b
constexpr int kSoftWarps = 8, kSoftThreads = 256;
constexpr long long kTimeoutClk = 4000000000ll;  // about 2 s
constexpr uint64_t kDrainNs = 200000000ull;
constexpr float kRescaleThreshold = 8.f;        // base-2 units

struct Misc {
  uint64_t full[2][kMaxRing], empty[kMaxRing], q_full, q_empty, s_full[2], s_free[2];
  uint64_t p_full[kTilePages], p_free[kTilePages], o_ready[2], o_full, o_free, drain;
  uint32_t tmem_base;
  int abort;
  float red[2][4][kRows];  // row maxima by page, double-buffered; then row sums
  float qinv[kRows];          // e4m3: 2^-k of every row's Q
  CtaRange range;
  const int2 *groups;         // shared pages: their groups' table, or null
  long long scratch[kThreads / 32 + 1];
};
template <bool F8>
constexpr int smem_bytes() { return Cfg<F8>::kOffMisc + int(sizeof(Misc)) + 1024; }
static_assert(smem_bytes<false>() <= 232448 && smem_bytes<true>() <= 232448, "shared memory budget");
}  // namespace pair

namespace {
using namespace pair;

__device__ __forceinline__ uint32_t bar(uint64_t &b) { return smem_u32(&b); }

// Block v of 128 rows: of a group's rows over its shared pages, of a request's
// rows over its own pages, or of a request's rows through its window.
template <int KIND>
__device__ __forceinline__ ViewReq make_view(const DecodeParams &p, int v, const int2 *groups) {
  if constexpr (KIND == kWindow) return window_block<kPairRows>(p, v);
  else if constexpr (KIND == kChunk) return chunk_block<kPairRows>(p, v);
  else return shared_view<kPairRows, KIND == kTails>(p, v, p.pair_blocks - p.pair_tails, groups);
}
template <int KIND>
static __device__ __noinline__ ViewReq view_call(const DecodeParams &p, int v, const int2 *groups) {
  return make_view<KIND>(p, v, groups);
}
// A call for the larger kinds, not inlined into the four roles: 3 to 8 % faster with
// an e4m3 cache (384 rows x 32 requests, window 2000: 70.5 us, inlined 73.8), the
// same with bf16.  Shared pages alone: inlined, 231 us against 235 (bf16, 4096
// rows over 32K shared tokens).
template <int KIND>
__device__ __forceinline__ ViewReq block_view(const DecodeParams &p, int v, const int2 *groups) {
  if constexpr (KIND == kWhole) return make_view<KIND>(p, v, groups);
  else return view_call<KIND>(p, v, groups);
}
// The view of block v of a chunked batch, for a role that has come to block v from an
// earlier one, of request `from`: ids grow with the requests, so that the next one or two
// are looked at, where a search takes a dozen loads one after the other.
static __device__ __noinline__ ViewReq chunk_call(const DecodeParams &p, int v, int from) {
  while (from + 1 < p.batch && chunk_base<kPairRows>(p, from + 1) <= v) ++from;
  return chunk_block_of<kPairRows>(p, v, from);
}
__device__ __forceinline__ int tiles_of(const ViewReq &view) { return (view.tiles + kTilePages - 1) / kTilePages; }

// Worker idx's range of a chunked batch, as schedule_range has it.  A thread takes blocks
// next to one another, so that it searches for the request of the first alone (304
// requests of one block, e4m3: 65 us a call; searched for one by one in two passes, 70).
// Block-wide.
template <int PC>
__device__ __forceinline__ void schedule_chunks(const DecodeParams &p, int idx, int workers, CtaRange *r,
                                                long long *scratch) {
  const int tid = threadIdx.x, nw = kThreads / 32, lane = tid & 31, warp = tid >> 5;
  const int V = p.pair_blocks, per = (V + kThreads - 1) / kThreads;
  const int v0 = min(V, tid * per), v1 = min(V, v0 + per);
  const int from = v0 < v1 ? chunk_request<kPairRows>(p, v0) : 0;
  long long mine = 0;
  for (int v = v0, b = from; v < v1; ++v) {
    while (b + 1 < p.batch && chunk_base<kPairRows>(p, b + 1) <= v) ++b;
    mine += request_cost(tiles_of(chunk_block_of<kPairRows>(p, v, b)), PC);
  }
  long long incl = mine;
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
  if (tid == 0) {
    r->total = C;
    r->g_eff = g_eff;
    r->start = start;
    r->end = has ? sched_start_short(idx + 1, C, g_eff) : 0;
  }
  // the first block whose tiles end after `start`: its predecessor's end at `at` - PC
  long long at = before + incl - mine;
  if (has && at - PC <= start && start < at + mine) {
    for (int v = v0, b = from; v < v1; ++v) {
      while (b + 1 < p.batch && chunk_base<kPairRows>(p, b + 1) <= v) ++b;
      const int tiles = tiles_of(chunk_block_of<kPairRows>(p, v, b));
      if (tiles > 0 && at + tiles > start && at - PC <= start) {
        r->v_begin = v;
        r->p_begin = at;
        break;
      }
      at += request_cost(tiles, PC);
    }
  }
  __syncthreads();
}

// The pieces of this pair's range, in order.
template <bool F8, int KIND>
struct Pieces {
  const DecodeParams &p;
  const CtaRange &r;
  int v, tiles;
  long long pv, t0, t1;
  ViewReq view;
  const Misc &m;
  __device__ Pieces(const DecodeParams &p_, const CtaRange &r_, const Misc &m_)
      : p(p_), r(r_), v(r_.v_begin), pv(r_.p_begin), m(m_) {}
  __device__ bool next() {
    while (v < p.pair_blocks && pv < r.end) {
      if constexpr (KIND == kChunk) view = v == r.v_begin ? block_view<KIND>(p, v, m.groups) : chunk_call(p, v, view.req);
      else view = block_view<KIND>(p, v, m.groups);
      tiles = tiles_of(view);
      if (tiles == 0) { ++v; continue; }
      t0 = max(r.start, pv) - pv;
      t1 = min(r.end, pv + tiles) - pv;
      if (t0 < t1) return true;
      advance();
    }
    return false;
  }
  __device__ void advance() { pv += request_cost(tiles, kPieceTiles<F8, KIND>); ++v; }
};

template <bool F8, int KIND>
__device__ __forceinline__ uint32_t total_tiles(const DecodeParams &p, const CtaRange &r, const Misc &m) {
  uint32_t n = 0;
  for (Pieces<F8, KIND> w(p, r, m); w.next(); w.advance()) n += uint32_t(w.t1 - w.t0);
  return n;
}

// Units in load order: K_0, K_1, V_0, K_2, V_1, ...  A bf16 range runs on like
// this across its pieces.  An e4m3 piece's first K comes after the last V of the
// piece before: its scores wait for Q, which the softmax warps split after that
// piece's epilogue, and K units waiting for it would keep V out of the ring.
// First unit of K_n and V_n (`first`, `last`: of the range, or of the piece).
template <bool F8>
__device__ __forceinline__ uint32_t k_unit(uint32_t n, bool first) {
  return (Cfg<F8>::kKUnits + Cfg<F8>::kVUnits) * n - (first ? 0 : Cfg<F8>::kVUnits);
}
template <bool F8>
__device__ __forceinline__ uint32_t v_unit(uint32_t n, bool last) {
  return (Cfg<F8>::kKUnits + Cfg<F8>::kVUnits) * n + (last ? 1 : 2) * Cfg<F8>::kKUnits;
}
// A slot has one "landed" barrier for K units and one for V units: the score
// and PV threads wait at their own pace, and a barrier shared by both kinds
// could complete a phase that one of them has not looked at yet, which its
// parity cannot tell from the phase before.
struct Landed {
  uint32_t phases = 0;  // bit s: parity of the kind's next use of slot s
  __device__ __forceinline__ uint32_t take(int s) {
    const uint32_t ph = (phases >> s) & 1u;
    phases ^= 1u << s;
    return ph;
  }
};
template <bool F8>
__device__ __forceinline__ int next_slot(int s) { return s + 1 == Cfg<F8>::kRing ? 0 : s + 1; }

// ------------------------------------------------------------------ producer

// One position in the tiles of a range, with the tile's pages.
template <bool F8, int KIND>
struct TileWalk {
  Pieces<F8, KIND> w;
  long long t;
  bool live;
  int page[kTilePages];
  __device__ TileWalk(const DecodeParams &p, const CtaRange &r, const Misc &m) : w(p, r, m), t(0) {
    live = w.next();
    if (live) t = w.t0;
    load();
  }
  // A page past the view repeats the last one (its tokens are masked), an
  // entry out of range reads page 0.
  __device__ void load() {
    if (!live) return;
    const int32_t *row = w.p.block_table + size_t(w.view.req) * w.p.max_pages;
#pragma unroll
    for (int i = 0; i < kTilePages; ++i) page[i] = __ldg(row + w.view.page(min(int(t) * kTilePages + i, w.view.tiles - 1)));
  }
  __device__ void check(int *err) {
#pragma unroll
    for (int i = 0; i < kTilePages; ++i)
      if (page[i] < 0 || page[i] >= w.p.num_pages) {
        atomicOr(err, kErrBadPage);
        page[i] = 0;
      }
  }
  // Every row of the tile's pages is seen (false for some such tiles of sinks): asked
  // once a tile, as the masks of four pages cost the producer a fifth of its time.
  __device__ __forceinline__ bool whole() const {
    const int k = int(t) * kTilePages - w.view.nsink, base = (w.view.first + k) * kPage;
    return k >= 0 && base >= w.view.lead && base <= w.view.end - kTilePages * kPage;
  }
  // rows of page i that some row of the block sees (none past the view)
  __device__ unsigned long long seen(int i) const {
    const int k = int(t) * kTilePages + i;
    return k < w.view.tiles ? w.view.seen_rows(w.p, k) : 0ull;
  }
  __device__ bool first() const { return t == w.t0; }
  __device__ void step() {
    if (++t >= w.t1) {
      w.advance();
      live = w.next();
      if (live) t = w.t0;
    }
    load();
  }
};

// A unit of V of whose rows only some are seen (bit r of `rows`: row r).  The
// others may hold anything, and weights of 0 do not keep a NaN out of the
// product: they are loaded from past the end of the pool (`none`), as zeros.
template <bool F8>
static __device__ __noinline__ void load_seen(uint32_t dst, uint32_t full, const CUtensorMap *tm_v,
                                              const CUtensorMap *tm_va, const CUtensorMap *tm_vr, int block, int atom,
                                              int none, uint64_t rows) {
  constexpr int kBlocks = F8 ? 2 : 4, kAtoms = F8 ? 8 : 4;
  constexpr uint64_t kAll = F8 ? ~0ull : 0xffffffffull;
  if ((rows & kAll) == kAll || (rows & kAll) == 0) {
    tma_load_4d_pair(dst, tm_v, full, 0, 0, block, rows & kAll ? atom : none);
    return;
  }
#pragma unroll 1
  for (int a = 0; a < kAtoms; ++a, rows >>= 8, dst += kBlocks * 1024) {
    const uint32_t m = uint32_t(rows) & 0xffu;
    if (m == 0xffu || m == 0) {
      tma_load_4d_pair(dst, tm_va, full, 0, 0, block, m ? atom + a : none);
      continue;
    }
#pragma unroll 1
    for (int k = 0; k < 8 * kBlocks; ++k)
      tma_load_4d_pair(dst + k * 128, tm_vr, full, 0, k & 7, block + (k >> 3), (m >> (k & 7)) & 1u ? atom + a : none);
  }
}

// One thread produces: a warp's votes and shuffles between the units made
// the producer the slowest role (470 cycles a unit, all 17 of a tile).
template <bool F8, int KIND>
__device__ __forceinline__ void produce(const DecodeParams &p, const CtaRange &r, Misc &m, uint32_t sQ,
                                        uint32_t sRing, uint32_t rank, const CUtensorMap *tm_q,
                                        const CUtensorMap *tm_k, const CUtensorMap *tm_k4, const CUtensorMap *tm_v,
                                        const CUtensorMap *tm_va, const CUtensorMap *tm_vr, int *err) {
  constexpr int kKUnits = Cfg<F8>::kKUnits;
  volatile int *abort = &m.abort;
  const bool leader = rank == 0;
  int at = 0;
  uint32_t lap = 1;  // parity of the empty barriers' last phase
  uint32_t q_it = 0;
  bool ok = true;
  const uint32_t full0 = map_to_rank(bar(m.full[0][0]), 0);
  const uint32_t q_full = map_to_rank(bar(m.q_full), 0);
  // slot of the next unit (kind 0: K, 1: V), emptied; the even CTA announces
  // both CTAs' bytes
  auto slot = [&](int kind, uint32_t bytes, uint32_t *full) {
    const int s = at;
    if (!mbar_wait_clk(bar(m.empty[s]), lap, abort, kTimeoutClk)) return -1;
    if (leader) mbar_arrive_expect_tx(bar(m.full[kind][s]), 2 * bytes);
    *full = full0 + 8 * (kind * kMaxRing + s);
    at = next_slot<F8>(s);
    if (at == 0) lap ^= 1;
    return s;
  };
  auto load_k = [&](const TileWalk<F8, KIND> &c) {
    if (!F8 && c.first()) {  // (e4m3: the softmax warps load and split Q)
      if (!mbar_wait_clk(bar(m.q_empty), (q_it & 1) ^ 1, abort, kTimeoutClk)) return false;
      ++q_it;
      if (leader) mbar_arrive_expect_tx(bar(m.q_full), 2 * Cfg<F8>::kQBytes);
      for (int i = 0; i < 9; ++i)
        tma_load_2d_pair(sQ + i * kRows * 128, tm_q, q_full, i * 64, c.w.view.row0 + int(rank) * kRows);
    }
    const int pg0 = rank ? c.page[2] : c.page[0], pg1 = rank ? c.page[3] : c.page[1];  // checked
    for (int kb = 0; kb < kKUnits; ++kb) {
      uint32_t full;
      const bool rope = F8 && kb == kKUnits - 1;  // e4m3: the last 64 dims, 64 bytes a row
      const int s = slot(0, rope ? kUnitBytes / 2 : kUnitBytes, &full);
      if (s < 0) return false;
      const uint32_t dst = sRing + s * kUnitBytes;
      if (rope) {
        tma_load_2d_pair(dst, tm_k4, full, 512, pg0 * kPage);
        tma_load_2d_pair(dst + 4096, tm_k4, full, 512, pg1 * kPage);
      } else {
        tma_load_4d_pair(dst, tm_k, full, 0, 0, kb, pg0 * 8);
        tma_load_4d_pair(dst + 8192, tm_k, full, 0, 0, kb, pg1 * 8);
      }
    }
    return true;
  };
  auto load_v = [&](const int (&page)[kTilePages], const unsigned long long (&seen)[kTilePages], bool whole) {
#pragma unroll
    for (int i = 0; i < kTilePages; ++i) {
      for (int h = 0; h < (F8 ? 1 : 2); ++h) {
        uint32_t full;
        const int s = slot(1, kUnitBytes, &full);
        if (s < 0) return false;
        const uint32_t dst = sRing + s * kUnitBytes;
        const int block = (F8 ? 2 : 4) * int(rank), atom = page[i] * 8 + 4 * h;
        if (KIND == kWhole || whole) tma_load_4d_pair(dst, tm_v, full, 0, 0, block, atom);
        else load_seen<F8>(dst, full, tm_v, tm_va, tm_vr, block, atom, p.num_pages * 8, seen[i] >> (32 * h));
      }
    }
    return true;
  };
  // c: the next tile to load K of; its pages are read a tile early, so that
  // their latency hides behind the units of the tile before
  TileWalk<F8, KIND> c(p, r, m);
  int last[kTilePages];  // pages of the tile whose V comes next, and their seen rows
  unsigned long long lseen[kTilePages] = {0, 0, 0, 0};
  bool have = false, lwhole = true;
  while (ok && (c.live || have)) {
    int pages[kTilePages];
    unsigned long long seen[kTilePages] = {0, 0, 0, 0};
    bool whole = true;
    const bool more = c.live;
    if (F8 && have && more && c.first()) {
      ok = load_v(last, lseen, lwhole);
      have = false;
      if (!ok) break;
    }
    if (more) {
      c.check(err);
#pragma unroll
      for (int i = 0; i < kTilePages; ++i) pages[i] = c.page[i];
      if (KIND != kWhole) {
        whole = c.whole();
        if (!whole) {
#pragma unroll
          for (int i = 0; i < kTilePages; ++i) seen[i] = c.seen(i);
        }
      }
      ok = load_k(c);
      c.step();
    }
    if (ok && have) ok = load_v(last, lseen, lwhole);
#pragma unroll
    for (int i = 0; i < kTilePages; ++i) {
      last[i] = pages[i];
      lseen[i] = seen[i];
    }
    have = more;
    lwhole = whole;
  }
  if (!ok) atomicOr(err, kErrTimeout);
}

// ------------------------------------------------------------------ MMAs (even CTA)

// A wait of a whole warp (the same answer in every lane).
__device__ __forceinline__ bool warp_wait(uint32_t b, uint32_t parity, volatile int *abort) {
  return __all_sync(0xffffffffu, mbar_wait_clk(b, parity, abort, kTimeoutClk));
}

template <bool F8, int KIND>
__device__ __forceinline__ void score_mmas(const DecodeParams &p, const CtaRange &r, Misc &m, uint32_t sQ,
                                           uint32_t sRing, uint32_t tmem, int *err) {
  volatile int *abort = &m.abort;
  constexpr int kKUnits = Cfg<F8>::kKUnits;
  const uint32_t idesc = F8 ? idesc_e4m3_f32(128, 256, false, false) : idesc_bf16_f32(128, 256, false, false);
  const uint64_t dq = smem_desc_sw128(sQ, 16, 1024), dk = smem_desc_sw128(sRing, 16, 1024);
  const uint64_t dk4 = smem_desc_sw64(sRing, 16, 512);  // e4m3
  Landed landed;
  uint32_t n = 0;
  uint32_t q_it = 0;
  bool ok = true;
  for (Pieces<F8, KIND> w(p, r, m); ok && w.next(); w.advance()) {
    for (long long t = w.t0; ok && t < w.t1; ++t, ++n) {
      const int b = int(n & 1);
      ok = warp_wait(bar(m.s_free[b]), ((n >> 1) & 1) ^ 1, abort);
      if (ok && t == w.t0) {
        ok = warp_wait(bar(m.q_full), q_it & 1, abort);
        ++q_it;
      }
      // orders these MMAs behind the reads of the S buffer; the waits for landed
      // units need no such fence
      tc_fence_after();
      int s = int(k_unit<F8>(n, t == w.t0 && (F8 || n == 0)) % Cfg<F8>::kRing);
      for (int kb = 0; ok && kb < kKUnits; ++kb, s = next_slot<F8>(s)) {
        ok = warp_wait(bar(m.full[0][s]), landed.take(s), abort);
        if (!ok) break;
        if (elect_one()) {
          if constexpr (F8) {
            // Q's two terms against the block of 128 dims (the last: 64, in
            // rows of 64 bytes), 32 dims a step
            const uint64_t dkb = kb == kKUnits - 1 ? dk4 : dk;
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                if (ks < 2 || kb < kKUnits - 1)
                  mma_f8_ss_pair(tmem + kColS + 128 * b, dq + ((term * kQTerm + kb * kRows * 128 + ks * 32) >> 4),
                                 dkb + ((s * kUnitBytes + ks * 32) >> 4), idesc, kb > 0 || term > 0 || ks > 0);
          } else
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_bf16_ss_pair(tmem + kColS + 128 * b, dq + ((kb * kRows * 128 + ks * 32) >> 4),
                             dk + ((s * kUnitBytes + ks * 32) >> 4), idesc, kb > 0 || ks > 0);
          mma_commit_pair(bar(m.empty[s]));
          if (kb == kKUnits - 1) {
            mma_commit_pair(bar(m.s_full[b]));
            if (t == w.t1 - 1) mma_commit_pair(bar(m.q_empty));
          }
        }
        __syncwarp();
      }
    }
  }
  if (elect_one()) {
    if (!ok) atomicOr(err, kErrTimeout);
    mma_commit_pair(bar(m.drain));
  }
  __syncwarp();
}

template <bool F8, int KIND>
__device__ __forceinline__ void pv_mmas(const DecodeParams &p, const CtaRange &r, Misc &m, uint32_t sP,
                                        uint32_t sRing, uint32_t tmem, int *err) {
  volatile int *abort = &m.abort;
  const uint32_t idesc = F8 ? idesc_e4m3_f32(128, 256, false, true) : idesc_bf16_f32(128, 256, false, true);
  const uint32_t idesc_lo = idesc_f8_f32(128, 256, false, true, kFmtE5M2, kFmtE4M3);  // e4m3: P's lo term
  const uint64_t dp = F8 ? smem_desc_noswz(sP, 128, 512) : smem_desc_sw128(sP, 16, 1024);
  // V, MN-major: 128-byte blocks of dims 1 KB apart, 8-token groups 4 KB (bf16)
  // or 2 KB (e4m3) apart
  const uint64_t dv = smem_desc_sw128(sRing, 1024, F8 ? 2048 : 4096);
  const uint32_t total = total_tiles<F8, KIND>(p, r, m);
  Landed landed;
  uint32_t n = 0;
  uint32_t o_it = 0;
  bool ok = true;
  for (Pieces<F8, KIND> w(p, r, m); ok && w.next(); w.advance(), ++o_it) {
    for (long long t = w.t0; ok && t < w.t1; ++t, ++n) {
      ok = warp_wait(bar(m.o_ready[n & 1]), (n >> 1) & 1, abort);
      if (ok && t == w.t0) ok = warp_wait(bar(m.o_free), (o_it & 1) ^ 1, abort);
      tc_fence_after();
      int s = int(v_unit<F8>(n, t == w.t1 - 1 && (F8 || n == total - 1)) % Cfg<F8>::kRing);
      for (int pg = 0; ok && pg < kTilePages; ++pg) {
        ok = warp_wait(bar(m.p_full[pg]), n & 1, abort);
        constexpr int kHalves = F8 ? 1 : 2;  // units of 64 or 32 tokens
        for (int h = 0; ok && h < kHalves; ++h, s = next_slot<F8>(s)) {
          ok = warp_wait(bar(m.full[1][s]), landed.take(s), abort);
          if (!ok) break;
          if (elect_one()) {
            if constexpr (F8) {
#pragma unroll
              for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const uint64_t a = dp + ((pg * 2 * kPTerm + ks * 256) >> 4);
                  const uint64_t v = dv + ((s * kUnitBytes + ks * 8192 + j * 1024) >> 4);
                  mma_f8_ss_pair(tmem + kColO + 128 * j, a, v, idesc, t > w.t0 || pg > 0 || ks > 0);
                  mma_f8_ss_pair(tmem + kColO + 128 * j, a + (kPTerm >> 4), v, idesc_lo, 1u);
                }
            } else
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                mma_bf16_ss_pair(tmem + kColO + 128 * j, dp + ((pg * kRows * 128 + (h * 2 + ks) * 32) >> 4),
                                 dv + ((s * kUnitBytes + ks * 8192 + j * 2048) >> 4), idesc,
                                 t > w.t0 || pg > 0 || h > 0 || ks > 0);
            mma_commit_pair(bar(m.empty[s]));
            if (h == kHalves - 1) {
              mma_commit_pair(bar(m.p_free[pg]));
              if (pg == kTilePages - 1 && t == w.t1 - 1) mma_commit_pair(bar(m.o_full));
            }
          }
          __syncwarp();
        }
      }
    }
  }
  if (elect_one()) {
    if (!ok) atomicOr(err, kErrTimeout);
    mma_commit_pair(bar(m.drain));
  }
  __syncwarp();
}

// ------------------------------------------------------------------ softmax and epilogue

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// O *= alpha (this thread's row), 128 columns of this warp's TMEM lanes.
static __device__ __noinline__ void rescale_rows(uint32_t taddr, float alpha) {
  for (int c = 0; c < 128; c += 16) {
    uint32_t o[16];
    tmem_ld16(taddr + c, o);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
    tmem_st16(taddr + c, o);
  }
  tmem_wait_st();
}

__device__ __forceinline__ void st_global_v8(float *dst, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// e4m3: the block's Q rows of this CTA (bf16) as two e4m3 terms, hi + lo, of
// 2^k q, with a 2^k for each row such that its largest |q| lies in [2^7, 2^8) (hi +
// lo is then exact down to 2^-9 of it).  The rows may be those of several requests:
// with one 2^k for all of them, one request's queries would set the precision of
// another's.  A row with an Inf or a NaN enters as NaN; rows past the block are
// zero.  All softmax threads, a warp eight rows, once a piece, when the piece
// before has read Q.  2^-k goes to m.qinv.
__device__ __forceinline__ bool split_q(const DecodeParams &p, Misc &m, unsigned char *smem, const ViewReq &view,
                                        uint32_t rank, int st, uint32_t piece, bool ok) {
  constexpr int kChunks = kDqk / 8;                       // 8 dims each
  constexpr int kWarpRows = kRows / kSoftWarps, kPer = kWarpRows * kChunks / 32;  // 8 rows; 18 chunks a lane
  static_assert(kWarpRows * kChunks == 32 * kPer, "Q chunks");
  const int warp = st >> 5, lane = st & 31, first = warp * kWarpRows;
  const int rows = min(kRows, max(0, view.rows - int(rank) * kRows));
  const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (size_t(view.row0) + rank * kRows + first) * kDqk);
  const int left = (rows - first) * kChunks;
  uint4 v[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) v[u] = lane + 32 * u < left ? __ldg(src + lane + 32 * u) : make_uint4(0, 0, 0, 0);
  float row_sc[kWarpRows];
  row_q_scales(v, lane, row_sc);
  if (lane == 0)
#pragma unroll
    for (int w = 0; w < kWarpRows; ++w) m.qinv[first + w] = inverse_q_scale(row_sc[w]);
  named_sync(1, kSoftThreads);  // (every thread reads its row's)
  ok = ok && __all_sync(0xffffffffu, mbar_wait_clk(bar(m.q_empty), (piece & 1) ^ 1, &m.abort, kTimeoutClk));
  if (!ok) return false;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int w0 = 32 * u / kChunks, next = (w0 + 1) * kChunks - 32 * u;  // lanes from `next` on: the row after w0
    const int w = w0 + (lane >= next ? 1 : 0), rr = first + w, c = lane + 32 * u - kChunks * w;
    const float sc = next < 32 && lane >= next ? row_sc[w0 + 1] : row_sc[w0];
    const uint32_t wv[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
    uint32_t hw[2] = {0, 0}, lw[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float f0 = __uint_as_float(wv[e] << 16) * sc, f1 = __uint_as_float(wv[e] & 0xffff0000u) * sc;
      const uint16_t h = float2_to_e4m3x2(f0, f1);
      const float2 bh = e4m3x2_to_float2(h);
      const uint16_t l = float2_to_e4m3x2(f0 - bh.x, f1 - bh.y);
      hw[e >> 1] |= uint32_t(h) << (16 * (e & 1));
      lw[e >> 1] |= uint32_t(l) << (16 * (e & 1));
    }
    // dims 8c .. 8c + 7: block c / 16, 16-byte chunk (c % 16) / 2 at its swizzled place
    const int b = c & 15;
    const int off = (c >> 4) * kRows * 128 + (rr >> 3) * 1024 + (rr & 7) * 128 + (((b >> 1) ^ (rr & 7)) << 4) +
                    8 * (b & 1);
    *reinterpret_cast<uint2 *>(smem + kOffQ + off) = make_uint2(hw[0], hw[1]);
    *reinterpret_cast<uint2 *>(smem + kOffQ + kQTerm + off) = make_uint2(lw[0], lw[1]);
  }
  fence_proxy_async_smem();
  __syncwarp();
  return true;
}

// Sends a warp's 32 rows of 128 bytes, lane i's row in v, to dst + i * stride (rows below
// `rows` only) through the warp's own part of P, which is free at a piece's end: a store
// instruction then writes four whole rows.  (A lane's row 16 bytes at a time: two blocks of
// one tile a pair took 33 us instead of 30.)
template <bool F8>
__device__ __forceinline__ void send_rows(unsigned char *own, const uint32_t (&v)[32], void *dst, size_t stride,
                                          int rows) {
  const int lane = threadIdx.x & 31, c = lane & 7;
  // e4m3: 16 rows in the place of each term
  auto place = [&](int i) { return own + (F8 ? (i >> 4) * kPTerm + (i & 15) * 128 : i * 128); };
#pragma unroll
  for (int k = 0; k < 8; ++k)
    *reinterpret_cast<uint4 *>(place(lane) + ((k ^ c) << 4)) =
        make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int i = 4 * k + (lane >> 3);
    const uint4 x = *reinterpret_cast<const uint4 *>(place(i) + ((c ^ (i & 7)) << 4));
    if (i < rows) *reinterpret_cast<uint4 *>(static_cast<unsigned char *>(dst) + i * stride + 16 * c) = x;
  }
  __syncwarp();
}

// A failed wait never leaves the loop: the warp goes on without working, so
// that the others find it at their barriers (later waits fail at once).
template <bool F8, int KIND>
__device__ __forceinline__ void softmax(const DecodeParams &p, const CtaRange &r, Misc &m, unsigned char *smem,
                                        uint32_t tmem, uint32_t rank, int pair_id, int *err) {
  volatile int *abort = &m.abort;
  const int st = int(threadIdx.x) - 128, warp = st >> 5, lane = st & 31;  // warps 0..7
  const int g = warp >> 2, q = warp & 3;             // column half, TMEM quarter (lanes 32q ..)
  const int row = 32 * (q & 1) + lane, pb = 2 * (q >> 1) + g;
  const uint32_t lanes = uint32_t(32 * q) << 16;
  const uint32_t t_s = tmem + lanes + kColS + 64 * g, t_o = tmem + lanes + kColO + 128 * g;
  float cs = p.score_scale_log2;
  unsigned char *prow = smem + Cfg<F8>::kOffP + pb * kRows * 128 +
                        (F8 ? (row >> 3) * 512 + (row & 7) * 16 : row * 128);
  const uint32_t q_full = map_to_rank(bar(m.q_full), 0);
  const uint32_t s_free0 = map_to_rank(bar(m.s_free[0]), 0);
  const uint32_t s_free1 = map_to_rank(bar(m.s_free[1]), 0);
  const uint32_t p_full = map_to_rank(bar(m.p_full[pb]), 0);
  const uint32_t o_ready = map_to_rank(bar(m.o_ready[0]), 0), o_free = map_to_rank(bar(m.o_free), 0);
  uint32_t n = 0;
  uint32_t o_it = 0;
  bool ok = true;
  Pieces<F8, KIND> w(p, r, m);
  for (bool more = w.next(); more; ++o_it) {
    const int grow = w.view.row0 + int(rank) * kRows + row;
    RowView rv;
    if constexpr (KIND == kChunk) rv = chunk_row_view(p, w.view, min(grow, w.view.row0 + w.view.rows - 1));
    else rv = row_view<KIND == kWindow>(p, w.view, min(grow, p.batch * p.heads - 1));
    const bool mine = int(rank) * kRows + row < w.view.rows;
    if constexpr (F8) {
      ok = split_q(p, m, smem, w.view, rank, st, o_it, ok);
      if (ok && lane == 0) mbar_arrive_cluster(q_full);
      cs = p.score_scale_log2 * p.kv_scale * m.qinv[row];
    }
    float mrun = -INFINITY, ell = 0.f, ellx = 0.f;
    for (long long t = w.t0; t < w.t1; ++t, ++n) {
      const int b = int(n & 1);
      ok = ok && __all_sync(0xffffffffu, mbar_wait_clk(bar(m.s_full[b]), (n >> 1) & 1, abort, kTimeoutClk));
      float x[64];
      if (ok) {
        tc_fence_after();
        uint32_t a[32], c[32];
        tmem_ld32(t_s + 128 * b, a);
        tmem_ld32(t_s + 128 * b + 32, c);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          x[i] = __uint_as_float(a[i]);
          x[32 + i] = __uint_as_float(c[i]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(b ? s_free1 : s_free0);
      } else {
#pragma unroll
        for (int i = 0; i < 64; ++i) x[i] = 0.f;
      }
      const int idx = int(t) * kTilePages + pb;  // page of the view
      const int base = w.view.page(idx) * kPage;
      const int left = idx < w.view.tiles ? rv.hi - base : 0;  // tokens of the page this row sees
      if (left < kPage) {
#pragma unroll
        for (int i = 0; i < 64; ++i) x[i] = i < left ? x[i] : -INFINITY;
      }
      if constexpr (KIND == kWindow) {
        const int skip = rv.lo - base, sink = p.sinks - base;
        if (skip > 0 && sink < kPage) {
#pragma unroll
          for (int i = 0; i < 64; ++i) x[i] = i >= skip || i < sink ? x[i] : -INFINITY;
        }
      }
      float mx4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int i = 4; i < 64; i += 4)
#pragma unroll
        for (int k = 0; k < 4; ++k) mx4[k] = fmaxf(mx4[k], x[i + k]);
      m.red[b][pb][row] = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
      named_sync(1, kSoftThreads);
      const float top = fmaxf(fmaxf(m.red[b][0][row], m.red[b][1][row]), fmaxf(m.red[b][2][row], m.red[b][3][row])) * cs;
      float alpha = 1.f;
      bool resc = false;
      if (t == w.t0) {
        mrun = top;
      } else if (top > mrun + kRescaleThreshold) {
        alpha = exp2f(mrun - top);
        mrun = top;
        resc = true;
      }
      // a row that has seen no token yet keeps a -inf maximum: its weights are 0
      const float mref = mrun == -INFINITY ? 0.f : mrun;
      // bf16: the weights in pairs; e4m3: hi terms (e4m3), then lo terms (e5m2)
      uint32_t pk[32];
      float lsum[2] = {0.f, 0.f}, xsum[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float e0 = exp2_approx(fmaf(x[2 * i], cs, -mref)), e1 = exp2_approx(fmaf(x[2 * i + 1], cs, -mref));
        xsum[0] += e0;
        xsum[1] += e1;
        if constexpr (F8) {
          const uint16_t hi = float2_to_e4m3x2(e0, e1);
          const float2 bh = e4m3x2_to_float2(hi);
          const uint16_t lo = float2_to_e5m2x2(e0 - bh.x, e1 - bh.y);
          const float2 bl = e5m2x2_to_float2(lo);
          lsum[0] += bh.x + bl.x;
          lsum[1] += bh.y + bl.y;
          pk[i >> 1] = i & 1 ? pk[i >> 1] | uint32_t(hi) << 16 : hi;
          pk[16 + (i >> 1)] = i & 1 ? pk[16 + (i >> 1)] | uint32_t(lo) << 16 : lo;
        } else {
          __nv_bfloat162 v = __floats2bfloat162_rn(e0, e1);
          pk[i] = *reinterpret_cast<uint32_t *>(&v);
          lsum[0] += __uint_as_float(pk[i] << 16);
          lsum[1] += __uint_as_float(pk[i] & 0xffff0000u);
        }
      }
      ell = ell * alpha + (lsum[0] + lsum[1]);
      ellx = ellx * alpha + (xsum[0] + xsum[1]);
      // O is this tile's to add to once every warp has said so: at once, or
      // after the rare rescale, which waits for the previous tile's products.
      // (Two barriers in turn: a warp may say so for tile i + 1 before the PV
      // thread has asked about tile i, but not for i + 2.)
      if (__any_sync(0xffffffffu, resc)) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait_clk(bar(m.p_free[kTilePages - 1]), (n - 1) & 1, abort, kTimeoutClk));
        if (ok) {
          tc_fence_after();
          rescale_rows(t_o, alpha);
          tc_fence_before();
        }
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive_cluster(o_ready + 8 * b);
      // the page's part of P is free once the previous tile's product with it is done
      if (n > 0)
        ok = ok && __all_sync(0xffffffffu, mbar_wait_clk(bar(m.p_free[pb]), (n - 1) & 1, abort, kTimeoutClk));
      if (ok) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4 *>(prow + (F8 ? (c >> 2) * kPTerm + (c & 3) * 128 : (c ^ (row & 7)) << 4)) =
              make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(p_full);
      }
    }
    // ---- this piece's partial: O / sum and the LSE of its rows
    named_sync(1, kSoftThreads);  // every thread is past its last read of the maxima
    m.red[0][pb][row] = ell;
    m.red[1][pb][row] = ellx;
    named_sync(1, kSoftThreads);
    const float sum = (m.red[0][0][row] + m.red[0][1][row]) + (m.red[0][2][row] + m.red[0][3][row]);
    const float sumx = (m.red[1][0][row] + m.red[1][1][row]) + (m.red[1][2][row] + m.red[1][3][row]);
    named_sync(1, kSoftThreads);  // read before the next piece writes maxima
    const float inv = sum > 0.f ? p.kv_scale / sum : 0.f;
    // chunks: the next piece is looked up while the products of this one end
    const ViewReq view = w.view;
    const long long pv = w.pv;
    const int v = w.v, tiles = w.tiles;
    if constexpr (KIND == kChunk) {
      w.advance();
      more = w.next();
    }
    ok = ok && __all_sync(0xffffffffu, mbar_wait_clk(bar(m.o_full), o_it & 1, abort, kTimeoutClk));
    const int c_first = sched_owner_short(pv, r.total, r.g_eff);
    const int pieces = sched_owner_short(pv + tiles - 1, r.total, r.g_eff) - c_first + 1;
    const bool split = !writes_rows(KIND) || pieces > 1;
    // shared pages and tails: every piece leaves a partial, in the slots of its
    // pair and block; a window's and a chunk's do when the block is cut, in the slots
    // of the split merge, its CTA r * pairs + c standing for half r of pair c
    const size_t slot = writes_rows(KIND) ? 2 * size_t(rank * p.pairs + pair_id) + (v != r.v_begin ? 1 : 0)
                                        : 2 * size_t(pair_id + v) + rank;
    if (ok) {
      tc_fence_after();
      const int d0 = 256 * (q >> 1) + 128 * g;
      float *dst = slot_out_ptr(p) + (slot * kSlotHeads + row) * kDv + d0;
      __nv_bfloat16 *out = p.out + size_t(grow) * kDv + d0;
      if constexpr (KIND == kChunk) {
        unsigned char *own = smem + Cfg<F8>::kOffP + pb * kRows * 128 + 32 * (q & 1) * (F8 ? 64 : 128);
        const int rows = view.rows - (int(rank) * kRows + row - lane);  // from this warp's first on
#pragma unroll 1
        for (int c = 0; c < 128; c += 64) {
          uint32_t o[2][32];
          tmem_ld32(t_o + c, o[0]);
          tmem_ld32(t_o + c + 32, o[1]);
          tmem_wait_ld();
          if (rows <= 0) continue;
#pragma unroll
          for (int i = 0; i < 64; ++i) o[i >> 5][i & 31] = __float_as_uint(__uint_as_float(o[i >> 5][i & 31]) * inv);
          if (split) {
            send_rows<F8>(own, o[0], dst - lane * kDv + c, kDv * 4, rows);
            send_rows<F8>(own, o[1], dst - lane * kDv + c + 32, kDv * 4, rows);
          } else {
            uint32_t v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              __nv_bfloat162 x2 = __floats2bfloat162_rn(__uint_as_float(o[i >> 4][2 * (i & 15)]),
                                                        __uint_as_float(o[i >> 4][2 * (i & 15) + 1]));
              v[i] = *reinterpret_cast<uint32_t *>(&x2);
            }
            send_rows<F8>(own, v, out - lane * kDv + c, kDv * 2, rows);
          }
        }
      } else
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t o[32];
        tmem_ld32(t_o + c, o);
        tmem_wait_ld();
        if (mine) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(o[i + k]) * inv;
            if (split) {
              st_global_v8(dst + c + i, v);
            } else {
              uint32_t h[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                __nv_bfloat162 x2 = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
                h[k] = *reinterpret_cast<uint32_t *>(&x2);
              }
              *reinterpret_cast<uint4 *>(out + c + i) = make_uint4(h[0], h[1], h[2], h[3]);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(o_free);
      if (mine && pb == 0) {
        const float lse2 = mrun + log2f(sumx);
        if (split) slot_lse_ptr(p)[slot * kSlotHeads + row] = lse2;
        else p.lse[grow] = lse_out(p, lse2);
      }
      if (st == 0 && pair_id == c_first) {
        if (KIND == kChunk) {  // a pair begins at most one block that others go on with: the pair's record
          if (rank == 0 && pieces > 1)
            info_ptr(p)[pair_id] = make_int4(pieces, view.row0, view.rows, v != r.v_begin ? 1 : 0);
        } else if (KIND == kWindow) {  // the record of this half's 64 rows
          if (view.rows > int(rank) * kRows)
            info_ptr(p)[(2 * (v / p.batch) + int(rank)) * p.batch + v % p.batch] =
                make_int4(int(rank) * p.pairs + c_first, pieces, int(slot), 0);
        } else if (rank == 0) {
          pair_info_ptr(p)[v] = make_int4(c_first, pieces, pair_id + v, 0);
        }
      }
    }
    if constexpr (KIND != kChunk) {
      w.advance();
      more = w.next();
    }
  }
  if (!ok) atomicOr(err, kErrTimeout);
}

template <bool F8, int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    decode_pair_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_k4,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_va,
                       const __grid_constant__ CUtensorMap tm_vr) {
  constexpr int kOffP = Cfg<F8>::kOffP, kOffRing = Cfg<F8>::kOffRing;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), pad = ((raw + 1023u) & ~1023u) - raw;
  unsigned char *smem = smem_raw + pad;
  const uint32_t sbase = raw + pad;
  Misc &m = *reinterpret_cast<Misc *>(smem + Cfg<F8>::kOffMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int pair_id = int(blockIdx.x) >> 1;
  int *err = error_word(p);

  if (tid == 0) {
    for (int s = 0; s < Cfg<F8>::kRing; ++s) {
      mbar_init(bar(m.full[0][s]), 1);
      mbar_init(bar(m.full[1][s]), 1);
      mbar_init(bar(m.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(m.s_full[b]), 1);
      mbar_init(bar(m.s_free[b]), 2 * kSoftWarps);
      mbar_init(bar(m.o_ready[b]), 2 * kSoftWarps);
    }
    mbar_init(bar(m.q_full), F8 ? 2 * kSoftWarps : 1);
    mbar_init(bar(m.q_empty), 1);
    for (int i = 0; i < kTilePages; ++i) {
      mbar_init(bar(m.p_full[i]), 4);  // a page's two warps in each CTA
      mbar_init(bar(m.p_free[i]), 1);
    }
    mbar_init(bar(m.o_full), 1);
    mbar_init(bar(m.o_free), 2 * kSoftWarps);
    mbar_init(bar(m.drain), 2);
    m.abort = 0;
    fence_barrier_init();
  }
  // Allocating TMEM for a pair acts on both SMs: the other CTA has to be
  // running by then.
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tmem_alloc_pair(smem_u32(&m.tmem_base), 512);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(F8 ? &tm_k4 : &tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // blocks without pages: no partials, or the neutral pair
  if constexpr (KIND == kWindow) {
    for (int v = int(blockIdx.x); v < p.pair_blocks; v += int(gridDim.x)) {
      const ViewReq w = window_block<kPairRows>(p, v);
      if (tid == 0) checked_len(p, w.req, err);
      if (w.tiles != 0) continue;
      if (tid < 2 && w.rows > tid * kRows)
        info_ptr(p)[(2 * (v / p.batch) + tid) * p.batch + v % p.batch] = make_int4(-1, 0, 0, 0);
      uint4 *dst = reinterpret_cast<uint4 *>(p.out + size_t(w.row0) * kDv);
      for (int i = tid; i < w.rows * kDv / 8; i += kThreads) dst[i] = make_uint4(0, 0, 0, 0);
      for (int i = tid; i < w.rows; i += kThreads) p.lse[size_t(w.row0) + i] = -INFINITY;
    }
  }
  if constexpr (KIND == kChunk) {
    if (rank == 0 && tid == 128) info_ptr(p)[pair_id] = make_int4(0, 0, 0, 0);  // (the thread that sets it)
    // the searches below read these again and again
    for (int i = 32 * tid; i <= min(p.batch, 2048); i += 32 * kThreads) {
      asm volatile("prefetch.global.L1 [%0];" ::"l"(p.chunk_starts + i));
      if (i < p.batch) asm volatile("prefetch.global.L1 [%0];" ::"l"(p.seq_lens + i));
    }
    const int step = int(gridDim.x) * kThreads;
    for (int b = int(blockIdx.x) * kThreads + tid; b < p.batch; b += step) {
      checked_len(p, b, err);
      const int s0 = p.chunk_starts[b], s1 = p.chunk_starts[b + 1];
      if (s0 < 0 || s1 < s0 || s1 > p.chunk_tokens) atomicOr(err, kErrBadLen);
    }
    // blocks that see nothing: found by a lane each, written by the warp
    for (int v0 = (int(blockIdx.x) * kThreads + tid) & ~31; v0 < p.pair_blocks; v0 += step) {
      ViewReq w;
      if (v0 + lane < p.pair_blocks) w = block_view<KIND>(p, v0 + lane, nullptr);
      for (uint32_t left = __ballot_sync(0xffffffffu, w.rows > 0 && w.tiles == 0); left; left &= left - 1) {
        const int from = __ffs(left) - 1;
        const size_t row0 = __shfl_sync(0xffffffffu, w.row0, from);
        const int rows = __shfl_sync(0xffffffffu, w.rows, from);
        uint4 *dst = reinterpret_cast<uint4 *>(p.out + row0 * kDv);
        for (int i = lane; i < rows * kDv / 8; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
        for (int i = lane; i < rows; i += 32) p.lse[row0 + i] = -INFINITY;
      }
    }
  }
  if constexpr (KIND == kChunk) {
    schedule_chunks<kPieceTiles<F8, KIND>>(p, pair_id, p.pairs, &m.range, m.scratch);
  } else if constexpr (KIND == kWindow) {
    schedule_range<kPieceTiles<F8, KIND>, true>(
        p.pair_blocks, pair_id, p.pairs, [&](int v) { return tiles_of(block_view<KIND>(p, v, nullptr)); }, &m.range,
        m.scratch);
  } else {
    const int2 *groups = schedule_views<kPieceTiles<F8, KIND>>(
        p, p.pair_blocks, pair_id, p.pairs,
        [&](int v, const int2 *table, bool *unsure) {
          const ViewReq view = block_view<KIND>(p, v, table);
          *unsure |= view.unsure;
          return tiles_of(view);
        },
        &m.range, m.scratch);
    if (tid == 0) m.groups = groups;
    for (int v = int(blockIdx.x) * kThreads + tid; v < p.pair_blocks; v += int(gridDim.x) * kThreads)
      if (block_view<KIND>(p, v, groups).tiles == 0) pair_info_ptr(p)[v] = make_int4(-1, 0, 0, 0);
    if (KIND == kTails)
      for (int b = int(blockIdx.x) * kThreads + tid; b < p.batch; b += int(gridDim.x) * kThreads)
        check_view(p, b, err);
  }
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers and TMEM are ready
  tc_fence_after();
  const uint32_t tmem = m.tmem_base;
  const CtaRange r = m.range;

  if (r.start < r.end) {
    if (warp == 0) {
      if (lane == 0)
        produce<F8, KIND>(p, r, m, sbase + kOffQ, sbase + kOffRing, rank, &tm_q, &tm_k, &tm_k4, &tm_v, &tm_va,
                         &tm_vr, err);
    } else if (warp == 1) {
      if (rank == 0) score_mmas<F8, KIND>(p, r, m, sbase + kOffQ, sbase + kOffRing, tmem, err);
    } else if (warp == 2) {
      if (rank == 0) pv_mmas<F8, KIND>(p, r, m, sbase + kOffP, sbase + kOffRing, tmem, err);
    } else if (warp >= 4) {
      softmax<F8, KIND>(p, r, m, smem, tmem, rank, pair_id, err);
    }
    // no MMA may still read this CTA's shared memory, and no copy write it:
    // the MMAs waited for every copy unless a wait gave up
    __syncthreads();
    if (tid == 0) {
      mbar_wait_drain(bar(m.drain), 0, kDrainNs);
      if (m.abort) {  // let copies in flight land
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 1000000ull) {
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
  cluster_sync();  // the pair leaves together: neither SM takes another CTA before both gave up their TMEM
}

template <bool F8, int KIND>
cudaError_t launch(const DecodeParams &p, const CUtensorMap &tm_q, const PairMaps &m, cudaStream_t stream) {
  static SmemLimitOnce smem_limit;
  const cudaError_t e = smem_limit.ensure(decode_pair_kernel<F8, KIND>, smem_bytes<F8>());
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * p.pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<F8>();
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_pair_kernel<F8, KIND>, p, tm_q, m.k, m.k4, m.v, m.va, m.vr);
}

}  // namespace

// Launched after the pair kernel: the merge of the cut blocks of windows, or of the
// shared pages' and the tails' partials.  (Without the tails here, those follow
// in the other kernel, and the merge after them.)
cudaError_t launch_split_merge(const DecodeParams &p, int grid, cudaStream_t stream);
cudaError_t launch_shared_merge(const DecodeParams &p, int grid, cudaStream_t stream);
cudaError_t launch_chunk_merge(const DecodeParams &p, cudaStream_t stream);

// tm_q is read for a bf16 cache, m.k4 for an e4m3 one.
cudaError_t launch_decode_pair(const DecodeParams &p, const CUtensorMap &tm_q, const PairMaps &m,
                               cudaStream_t stream) {
  const bool f8 = p.kv_e4m3 != 0;
  if (p.view == kViewChunk) {
    const cudaError_t e = f8 ? launch<true, kChunk>(p, tm_q, m, stream) : launch<false, kChunk>(p, tm_q, m, stream);
    return e == cudaSuccess ? launch_chunk_merge(p, stream) : e;
  }
  if (p.view == kViewWindow) {
    const cudaError_t e = f8 ? launch<true, kWindow>(p, tm_q, m, stream) : launch<false, kWindow>(p, tm_q, m, stream);
    return e == cudaSuccess ? launch_split_merge(p, 2 * p.pairs, stream) : e;
  }
  if (p.pair_tails) {
    const cudaError_t e = f8 ? launch<true, kTails>(p, tm_q, m, stream) : launch<false, kTails>(p, tm_q, m, stream);
    return e == cudaSuccess ? launch_shared_merge(p, 2 * p.pairs, stream) : e;
  }
  return f8 ? launch<true, kWhole>(p, tm_q, m, stream) : launch<false, kWhole>(p, tm_q, m, stream);
}

}  // namespace mla
