// Attention of many query tokens over expanded keys and values (a head's 128 score dims
// and 128 value dims from the latent's up-projection, 64 rope dims shared by all heads):
//
//   s_ij = scale (q_i . [k_j ; rope_j]),  out_i = sum_j softmax(s_i)_j v_j
//
// 640 flops a (query head, key): two products with a softmax between them, bound by the
// tensor cores once a head's keys are read for some 100 queries.
//
// A block of 512 query tokens of one head belongs to a pair of CTAs (cta_group::2,
// M = 256): two halves of 256 tokens, 128 of each half in either CTA.  Each CTA loads
// half of every operand B (64 of a tile's 128 keys for the scores, 64 of the 128 value
// dims), so that a tile costs an SM 40 KB of loads for 512 queries, and two stages fit
// beside the queries (96 KB) and the rows on their way out (32 KB).
//
// TMEM (512 columns): scores of half 0 and 1 (128 each), outputs of half 0 and 1 (128
// each).  The softmax weights of a half, bf16, overlay its scores and are operand A of
// the second product straight from TMEM: nothing of them passes through shared memory.
//
// Roles (384 threads): warp 0 loads, warp 1 of the even CTA issues the MMAs, warp 3 looks
// the pieces of work up, warps 4..7 and 8..11 the softmax of half 0 and 1, a thread a row
// (no exchange between threads).  The halves take turns on the tensor cores: S0(j+1)
// follows P0(j) V(j) while the softmax of half 1 works on S1(j), and the other way round.  As MMAs complete in order,
// "S_h(j) is ready" also says that P_h(j-1) V(j-1) is done, so one barrier each way and
// half is all that the softmax needs, the rare rescale of an output (a maximum that grew
// by more than 2^8, as in the decode kernel) and a block's epilogue included.
//
// A block of up to 256 tokens fits one half.  Then both work on its rows, each on every
// second tile, and join their outputs at its end; blocks of one tile go to the halves in
// turn.  With one half only, the softmax and the products of a tile follow one another.
//
// Work: the 128-key tiles of all (head, block) in one line, head by head, cut into equal
// ranges, one a pair: the triangle of a causal mask evens out, and few queries over long
// keys spread over all SMs.  At most two blocks a pair are cut; their pieces leave fp32
// partials for a merge by their LSE.
//
// Measured: 8,192 queries over as many keys, 16 heads, no mask: 379 to 393 us, 1,750 to
// 1,810 TFLOP/s, 0.93 to 0.96 of the measured cuBLAS rate; 128 heads, causal: 1,670 to
// 1,700 us, 1,620 to 1,650; 2,048 queries over 10,240 keys, 128 heads: 1,010 us, 1,530 (all
// three under the power cap).  A tile of both halves takes some 3,300
// cycles where the clock is not the bound: the softmax of a half 1,500 (its 128
// exponentials a row are 512 of them), its products 1,280, the rest hand-overs.
#include "prefill_expanded.cuh"
#include "sm100.cuh"

namespace mla {
using namespace sm100;

namespace {

constexpr int kThreads = 384;
constexpr int kHalf = 256;     // query tokens of a half
constexpr int kKeys = 128;     // of a tile
constexpr int kKStages = 2, kVStages = 2;  // (three are no faster, and leave less room for outgoing rows)
constexpr int kQHalfBytes = 3 * 128 * 128;   // [dim block of 64][128 tokens][128 B], swizzled
constexpr int kKBytes = 3 * 64 * 128;        // [dim block of 64][64 keys][128 B]
constexpr int kVBytes = 128 * 128;           // [128 keys][128 B]
constexpr int kOffK = 2 * kQHalfBytes;
constexpr int kOffV = kOffK + kKStages * kKBytes;
constexpr int kStageRows = 32 * 128;         // rows of a softmax warp on their way out
constexpr int kOffOut = kOffV + kVStages * kVBytes;
constexpr int kOffMisc = kOffOut + 8 * kStageRows;
constexpr int kItems = 4;                    // pieces of work looked ahead
constexpr uint32_t kColS = 0, kColO = 256;   // half h: + 128 h
// Work is counted in tiles of one half.  A piece's boundary (Q, first scores, epilogue):
constexpr int kBoundary = 5;
constexpr long long kTimeoutClk = 4000000000ll;  // about 2 s
constexpr uint64_t kDrainNs = 200000000ull;
constexpr float kRescaleThreshold = 8.f;     // base-2 units

// A piece: tiles t0 .. t0 + n of a block of a head, of which half h takes the first
// cnt[h]; row i of the block sees the first min(max(hi0 + i, 0), nk) keys.  Split: half
// `half`, whose place the queries take, has the tiles t0, t0 + 2, ..., the other one
// those between; the halves go on taking turns from a piece to the next.
struct Item {
  int n;             // 0: no more
  int head, q0, rows, k0, t0, hi0, nk, end;
  int cnt[2];
  int pieces;        // of the block, this one among them
  int first;         // this pair begins the block
  int split, half;
};

struct Misc {
  Item items[kItems];
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][2], o_full[2], drain;  // p_full: [half][64 keys]
  uint64_t join[2];        // of the softmax warps
  uint32_t tmem_base;
  int abort;
  float stats[2][2][128];  // split blocks: maximum and sum of each half's rows
  CtaRange range;
  long long scratch[kThreads / 32 + 1];
};
constexpr int kSmemBytes = kOffMisc + int(sizeof(Misc)) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");

__device__ __forceinline__ uint32_t bar(uint64_t &b) { return smem_u32(&b); }
__device__ __forceinline__ int *error_word(const ExpandedParams &p) { return reinterpret_cast<int *>(p.ws); }
__device__ __forceinline__ int4 *records(const ExpandedParams &p) {
  return reinterpret_cast<int4 *>(p.ws + expanded_layout(p.pairs).rec);
}
__device__ __forceinline__ float *slot_lse(const ExpandedParams &p) {
  return reinterpret_cast<float *>(p.ws + expanded_layout(p.pairs).lse);
}
__device__ __forceinline__ float *slot_out(const ExpandedParams &p) {
  return reinterpret_cast<float *>(p.ws + expanded_layout(p.pairs).out);
}

__device__ __forceinline__ int start_in(const int32_t *starts, int b, int most) {
  return min(max(starts[b], 0), most);
}

// A block of up to 512 query tokens of one request.  Request b's blocks have ids
// floor(its first token / 512) + b and up, which leaves it as many as it needs; ids
// between are empty.
struct Block {
  int rows = 0;      // query tokens
  int q0 = 0;        // the first of them
  int k0 = 0;        // the request's first key
  int hi0 = 0, nk = 0;  // row i sees the first min(max(hi0 + i, 0), nk) keys
  int tiles = 0;     // of 128 keys that some row sees
  int half0 = 0;     // of these, the tiles that a row of half 0 sees
  __device__ __forceinline__ int sees(int row) const {
    return int(min(max((long long)hi0 + row, 0ll), (long long)nk));
  }
  __device__ __forceinline__ int end() const { return sees(rows - 1); }
  // one half holds all rows: the halves then share them and take turns at the tiles
  __device__ __forceinline__ bool split() const { return rows <= kHalf; }
  __device__ __forceinline__ int weight() const { return split() ? 1 : 2; }
  __device__ __forceinline__ long long cost() const {
    return tiles ? (long long)tiles * weight() + kBoundary : 0;
  }
  // tiles of half h among t0 .. t1 - 1 (not split)
  __device__ __forceinline__ int count(int h, int t0, int t1) const {
    return max(0, min(t1, h ? tiles : half0) - t0);
  }
};

__device__ __forceinline__ Block make_block(const ExpandedParams &p, int u) {
  Block b;
  int lo = 0, hi = p.batch - 1;  // the last request whose blocks start at or before u
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start_in(p.q_starts, mid, p.q_tokens) / kExpRows + mid <= u) lo = mid;
    else hi = mid - 1;
  }
  const int s0 = start_in(p.q_starts, lo, p.q_tokens), n = start_in(p.q_starts, lo + 1, p.q_tokens) - s0;
  const long long first = (long long)(u - s0 / kExpRows - lo) * kExpRows;
  if (first < 0 || first >= n) return b;
  b.rows = min(kExpRows, n - int(first));
  b.q0 = s0 + int(first);
  b.k0 = start_in(p.k_starts, lo, p.k_tokens);
  b.nk = max(0, start_in(p.k_starts, lo + 1, p.k_tokens) - b.k0);
  // (without a mask, hi0 is large enough for every row; nk <= 2^30)
  b.hi0 = p.causal ? b.nk - n + int(first) + 1 : b.nk;
  b.tiles = (b.end() + kKeys - 1) / kKeys;
  b.half0 = (b.sees(min(b.rows, kHalf) - 1) + kKeys - 1) / kKeys;
  return b;
}

// This pair's range of the line of all heads' blocks, which is the line of one head
// `heads` times over.  Block-wide.
__device__ __forceinline__ void schedule_heads(const ExpandedParams &p, int idx, CtaRange *r, long long *scratch) {
  const int tid = threadIdx.x, nw = kThreads / 32, lane = tid & 31, warp = tid >> 5;
  long long mine = 0;
  for (int u = tid; u < p.blocks; u += kThreads) mine += make_block(p, u).cost();
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) scratch[warp] = mine;
  __syncthreads();
  long long one = 0;
  for (int w = 0; w < nw; ++w) one += scratch[w];
  const long long C = one * p.heads;
  // (at least two units a pair: every pair inside a block has a whole tile's first unit)
  const int g = int(C / 2 < (long long)p.pairs ? C / 2 : (long long)p.pairs);
  const bool has = idx < g;
  const long long start = has ? sched_start(idx, C, g) : 0, end = has ? sched_start(idx + 1, C, g) : 0;
  const long long h0 = has ? start / one : 0, r0 = start - h0 * one;
  if (tid == 0) {
    r->total = C;
    r->g_eff = g;
    r->start = start;
    r->end = end;
    r->v_begin = int((h0 + 1) * p.blocks);  // where r0 lies behind the last block's tiles
    r->p_begin = (h0 + 1) * one;
  }
  __syncthreads();  // (scratch is read, the defaults are written)
  if (!has) return;
  // the first block whose tiles end after r0; its predecessor's end at `excl - kBoundary`
  long long base = 0;
  for (int u0 = 0; u0 < p.blocks && base - kBoundary <= r0; u0 += kThreads) {
    const int u = u0 + tid;
    const long long cst = u < p.blocks ? make_block(p, u).cost() : 0;
    long long incl = cst;
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    long long before = 0, chunk = 0;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) before += scratch[w];
      chunk += scratch[w];
    }
    const long long excl = base + before + incl - cst;
    if (cst > 0 && excl + cst - kBoundary > r0 && excl - kBoundary <= r0) {
      r->v_begin = int(h0 * p.blocks) + u;
      r->p_begin = h0 * one + excl;
    }
    base += chunk;
  }
  __syncthreads();
}

// The pieces of this pair's range, in order, by one warp, a few ahead of the others: worked
// out by every role for itself between two pieces, this cost the softmax and the MMAs some
// 3,800 cycles a piece.  A lane holds a block, so that a batch padded with empty requests
// is passed 32 at a time.
__device__ __forceinline__ void look_ahead(const ExpandedParams &p, Misc &m, int pair_id) {
  constexpr uint32_t kAll = 0xffffffffu;
  const CtaRange &r = m.range;
  const int lane = threadIdx.x & 31;
  const long long start = r.start, end = r.end;
  int head = r.v_begin / p.blocks, u0 = (r.v_begin - head * p.blocks) & ~31, held = -1, slot = 0;
  uint32_t lap = 1;
  bool ok = true;
  int half = 0;  // whose turn it is
  Block b;
  long long pv = 0;   // cost before block u0 of this head
  bool first = true;
  while (ok && head < p.heads) {
    if (held != u0) b = u0 + lane < p.blocks ? make_block(p, u0 + lane) : Block();
    held = u0;
    long long incl = b.cost();
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += y;
    }
    if (first) {  // p_begin is the cost before block v_begin, some lane of this group
      const int from = (r.v_begin - head * p.blocks) & 31;
      pv = r.p_begin - __shfl_sync(kAll, incl - b.cost(), from);
      first = false;
    }
    if (pv >= end) break;
    const long long at = pv + incl - b.cost();  // of this lane's block
    // a tile belongs to the pair that has its first unit
    const int wgt = b.weight();
    const int t0 = int((max(start, at) - at + wgt - 1) / wgt);
    const int t1 = int((min(end, at + (long long)b.tiles * wgt) - at + wgt - 1) / wgt);
    const bool mine = b.tiles > 0 && at < end && t0 < t1;
    Item it;
    if (mine) {
      const int c_first = sched_owner_short(at, r.total, r.g_eff);
      it.n = t1 - t0;
      it.head = head;
      it.q0 = b.q0;
      it.rows = b.rows;
      it.k0 = b.k0;
      it.t0 = t0;
      it.hi0 = b.hi0;
      it.nk = b.nk;
      it.end = b.end();
      it.pieces = sched_owner_short(at + (long long)(b.tiles - 1) * wgt, r.total, r.g_eff) - c_first + 1;
      it.first = pair_id == c_first;
      it.split = b.split();
    }
    for (uint32_t left = __ballot_sync(kAll, mine); ok && left; left &= left - 1) {
      const int from = __ffs(left) - 1;
      ok = __all_sync(kAll, mbar_wait_clk(bar(m.item_empty[slot]), lap, &m.abort, kTimeoutClk));
      const int split = __shfl_sync(kAll, int(b.split()), from), n = __shfl_sync(kAll, t1 - t0, from);
      if (ok && lane == from) {
        it.half = split ? half : 0;
        it.cnt[0] = split ? (n + 1 - half) / 2 : b.count(0, t0, t1);
        it.cnt[1] = split ? n - it.cnt[0] : b.count(1, t0, t1);
        m.items[slot] = it;
        mbar_arrive(bar(m.item_full[slot]));
      }
      __syncwarp();
      half = split ? (half + n) & 1 : 0;
      if (++slot == kItems) slot = 0, lap ^= 1;
    }
    pv += __shfl_sync(kAll, incl, 31);
    u0 += 32;
    if (u0 >= p.blocks) u0 = 0, ++head;
  }
  ok = ok && __all_sync(kAll, mbar_wait_clk(bar(m.item_empty[slot]), lap, &m.abort, kTimeoutClk));
  if (ok && lane == 0) {
    m.items[slot].n = 0;
    mbar_arrive(bar(m.item_full[slot]));
  }
  __syncwarp();
}

// A role's way through them.  One lane a warp waits and says it has read.
struct Items {
  Misc &m;
  int slot = 0;
  uint32_t lap = 0;
  __device__ __forceinline__ explicit Items(Misc &m_) : m(m_) {}
  // the next piece (n = 0: none, or a wait that gave up, then also !*ok); WARP: by a
  // whole warp, else by one thread
  template <bool WARP>
  __device__ __forceinline__ Item next(bool *ok) {
    bool got = mbar_wait_clk(bar(m.item_full[slot]), lap, &m.abort, kTimeoutClk);
    if (WARP) got = __all_sync(0xffffffffu, got);
    if (!got) {
      *ok = false;
      return Item{};
    }
    const Item it = m.items[slot];
    if (WARP) __syncwarp();
    if (!WARP || (threadIdx.x & 31) == 0) mbar_arrive(bar(m.item_empty[slot]));
    if (++slot == kItems) slot = 0, lap ^= 1;
    return it;
  }
};

// ------------------------------------------------------------------ producer

// The value rows of a tile of which only the first `left` (< 128) are seen: the others may
// hold anything (the next request's rows, or what was there), and weights of 0 do not
// keep a NaN out of the product.  They are loaded from past the end, as zeros.
static __device__ __noinline__ void load_seen_v(uint32_t dst, uint32_t full, const CUtensorMap *tm_va,
                                                const CUtensorMap *tm_vr, int d0, int head, int key, int left,
                                                int none) {
#pragma unroll 1
  for (int a = 0; a < kKeys; a += 8) {
    if (a + 8 <= left || a >= left) {
      tma_load_3d_pair(dst + a * 128, tm_va, full, d0, head, a < left ? key + a : none);
      continue;
    }
#pragma unroll 1
    for (int k = a; k < a + 8; ++k)
      tma_load_3d_pair(dst + k * 128, tm_vr, full, d0, head, k < left ? key + k : none);
  }
}

__device__ __forceinline__ void produce(const ExpandedParams &p, Misc &m, uint32_t sbase,
                                        uint32_t rank, const CUtensorMap *tm_q, const CUtensorMap *tm_kn,
                                        const CUtensorMap *tm_kr, const CUtensorMap *tm_v, const CUtensorMap *tm_va,
                                        const CUtensorMap *tm_vr, int *err) {
  volatile int *abort = &m.abort;
  const bool leader = rank == 0;
  const uint32_t k_full = map_to_rank(bar(m.k_full[0]), 0), v_full = map_to_rank(bar(m.v_full[0]), 0);
  const uint32_t q_full = map_to_rank(bar(m.q_full[0]), 0);
  int kst = 0, vst = 0;
  uint32_t k_lap = 1, v_lap = 1, q_lap[2] = {1, 1};  // parity of the empty barriers' last phase
  bool ok = true;
  Items items(m);
  auto load_k = [&](const Item &w, int j) {
    const int key = w.k0 + (w.t0 + j) * kKeys + 64 * int(rank);
    if (!mbar_wait_clk(bar(m.k_empty[kst]), k_lap, abort, kTimeoutClk)) return false;
    if (leader) mbar_arrive_expect_tx(bar(m.k_full[kst]), 2 * kKBytes);
    const uint32_t dst = sbase + kOffK + kst * kKBytes;
    tma_load_3d_pair(dst, tm_kn, k_full + 8 * kst, 0, w.head, key);
    tma_load_3d_pair(dst + 8192, tm_kn, k_full + 8 * kst, 64, w.head, key);
    tma_load_2d_pair(dst + 16384, tm_kr, k_full + 8 * kst, 0, key);
    if (++kst == kKStages) kst = 0, k_lap ^= 1;
    return true;
  };
  auto load_v = [&](int head, int key, int left) {
    if (!mbar_wait_clk(bar(m.v_empty[vst]), v_lap, abort, kTimeoutClk)) return false;
    if (leader) mbar_arrive_expect_tx(bar(m.v_full[vst]), 2 * kVBytes);
    const uint32_t dst = sbase + kOffV + vst * kVBytes;
    if (left >= kKeys) tma_load_3d_pair(dst, tm_v, v_full + 8 * vst, 64 * int(rank), head, key);
    else load_seen_v(dst, v_full + 8 * vst, tm_va, tm_vr, 64 * int(rank), head, key, left, p.k_tokens);
    if (++vst == kVStages) vst = 0, v_lap ^= 1;
    return true;
  };
  auto load_q = [&](const Item &w, int h) {
    if (!mbar_wait_clk(bar(m.q_empty[h]), q_lap[h], abort, kTimeoutClk)) return false;
    q_lap[h] ^= 1;
    if (leader) mbar_arrive_expect_tx(bar(m.q_full[h]), 2 * kQHalfBytes);
    for (int i = 0; i < 3; ++i)
      tma_load_3d_pair(sbase + h * kQHalfBytes + i * 16384, tm_q, q_full + 8 * h, 64 * i, w.head,
                       w.q0 + (w.split ? 0 : kHalf * h) + 128 * int(rank));
    return true;
  };
  // Keys run a tile ahead of values, which the products need later, from piece to piece
  // too: (head, key, keys left) is the tile whose values are still to come.  The queries
  // of a split piece after one of an odd number of tiles have a place that it leaves free.
  // After an even number they have its place again and wait for its last scores, and so do
  // the owed values behind them; a place that took turns by itself was no faster (100
  // requests of 256 queries over 256 keys, 16 heads: 116.6 us against 116.1).  The queries
  // of other pieces wait for the last scores before them, and the values go first.
  int v_head = 0, v_key = 0, v_left = 0;
  for (Item w = items.next<false>(&ok); ok && w.n; w = items.next<false>(&ok)) {
    for (int j = 0; ok && j < w.n; ++j) {
      ok = load_k(w, j);
      if (ok && j == 0 && w.split) ok = load_q(w, w.half);
      if (ok && v_left > 0) ok = load_v(v_head, v_key, v_left);
      if (j == 0 && !w.split)
        for (int h = 0; ok && h < 2; ++h)
          if (w.cnt[h]) ok = load_q(w, h);
      v_head = w.head;
      v_key = w.k0 + (w.t0 + j) * kKeys;
      v_left = w.end - (w.t0 + j) * kKeys;
    }
  }
  if (ok && v_left > 0) ok = load_v(v_head, v_key, v_left);
  if (!ok) atomicOr(err, kErrTimeout);
}

// ------------------------------------------------------------------ MMAs (even CTA)

// A wait of a whole warp (the same answer in every lane).
__device__ __forceinline__ bool warp_wait(uint32_t b, uint32_t parity, volatile int *abort) {
  return __all_sync(0xffffffffu, mbar_wait_clk(b, parity, abort, kTimeoutClk));
}

__device__ __forceinline__ void mmas(Misc &m, uint32_t sbase, uint32_t tmem, int *err) {
  volatile int *abort = &m.abort;
  const uint32_t idesc_s = idesc_bf16_f32(256, 128, false, false), idesc_o = idesc_bf16_f32(256, 128, false, true);
  const uint64_t dq = smem_desc_sw128(sbase, 16, 1024), dk = smem_desc_sw128(sbase + kOffK, 16, 1024);
  const uint64_t dv = smem_desc_sw128(sbase + kOffV, 16384, 1024);  // MN-major: 8-key groups 1 KB apart
  int kst = 0, vst = 0;
  uint32_t k_lap = 0, v_lap = 0, q_lap = 0, p_lap = 0;  // q, p: bit h
  bool ok = true;
  // half h's weights times the values of the tile at vst; the first 64 keys' product runs
  // while the softmax works on the others' weights (five requests of 215..667 queries: 190
  // -> 179 us)
  auto values = [&](int h, bool begin, bool end) {
    if (!warp_wait(bar(m.v_full[vst]), v_lap, abort)) return false;
    const uint32_t o = tmem + kColO + 128 * h, a = tmem + kColS + 128 * h;
    const uint64_t v = dv + ((vst * kVBytes) >> 4);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      if (!warp_wait(bar(m.p_full[h][part]), (p_lap >> h) & 1, abort)) return false;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int ks = 4 * part; ks < 4 * part + 4; ++ks)
          mma_bf16_ts_pair(o, a + 8 * ks, v + ((ks * 2048) >> 4), idesc_o, !begin || ks > 0);
        if (part && end) mma_commit_pair(bar(m.o_full[h]));
      }
      __syncwarp();
    }
    p_lap ^= 1u << h;
    return true;
  };
  // half h's scores of the tile at kst, of the queries in place qh
  auto scores = [&](int h, int qh, bool begin, bool end) {
    if (begin) {
      if (!warp_wait(bar(m.q_full[qh]), (q_lap >> qh) & 1, abort)) return false;
      q_lap ^= 1u << qh;
    }
    if (elect_one()) {
      const uint64_t q = dq + ((qh * kQHalfBytes) >> 4), k = dk + ((kst * kKBytes) >> 4);
#pragma unroll
      for (int ks = 0; ks < 12; ++ks)
        mma_bf16_ss_pair(tmem + kColS + 128 * h, q + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4),
                         k + (((ks >> 2) * 8192 + (ks & 3) * 32) >> 4), idesc_s, ks > 0);
      mma_commit_pair(bar(m.s_full[h]));
      if (end) mma_commit_pair(bar(m.q_empty[qh]));
    }
    __syncwarp();
    return true;
  };
  auto done_values = [&] {
    if (elect_one()) mma_commit_pair(bar(m.v_empty[vst]));
    __syncwarp();
    if (++vst == kVStages) vst = 0, v_lap ^= 1;
  };
  auto done_scores = [&] {
    if (elect_one()) mma_commit_pair(bar(m.k_empty[kst]));
    __syncwarp();
    if (++kst == kKStages) kst = 0, k_lap ^= 1;
  };
  // Split tiles whose weights are still to come: bit h, and whether they begin or end
  // their half's part of a piece.  They are multiplied in the tiles' order, `next` first.
  uint32_t owed = 0, begins = 0, ends = 0;
  int next = 0;
  auto settle = [&](int h) {
    if (!values(h, (begins >> h) & 1, (ends >> h) & 1)) return false;
    done_values();
    owed &= ~(1u << h);
    next = h ^ 1;
    return true;
  };
  Items items(m);
  for (Item w = items.next<true>(&ok); ok && w.n; w = items.next<true>(&ok)) {
    const int n = w.n;
    if (w.split) {
      for (int j = 0; ok && j < n; ++j) {
        const int h = w.half ^ (j & 1);
        if (!owed) next = h;
        if ((owed >> h) & 1) ok = settle(h);
        ok = ok && warp_wait(bar(m.k_full[kst]), k_lap, abort) && scores(h, w.half, j == 0, j == n - 1);
        if (!ok) break;
        done_scores();
        owed |= 1u << h;
        begins = (begins & ~(1u << h)) | uint32_t(j < 2) << h;
        ends = (ends & ~(1u << h)) | uint32_t(j >= n - 2) << h;
      }
      continue;
    }
    while (ok && owed) ok = settle(next);
    // step j: the weights of tile j - 1 times its values, then tile j's scores, half by half
    for (int j = 0; ok && j <= n; ++j) {
      if (j < n) ok = warp_wait(bar(m.k_full[kst]), k_lap, abort);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (ok && j > 0 && j <= w.cnt[h]) {
          // (both halves wait for the same values)
          ok = values(h, j == 1, j == w.cnt[h]);
        }
        if (ok && j < w.cnt[h]) ok = scores(h, h, j == 0, j == w.cnt[h] - 1);
      }
      if (!ok) break;
      if (j > 0) done_values();
      if (j < n) done_scores();
    }
  }
  while (ok && owed) ok = settle(next);
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
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{ .reg .b64 x, y, z, d; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7};\n"
      "fma.rn.f32x2 d, x, y, z; mov.b64 {%0, %1}, d; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}

// Sends a warp's 32 rows of 128 bytes, lane i's row in v, to dst + i * stride (rows below
// `rows` only): through shared memory, so that a store instruction writes four whole rows
// and not a piece of 32 (which took the epilogue 4,000 to 6,000 cycles).
__device__ __forceinline__ void send_rows(unsigned char *stage, const uint32_t (&v)[32], void *dst, size_t stride,
                                          int rows) {
  const int lane = threadIdx.x & 31;
  const int c = lane & 7;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    *reinterpret_cast<uint4 *>(stage + lane * 128 + ((k ^ c) << 4)) =
        make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int i = 4 * k + (lane >> 3);
    const uint4 x = *reinterpret_cast<const uint4 *>(stage + i * 128 + ((c ^ (i & 7)) << 4));
    if (i < rows) *reinterpret_cast<uint4 *>(static_cast<unsigned char *>(dst) + i * stride + 16 * c) = x;
  }
  __syncwarp();
}

__device__ __forceinline__ void softmax(const ExpandedParams &p, Misc &m, unsigned char *smem, uint32_t tmem,
                                        uint32_t rank, int pair_id, int *err) {
  volatile int *abort = &m.abort;
  const int warp = int(threadIdx.x >> 5) - 4, lane = threadIdx.x & 31;
  const int h = warp >> 2, q = warp & 3;
  const int hrow = 32 * q + lane;
  const uint32_t lanes = uint32_t(32 * q) << 16;
  const uint32_t t_s = tmem + lanes + kColS + 128 * h, t_o = tmem + lanes + kColO + 128 * h,
                 t_o2 = tmem + lanes + kColO + 128 * (h ^ 1);
  const uint32_t p_full = map_to_rank(bar(m.p_full[h][0]), 0);
  const float cs = p.score_scale_log2;
  unsigned char *stage = smem + kOffOut + warp * kStageRows;
  uint32_t s_lap = 0, o_lap = 0, join_lap = 0;
  // (no hardware barrier: a warp whose wait gave up would leave the others in it)
  auto join = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(m.join[k]));
    return bool(__all_sync(0xffffffffu, mbar_wait_clk(bar(m.join[k]), join_lap, abort, kTimeoutClk)));
  };
  bool ok = true;
  Items items(m);
  Item w = items.next<true>(&ok);
  while (ok && w.n) {
    const int cnt = h ? w.cnt[1] : w.cnt[0];
    const int row = (w.split ? 0 : kHalf * h) + 128 * int(rank) + hrow;  // within the block
    // keys from the tile on that the row sees
    int left = (row < w.rows ? int(min(max((long long)w.hi0 + row, 0ll), (long long)w.nk)) : 0) -
               (w.t0 + (w.split ? h ^ w.half : 0)) * kKeys;
    float mrun = -INFINITY, sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < cnt; ++j, left -= w.split ? 2 * kKeys : kKeys) {
      ok = __all_sync(0xffffffffu, mbar_wait_clk(bar(m.s_full[h]), s_lap, abort, kTimeoutClk));
      s_lap ^= 1;
      if (!ok) break;
      tc_fence_after();
      uint32_t a[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, a[c]);
      tmem_wait_ld();
      if (left < kKeys) {
#pragma unroll
        for (int i = 0; i < kKeys; ++i) a[i >> 5][i & 31] = i < left ? a[i >> 5][i & 31] : 0xff800000u;
      }
      auto x = [&](int i) { return __uint_as_float(a[i >> 5][i & 31]); };
      float mx[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) mx[k] = fmaxf(x(k), x(8 + k));
#pragma unroll
      for (int i = 16; i < kKeys; i += 16)
#pragma unroll
        for (int k = 0; k < 8; ++k) mx[k] = max3(mx[k], x(i + k), x(i + 8 + k));
      const float top = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * cs;
      float alpha = 1.f;
      if (j == 0) {
        mrun = top;
      } else if (top > mrun + kRescaleThreshold) {
        alpha = exp2f(mrun - top);
        mrun = top;
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[k] *= alpha;
      }
      if (__any_sync(0xffffffffu, alpha != 1.f)) {  // O *= alpha
#pragma unroll 1
        for (int c = 0; c < kDvx; c += 16) {
          uint32_t o[16];
          tmem_ld16(t_o + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st16(t_o + c, o);
        }
      }
      // a row that has seen no key yet keeps a -inf maximum: its weights are 0
      const float mref = mrun == -INFINITY ? 0.f : mrun;
      const float2 cs2 = make_float2(cs, cs), mn2 = make_float2(-mref, -mref);
      // (sums one by one: the packed addition made the loop half as slow again)
      uint32_t pk[4][16];
#pragma unroll
      for (int i = 0; i < kKeys / 2; ++i) {
        const float2 y = fma2(make_float2(x(2 * i), x(2 * i + 1)), cs2, mn2);
        const float e0 = exp2_approx(y.x), e1 = exp2_approx(y.y);
        sum[i & 1] += e0;
        sum[2 + (i & 1)] += e1;
        pk[i >> 4][i & 15] = pack_bf16(e0, e1);
        if (i == 31) {  // 64 keys' weights are on their way, and said to be there 16 keys later
#pragma unroll
          for (int c = 0; c < 2; ++c) tmem_st16(t_s + 16 * c, pk[c]);
        }
        if (i == 39) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(p_full);
        }
      }
#pragma unroll
      for (int c = 2; c < 4; ++c) tmem_st16(t_s + 16 * c, pk[c]);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(p_full + 8);
    }
    // ---- the piece's rows: O / sum and the LSE
    float total = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    // (before the piece's stores: an arrival waits for those that its thread has made)
    const Item next = items.next<true>(&ok);
    if (w.split && cnt == 0) {  // the other half has the piece's only tile
      w = next;
      continue;
    }
    const bool joined = w.split && w.n > 1;
    if (cnt > 0) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait_clk(bar(m.o_full[h]), o_lap, abort, kTimeoutClk));
      o_lap ^= 1;
    }
    float mine = 1.f, other = 0.f;  // weights of the halves' outputs
    if (joined) {  // the two halves' pieces of a row: this thread's, and that of the other half's thread
      m.stats[h][0][hrow] = mrun;
      m.stats[h][1][hrow] = total;
      tc_fence_before();
      ok = ok && join(0);  // both outputs are ready
      const float m2 = m.stats[h ^ 1][0][hrow], top = fmaxf(mrun, m2), mref = top == -INFINITY ? 0.f : top;
      mine = exp2f(mrun - mref);
      other = exp2f(m2 - mref);
      total = mine * total + other * m.stats[h ^ 1][1][hrow];
      mrun = top;
    }
    if (!ok) break;
    const float inv = total > 0.f ? 1.f / total : 0.f;
    const float lse2 = mrun + log2f(total);
    mine *= inv;
    other *= inv;
    // a pair's slot 0: a block that another pair began; slot 1: one that it begins
    const size_t slot = (2 * size_t(pair_id) + (w.t0 == 0 ? 1 : 0)) * kExpRows + row;
    const size_t orow = size_t(w.q0 + row) * p.heads + w.head;
    const bool cut = w.pieces > 1;
    const int rows = w.rows - (row - lane);  // from this warp's first on
    tc_fence_after();
    // (uniform: a warp without rows has only its place in the barriers)
    if (rows > 0) {
      if (lane < rows && !(joined && h)) {
        if (cut) slot_lse(p)[slot] = lse2;
        else p.lse[orow] = p.lse_base2 ? lse2 : lse2 * kLn2;
      }
      // joined: half h writes dims 64 h .. 64 h + 63
      const int c_end = joined ? 64 * h + 64 : kDvx;
#pragma unroll 1
      for (int c = joined ? 64 * h : 0; c < c_end; c += 64) {
        uint32_t o[2][32];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (cnt > 0) {
            tmem_ld32(t_o + c + 32 * k, o[k]);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[k][i] = __float_as_uint(__uint_as_float(o[k][i]) * mine);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[k][i] = 0;
          }
          if (joined) {
            uint32_t z[32];
            tmem_ld32(t_o2 + c + 32 * k, z);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[k][i] = __float_as_uint(fmaf(__uint_as_float(z[i]), other, __uint_as_float(o[k][i])));
          }
        }
        if (cut) {
          float *dst = slot_out(p) + (slot - lane) * kDvx + c;
          send_rows(stage, o[0], dst, kDvx * 4, rows);
          send_rows(stage, o[1], dst + 32, kDvx * 4, rows);
        } else {
          uint32_t v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            v[i] = pack_bf16(__uint_as_float(o[i >> 4][2 * (i & 15)]), __uint_as_float(o[i >> 4][2 * (i & 15) + 1]));
          send_rows(stage, v, p.out + (orow - size_t(lane) * p.heads) * kDvx + c, size_t(p.heads) * kDvx * 2, rows);
        }
      }
    }
    tc_fence_before();
    if (joined) {  // both outputs and their statistics are read
      ok = join(1);
      join_lap ^= 1;
    }
    if (cut && w.first && rank == 0 && (threadIdx.x & 127) == 0 && h == (joined ? 0 : w.half))
      records(p)[pair_id] = make_int4(w.pieces, w.q0, w.rows, w.head);
    w = next;
  }
  if (!ok) atomicOr(err, kErrTimeout);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prefill_expanded_kernel(const __grid_constant__ ExpandedParams p, const __grid_constant__ CUtensorMap tm_q,
                            const __grid_constant__ CUtensorMap tm_kn, const __grid_constant__ CUtensorMap tm_kr,
                            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_va,
                            const __grid_constant__ CUtensorMap tm_vr) {
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), pad = ((raw + 1023u) & ~1023u) - raw;
  const uint32_t sbase = raw + pad;
  Misc &m = *reinterpret_cast<Misc *>(smem_raw + pad + kOffMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int pair_id = int(blockIdx.x) >> 1;
  int *err = error_word(p);

  if (tid == 0) {
    for (int i = 0; i < kItems; ++i) {
      mbar_init(bar(m.item_full[i]), 1);
      mbar_init(bar(m.item_empty[i]), rank == 0 ? 10 : 9);  // loads, softmax warps; MMAs
    }
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(bar(m.k_full[s]), 1);
      mbar_init(bar(m.k_empty[s]), 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(bar(m.v_full[s]), 1);
      mbar_init(bar(m.v_empty[s]), 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(bar(m.q_full[h]), 1);
      mbar_init(bar(m.q_empty[h]), 1);
      mbar_init(bar(m.s_full[h]), 1);
      for (int part = 0; part < 2; ++part) mbar_init(bar(m.p_full[h][part]), 8);  // a half's four warps in each CTA
      mbar_init(bar(m.o_full[h]), 1);
      mbar_init(bar(m.join[h]), 8);
    }
    mbar_init(bar(m.drain), 1);
    m.abort = 0;
    fence_barrier_init();
  }
  // Allocating TMEM for a pair acts on both SMs: the other CTA has to be running by then.
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tmem_alloc_pair(smem_u32(&m.tmem_base), 512);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_kn);
    tma_prefetch_desc(&tm_kr);
    tma_prefetch_desc(&tm_v);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (rank == 0 && tid == 128) records(p)[pair_id] = make_int4(0, 0, 0, 0);  // (ordered before the one that may follow by the barriers below)
  const int step = int(gridDim.x) * kThreads;
  for (int b = int(blockIdx.x) * kThreads + tid; b < p.batch; b += step) {
    const int q0 = p.q_starts[b], q1 = p.q_starts[b + 1], k0 = p.k_starts[b], k1 = p.k_starts[b + 1];
    if (q0 < 0 || q1 < q0 || q1 > p.q_tokens || k0 < 0 || k1 < k0 || k1 > p.k_tokens) atomicOr(err, kErrBadLen);
  }
  // blocks that see nothing: found by a lane each, written by the warp
  for (int u0 = (int(blockIdx.x) * kThreads + tid) & ~31; u0 < p.blocks; u0 += step) {
    Block b;
    if (u0 + lane < p.blocks) b = make_block(p, u0 + lane);
    for (uint32_t left = __ballot_sync(0xffffffffu, b.rows > 0 && b.tiles == 0); left; left &= left - 1) {
      const int from = __ffs(left) - 1;
      const size_t row0 = size_t(__shfl_sync(0xffffffffu, b.q0, from)) * p.heads;
      const int rows = __shfl_sync(0xffffffffu, b.rows, from) * p.heads;
      uint4 *dst = reinterpret_cast<uint4 *>(p.out + row0 * kDvx);
      for (int i = lane; i < rows * kDvx / 8; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
      for (int i = lane; i < rows; i += 32) p.lse[row0 + i] = -INFINITY;
    }
  }
  schedule_heads(p, pair_id, &m.range, m.scratch);
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers and TMEM are ready
  tc_fence_after();
  const uint32_t tmem = m.tmem_base;
  const CtaRange &r = m.range;

  if (r.start < r.end) {
    if (warp == 0) {
      if (lane == 0) produce(p, m, sbase, rank, &tm_q, &tm_kn, &tm_kr, &tm_v, &tm_va, &tm_vr, err);
    } else if (warp == 1) {
      if (rank == 0) mmas(m, sbase, tmem, err);
    } else if (warp == 3) {
      look_ahead(p, m, pair_id);
    } else if (warp >= 4) {
      softmax(p, m, smem_raw + pad, tmem, rank, pair_id, err);
    }
    // no MMA may still read this CTA's shared memory, and no copy write it: the MMAs
    // waited for every copy unless a wait gave up
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

// ------------------------------------------------------------------ merge

// The blocks that the schedule cut: pair c's record is that of the block it begins and
// others go on with.  A warp a row: the LSE-weighted combine of its pieces, the first in
// slot 1 of pair c, the others in slot 0 of the pairs after it.
constexpr int kMergeWarps = 8;
__global__ void __launch_bounds__(kMergeWarps * 32) expanded_merge_kernel(const __grid_constant__ ExpandedParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  const int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  const int4 rec = records(p)[c];
  // (a call whose bounded wait gave up may leave anything here)
  if (rec.x < 2 || rec.x > p.pairs - c || rec.z > kExpRows || row >= rec.z || rec.y < 0 ||
      rec.y > p.q_tokens - rec.z || rec.w < 0 || rec.w >= p.heads)
    return;
  const int ns = rec.x;
  auto slot = [&](int k) { return (size_t(2) * (c + k) + (k == 0 ? 1 : 0)) * kExpRows + row; };
  const float *sl = slot_lse(p);
  float mx = -INFINITY;
  for (int k = lane; k < ns; k += 32) mx = fmaxf(mx, sl[slot(k)]);
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float mref = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < ns; ++k) {
    const float w = exp2f(sl[slot(k)] - mref);
    const float4 x = reinterpret_cast<const float4 *>(slot_out(p) + slot(k) * kDvx)[lane];
    sum += w;
    acc.x += w * x.x;
    acc.y += w * x.y;
    acc.z += w * x.z;
    acc.w += w * x.w;
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const size_t orow = size_t(rec.y + row) * p.heads + rec.w;
  reinterpret_cast<uint2 *>(p.out + orow * kDvx)[lane] =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (lane == 0) {
    const float lse2 = sum == 0.f ? -INFINITY : mref + log2f(sum);
    p.lse[orow] = p.lse_base2 ? lse2 : lse2 * kLn2;
  }
}

}  // namespace

cudaError_t launch_prefill_expanded(const ExpandedParams &p, const ExpandedMaps &m, cudaStream_t stream) {
  static SmemLimitOnce smem_limit;
  cudaError_t e = smem_limit.ensure(prefill_expanded_kernel, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * p.pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, prefill_expanded_kernel, p, m.q, m.k_nope, m.k_rope, m.v, m.va, m.vr);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(p.pairs, kExpRows / kMergeWarps);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, expanded_merge_kernel, p);
}

}  // namespace mla
