// Chunks of rows between contiguous buffers and the paged latent cache: a ragged
// batch of new tokens written into it (quantised to e4m3 where the cache is), and
// cached rows read back as bf16.
//
//   append: row r of the chunk, token t = positions[b] + r - starts[b] of its request
//           b, goes to cache row 64 table[b][t / 64] + t mod 64 as its bits, or as
//           e4m3(fp32(x) / scale), rounded to nearest even and saturated.
//   read:   the other way: the bits, or bf16(fp32(fp32(code) * scale)).
//
// Both move 1152 B (bf16) or 1152 + 576 B (e4m3) a row each way and compute next to
// nothing but the quotients of an e4m3 append: HBM bounds the others (65,536 bf16 rows
// written 25.5 us, 5,910 GB/s, read 26.3; 59,600 e4m3 rows read 19.8, 5,230 GB/s; 24,200
// rows into an e4m3 cache 13.7 us, 3,030 GB/s, all over buffers in turn).  A warp takes four rows, which are nine 16-byte (e4m3
// side: 8-byte) chunks a lane, all in flight at once; eight lanes look each row's place
// up, for an append while the loads are on their way.
#include "common.cuh"

namespace mla {
namespace {

constexpr int kWarps = 4;
constexpr int kRowsPerWarp = 4;
constexpr int kLoads = kRowsPerWarp * kDqk / 8 / 32;  // chunks of 8 values a lane
static_assert(kLoads * 32 * 8 == kRowsPerWarp * kDqk, "whole rows");
constexpr int kErrChunkBadPage = 1, kErrChunkBadStart = 2;

struct ChunkRows {
  const int32_t *block_table;  // [batch, max_pages]
  const int32_t *starts;       // [batch + 1]
  const int32_t *positions;    // [batch]
  int batch, rows, max_pages, num_pages, part_id, num_parts;
  long long stride;            // values between rows of the contiguous buffer
  float scale, inverse;        // e4m3: 1 / scale, or 0 to divide
  int32_t *error_word;
  int row_ctas;                // of the grid; with an error word others check the starts
};

constexpr long long kNoRow = -1, kBadRow = -2;

// The cache row of row r0 + lane / 8, eight lanes a row: kNoRow where the row is nobody's
// (outside all requests, of a request with a negative position, or another partition's),
// kBadRow where the table has no page for it.  The request is the last that starts at or
// before the row, found in eighths: two rounds of loads for 64 requests, where halving
// takes six one after the other.
__device__ __forceinline__ long long cache_row(const ChunkRows &c, int r0) {
  const int lane = threadIdx.x & 31, group = lane >> 3, k = lane & 7, r = r0 + group;
  bool in = r < c.rows && r >= c.starts[0] && r < c.starts[c.batch];
  int lo = 0, n = c.batch;  // it is one of n from lo on
  while (__any_sync(0xffffffffu, n > 1)) {
    const int step = (n + 7) / 8, at = k * step;
    const bool before = k == 0 || (at < n && c.starts[lo + at] <= r);
    const int found = __popc((__ballot_sync(0xffffffffu, before) >> (8 * group)) & 0xffu) - 1;
    lo += found * step;
    n = min(step, n - found * step);
  }
  const int first = c.positions[lo], i = r - c.starts[lo];
  in = in && first >= 0 && i >= 0;
  const long long t = (long long)first + i;
  if (!in || (c.num_parts > 1 && t % c.num_parts != c.part_id)) return kNoRow;
  const long long lp = t / kPage;
  const int pg = lp < c.max_pages ? c.block_table[(long long)lo * c.max_pages + lp] : -1;
  if (pg < 0 || pg >= c.num_pages) return kBadRow;
  return (long long)pg * kPage + t % kPage;
}

// The fp32 quotient x / scale, rounded to nearest, from the inverse of the scale rounded to
// nearest: the product is within a unit of its last place, and one step with the exact
// remainder rounds it right (Markstein, 1990).  Exact as long as nothing under- or
// overflows: |x| in [2^-60, 2^60) and the scale in [2^-30, 2^30].  Zeros keep their sign.
// (65,536 rows: 23.9 us; with a division each 27.3, bound by the instructions.)
__device__ __forceinline__ float quotient(float x, float scale, float inverse, bool *plain) {
  const uint32_t bits = __float_as_uint(x) & 0x7fffffffu;
  *plain = *plain && (bits == 0 || bits - 0x21800000u < 0x5d800000u - 0x21800000u);
  const float q = x * inverse;
  const float y = fmaf(fmaf(-q, scale, x), inverse, q);
  return bits == 0 ? x : y;
}

// Eight bf16 values as e4m3 codes of x / scale.
__device__ __forceinline__ uint2 quantise(uint4 v, float scale, float inverse) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  bool plain = inverse != 0.f;
  uint32_t o[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float lo = quotient(__uint_as_float(w[k] << 16), scale, inverse, &plain);
    const float hi = quotient(__uint_as_float(w[k] & 0xffff0000u), scale, inverse, &plain);
    o[k >> 1] |= uint32_t(float2_to_e4m3x2(lo, hi)) << (16 * (k & 1));
  }
  if (!plain) {  // something tiny, huge or not finite among the eight
    o[0] = o[1] = 0;
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      const uint32_t x = k == 0 ? w[0] : k == 1 ? w[1] : k == 2 ? w[2] : w[3];
      const uint32_t two = float2_to_e4m3x2(__fdiv_rn(__uint_as_float(x << 16), scale),
                                            __fdiv_rn(__uint_as_float(x & 0xffff0000u), scale));
      if (k < 2) o[0] |= two << (16 * k);
      else o[1] |= two << (16 * (k - 2));
    }
  }
  return make_uint2(o[0], o[1]);
}

__device__ __forceinline__ uint4 dequantise(uint2 v, float scale) {
  const uint32_t w[2] = {v.x, v.y};
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = e4m3x2_to_float2(uint16_t(w[k >> 1] >> (16 * (k & 1))));
    __nv_bfloat162 h = __floats2bfloat162_rn(f.x * scale, f.y * scale);
    o[k] = *reinterpret_cast<uint32_t *>(&h);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// A load that stays where it is written, before the look-ups.
__device__ __forceinline__ uint4 load_now(const void *p) {
  uint4 v;
  asm volatile("ld.global.cs.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Starts that fall or leave the buffer make rows nobody's that should be somebody's.  CTAs
// behind the rows' own look for them, a thread a request: a read of 59,600 rows takes 14.6
// us with them and without; with the test in warps of the rows' CTAs 15.9.
__device__ __forceinline__ void check_starts(const ChunkRows &c) {
  const long long b = ((long long)blockIdx.x - c.row_ctas) * (kWarps * 32) + threadIdx.x;
  if (b >= c.batch) return;
  const int s0 = c.starts[b], s1 = c.starts[b + 1];
  if (s0 < 0 || s1 < s0 || s1 > c.rows) atomicOr(c.error_word, kErrChunkBadStart);
}

// READ: cache -> buffer, else buffer -> cache.
template <bool READ, bool F8>
__global__ void __launch_bounds__(kWarps * 32) kv_chunk_kernel(const __grid_constant__ ChunkRows c,
                                                               unsigned char *cache, __nv_bfloat16 *buffer) {
  const int warp = int(blockIdx.x) * kWarps + int(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (blockIdx.x >= unsigned(c.row_ctas)) {
    check_starts(c);
    return;
  }
  if (warp >= (c.rows + kRowsPerWarp - 1) / kRowsPerWarp) return;
  const int r0 = warp * kRowsPerWarp;
  constexpr int kChunks = kDqk / 8;           // of a row
  constexpr int kBytes = F8 ? 8 : 16;         // of a chunk in the cache
  uint4 v[kLoads];
  if constexpr (!READ) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int r = r0 + (lane + 32 * u) / kChunks, k = (lane + 32 * u) % kChunks;
      v[u] = load_now(reinterpret_cast<const uint4 *>(buffer + min(r, c.rows - 1) * c.stride) + k);
    }
  }
  const long long mine = cache_row(c, r0);
  if (mine == kBadRow && c.error_word && (lane & 7) == 0) atomicOr(c.error_word, kErrChunkBadPage);
  auto place = [&](int u) {  // chunk u of this lane in the cache, or a negative number
    const long long row = __shfl_sync(0xffffffffu, mine, (lane + 32 * u) / kChunks * 8);
    return row < 0 ? row : row * (kDqk * kBytes / 8) + (lane + 32 * u) % kChunks * kBytes;
  };
  if constexpr (READ) {
    uint2 w[kLoads];
    long long at[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      at[u] = place(u);
      v[u] = make_uint4(0, 0, 0, 0);
      w[u] = make_uint2(0, 0);
      if (at[u] < 0) continue;
      if constexpr (F8) w[u] = __ldcs(reinterpret_cast<const uint2 *>(cache + at[u]));
      else v[u] = __ldcs(reinterpret_cast<const uint4 *>(cache + at[u]));
    }
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      if (at[u] == kNoRow) continue;
      if constexpr (F8) v[u] = dequantise(w[u], c.scale);
      const int r = r0 + (lane + 32 * u) / kChunks, k = (lane + 32 * u) % kChunks;
      reinterpret_cast<uint4 *>(buffer + r * c.stride)[k] = v[u];
    }
  } else {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const long long at = place(u);
      if (at < 0) continue;
      if constexpr (F8) *reinterpret_cast<uint2 *>(cache + at) = quantise(v[u], c.scale, c.inverse);
      else *reinterpret_cast<uint4 *>(cache + at) = v[u];
    }
  }
}

}  // namespace

cudaError_t launch_kv_chunk(bool read, void *cache, void *buffer, long long stride, const int32_t *block_table,
                            const int32_t *starts, const int32_t *positions, int rows, int batch, int part_id,
                            int num_parts, int num_pages, int max_pages, int e4m3, float kv_scale,
                            int32_t *error_word, cudaStream_t stream) {
  const float inverse = kv_scale >= 0x1p-30f && kv_scale <= 0x1p30f ? 1.f / kv_scale : 0.f;
  const int per = kWarps * kRowsPerWarp, row_ctas = int((rows + (long long)per - 1) / per);
  const ChunkRows c{block_table, starts,    positions, batch,    rows,    max_pages,  num_pages,
                    part_id,     num_parts, stride,    kv_scale, inverse, error_word, row_ctas};
  const unsigned grid = row_ctas + (error_word ? unsigned((batch + kWarps * 32ll - 1) / (kWarps * 32)) : 0u);
  auto *kernel = read ? (e4m3 ? kv_chunk_kernel<true, true> : kv_chunk_kernel<true, false>)
                      : (e4m3 ? kv_chunk_kernel<false, true> : kv_chunk_kernel<false, false>);
  kernel<<<grid, kWarps * 32, 0, stream>>>(c, static_cast<unsigned char *>(cache),
                                           static_cast<__nv_bfloat16 *>(buffer));
  return cudaGetLastError();
}

}  // namespace mla
