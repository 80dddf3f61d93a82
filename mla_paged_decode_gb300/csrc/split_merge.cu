// Merge of the requests that the stream-K schedule cut across CTAs (the
// split-KV reduce inside one partition).  Each split left a normalised fp32
// output and its base-2 LSE in a workspace slot, and the request's first CTA
// recorded {first CTA, number of splits, its slot}; split k > 0 lives in slot
// 2 (first + k).  The merge is the LSE-weighted combine of those splits.
//
// One CTA per (virtual request, 4 heads), a warp per head (few registers,
// so that the whole grid is resident in one wave): each lane owns 16
// of the 512 value dims (64 contiguous bytes of every split's row), issues
// the loads of the first splits before the weights are known, reduces the
// split LSEs with shuffles (max, then the sum of 2^(lse_k - max)), and
// accumulates the remaining splits 2 at a time.
#include "common.cuh"
#include "splits.cuh"

namespace mla {

constexpr int kMergeWarps = 4;  // heads per CTA
constexpr int kMergeBatch = 2;  // splits whose loads are in flight together

// The base-2 LSE of a merged row whose weights sum up to `sum`: -inf only for a row
// that saw no token.  A NaN partial (its query held a NaN or an Inf) makes the sum
// NaN and stays NaN, as in a row that one CTA holds whole: -inf would mark the row
// as empty, and a later merge would drop it.
__device__ __forceinline__ float merged_lse2(float mref, float sum) {
  return sum == 0.f ? -INFINITY : mref + log2f(sum);
}

// One warp merges row hl of request v, which the schedule split into
// info.y >= 2 pieces (info = the record its first CTA left): the
// LSE-weighted combine of the splits' normalised fp32 partials.  Returns this
// lane's 16 output dims as bf16 pairs and the row's base-2 LSE (-inf for a
// row that no split saw).
__device__ __forceinline__ void merge_split_row(const DecodeParams &p, int4 info, int hl,
                                                uint32_t (&pk)[8], float *lse2) {
  const int lane = threadIdx.x & 31;
  const int ns = info.y;
  const float *sl = slot_lse_ptr(p);
  const float *so = slot_out_ptr(p);
  auto slot_of_split = [&](int k) { return k == 0 ? info.z : 2 * (info.x + k); };
  auto part = [&](int k, int i) {  // float4 i (0..3) of this lane's 16 dims in split k
    return reinterpret_cast<const float4 *>(so + (size_t(slot_of_split(k)) * kSlotHeads + hl) * kDv)
        [4 * lane + i];
  };
  auto lse_of = [&](int k) { return sl[slot_of_split(k) * kSlotHeads + hl]; };

  float4 x[kMergeBatch][4];
#pragma unroll
  for (int u = 0; u < kMergeBatch; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) x[u][i] = u < ns ? part(u, i) : make_float4(0.f, 0.f, 0.f, 0.f);

  float mx = -INFINITY;
  for (int k = lane; k < ns; k += 32) mx = fmaxf(mx, lse_of(k));
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  // a query row that sees no token in any split (several query tokens per
  // request) has mx = -inf: every weight is then 0 and the row the neutral pair
  const float mref = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f;
  for (int k = lane; k < ns; k += 32) sum += exp2f(lse_of(k) - mref);
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);

  float4 acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < ns; k0 += kMergeBatch) {
    if (k0 > 0) {
#pragma unroll
      for (int u = 0; u < kMergeBatch; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[u][i] = k0 + u < ns ? part(k0 + u, i) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      const float w = k0 + u < ns ? exp2f(lse_of(k0 + u) - mref) : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i].x += w * x[u][i].x; acc[i].y += w * x[u][i].y;
        acc[i].z += w * x[u][i].z; acc[i].w += w * x[u][i].w;
      }
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(acc[i].x * inv, acc[i].y * inv);
    __nv_bfloat162 hi = __floats2bfloat162_rn(acc[i].z * inv, acc[i].w * inv);
    pk[2 * i] = *reinterpret_cast<uint32_t *>(&lo);
    pk[2 * i + 1] = *reinterpret_cast<uint32_t *>(&hi);
  }
  *lse2 = merged_lse2(mref, sum);
}

__device__ __forceinline__ void store_row(__nv_bfloat16 *row, const uint32_t (&pk)[8]) {
  uint4 *dst = reinterpret_cast<uint4 *>(row + 16 * (threadIdx.x & 31));
  dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
  dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
}

__global__ void __launch_bounds__(kMergeWarps * 32, 7) split_merge_kernel(DecodeParams p, int grid) {
  // launched as a programmatic dependent of the decode kernel: wait until its
  // grid has completed and its writes are visible
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int v = blockIdx.x;
  const int b = vreq_row(p, v), g = vreq_group(p, v);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hl = blockIdx.y * kMergeWarps + warp;  // head within the group
  const int group_heads = min(p.heads_per_group, p.heads - g * p.heads_per_group);
  if (hl >= group_heads) return;
  const int4 info = info_ptr(p)[v];
  if (!is_split(info, grid)) return;
  uint32_t pk[8];
  float lse2;
  merge_split_row(p, info, hl, pk, &lse2);
  const size_t row = size_t(b) * p.heads + size_t(g) * p.heads_per_group + hl;
  store_row(p.out + row * kDv, pk);
  if (lane == 0) p.lse[row] = lse_out(p, lse2);
}

// All partitions in one call (the decode ran them in one launch): one CTA
// per (request, row), warp q for partition q.  Warp q completes partition
// q's row -- the split merge when the decode's schedule cut that partition
// of the request across CTAs, else it reads back what the decode wrote --
// and leaves the bf16 row and its base-2 LSE in shared memory; then the CTA
// merges the P partitions with the LSE rule into comb_out / comb_lse: the
// LSE combine (the rank merge of the pages' DCP) fused into the split merge.
constexpr int kDcpMaxParts = 8;

__global__ void __launch_bounds__(kDcpMaxParts * 32) dcp_merge_combine_kernel(DecodeParams p,
                                                                              int grid) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ alignas(16) uint32_t s_val[kDcpMaxParts][kDv / 2];  // bf16 pairs
  __shared__ float s_lse[kDcpMaxParts];
  const int P = p.num_parts, rows = p.heads;
  const int b = blockIdx.x / rows, r = blockIdx.x - b * rows;
  const int g = r / p.heads_per_group, hl = r - g * p.heads_per_group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  {
    const int bv = warp * p.req_batch + b;  // partition `warp` of request b
    const int v = vreq_index(p, bv, g);
    const size_t prow = size_t(bv) * rows + r;
    uint32_t pk[8];
    float l;  // the partition's lse as returned (in the output base)
    const int4 info = info_ptr(p)[v];
    if (is_split(info, grid)) {
      float lse2;
      merge_split_row(p, info, hl, pk, &lse2);
      store_row(p.out + prow * kDv, pk);
      l = lse_out(p, lse2);
      if (lane == 0) p.lse[prow] = l;
    } else {  // written by the decode (the neutral pair if it owned nothing)
      const uint4 *src = reinterpret_cast<const uint4 *>(p.out + prow * kDv + 16 * lane);
      const uint4 a = src[0], c = src[1];
      pk[0] = a.x; pk[1] = a.y; pk[2] = a.z; pk[3] = a.w;
      pk[4] = c.x; pk[5] = c.y; pk[6] = c.z; pk[7] = c.w;
      l = p.lse[prow];
    }
    uint4 *dst = reinterpret_cast<uint4 *>(&s_val[warp][8 * lane]);
    dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
    if (lane == 0) s_lse[warp] = l;
  }
  __syncthreads();
  // The combine of the returned partials and lses, with the arithmetic of
  // lse_combine_kernel (same expressions, same shuffle tree for the sum), so
  // that the result equals mla_lse_combine's bit for bit.
  const float to2 = p.lse_base2 ? 1.f : kLog2e;
  float mx = -INFINITY;
  for (int q = 0; q < P; ++q) mx = max_nan(mx, s_lse[q] * to2);
  const size_t orow = size_t(b) * rows + r;
  uint4 *dst = reinterpret_cast<uint4 *>(p.comb_out + orow * kDv);
  constexpr int kChunks = kDv / 8;  // 16-byte chunks of a row
  if (mx == -INFINITY) {  // no partition owned a token of this row: the neutral pair
    for (int c = threadIdx.x; c < kChunks; c += blockDim.x) dst[c] = make_uint4(0, 0, 0, 0);
    if (p.comb_lse && threadIdx.x == 0) p.comb_lse[orow] = -INFINITY;
    return;
  }
  float w[kDcpMaxParts];
#pragma unroll
  for (int q = 0; q < kDcpMaxParts; ++q) w[q] = q < P ? exp2f(s_lse[q] * to2 - mx) : 0.f;
  const int lane_q = threadIdx.x & 31;
  float sum = lane_q < P ? exp2f(s_lse[lane_q] * to2 - mx) : 0.f;
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float inv = 1.f / sum;
  for (int c = threadIdx.x; c < kChunks; c += blockDim.x) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < kDcpMaxParts; ++q) {
      if (w[q] == 0.f) continue;
      const uint4 u = reinterpret_cast<const uint4 *>(s_val[q])[c];
      const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] = fmaf(w[q], __uint_as_float(x[i] << 16), acc[2 * i]);
        acc[2 * i + 1] = fmaf(w[q], __uint_as_float(x[i] & 0xffff0000u), acc[2 * i + 1]);
      }
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 t2 = __floats2bfloat162_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
      o[i] = *reinterpret_cast<uint32_t *>(&t2);
    }
    dst[c] = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (p.comb_lse && threadIdx.x == 0) {
    const float l2 = mx + log2f(sum);
    p.comb_lse[orow] = p.lse_base2 ? l2 : l2 * kLn2;
  }
}

// Shared pages: a row's partials are those of its group's block over the
// shared pages and those of its request over its own; the result is the
// LSE-weighted combine of all of them, each lane of a warp four runs of four
// value dims.  Many rows: a warp per row.  Few rows (WIDE): the schedule
// spreads them over all SMs, a row may have over a hundred partials, and a CTA
// takes a row, each of its warps every fourth partial (64 rows over 8K shared
// tokens: 45 us a call with a warp per row).
template <bool WIDE>
__global__ void __launch_bounds__(kMergeWarps * 32, 7) shared_merge_kernel(DecodeParams p, int slots) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = WIDE ? blockIdx.x : blockIdx.x * kMergeWarps + warp;
  if (row >= p.batch * p.heads) return;
  const int k_first = WIDE ? warp : 0, k_step = WIDE ? kMergeWarps : 1;  // this warp's partials
  const int b = row / p.heads, r = row - b * p.heads;
  const int g = group_of_request(p, b);
  const int local = row - group_start(p, g) * p.heads;
  // slots of the two sets: first, stride, number; the row's place in them
  int first[2] = {0, 0}, num[2] = {0, 0}, hl[2] = {local & 63, r & 63};
  const int stride[2] = {p.pair_blocks ? 2 : 1, p.pair_tails ? 2 : 1};  // a pair's piece has a slot per CTA
  if (local >= 0) {
    const int blocks = p.pair_blocks ? p.pair_blocks - p.pair_tails : p.prefix_blocks;
    const int v = p.pair_blocks ? block_base<128>(p, g) + (local >> 7) : block_base<64>(p, g) + (local >> 6);
    if (v < blocks) {
      const int4 i = p.pair_blocks ? pair_info_ptr(p)[v] : info_ptr(p)[v];
      if (has_pieces(i, stride[0], slots))
        first[0] = i.z * stride[0] + ((local >> 6) & (stride[0] - 1)), num[0] = i.y;
    }
  }
  {
    const int4 i = p.pair_tails ? pair_info_ptr(p)[p.pair_blocks - p.pair_tails + (r >> 7) * p.batch + b]
                                : info_ptr(p)[p.prefix_blocks + (r >> 6) * p.batch + b];
    if (has_pieces(i, stride[1], slots))
      first[1] = i.z * stride[1] + ((r >> 6) & (stride[1] - 1)), num[1] = i.y;
  }
  const int ns = num[0] + num[1];
  const float *sl = slot_lse_ptr(p);
  const float *so = slot_out_ptr(p);
  auto at = [&](int k) {
    const int s = k < num[0] ? first[0] + k * stride[0] : first[1] + (k - num[0]) * stride[1];
    return size_t(s) * kSlotHeads + hl[k < num[0] ? 0 : 1];
  };
  // the first partials' loads go out before the weights are known
  float4 x[kMergeBatch][4];
  auto load = [&](int k0) {
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      const float4 *src = reinterpret_cast<const float4 *>(so + at(min(k0 + u * k_step, ns - 1)) * kDv);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[u][i] = src[lane + 32 * i];
    }
  };
  if (ns > 0) load(k_first);
  float mx = -INFINITY;
  for (int k = lane; k < ns; k += 32) mx = fmaxf(mx, sl[at(k)]);
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float mref = mx == -INFINITY ? 0.f : mx;
  float4 acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int k0 = k_first; k0 < ns; k0 += kMergeBatch * k_step) {
    if (k0 > k_first) load(k0);
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      const int k = k0 + u * k_step;
      const float w = k < ns ? exp2f(sl[at(k)] - mref) : 0.f;
      sum += w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i].x += w * x[u][i].x; acc[i].y += w * x[u][i].y;
        acc[i].z += w * x[u][i].z; acc[i].w += w * x[u][i].w;
      }
    }
  }
  if constexpr (WIDE) {  // the warps' sums, in the order of the warps
    __shared__ float4 s_acc[kMergeWarps][4][32];
    __shared__ float s_sum[kMergeWarps];
#pragma unroll
    for (int i = 0; i < 4; ++i) s_acc[warp][i][lane] = acc[i];
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < kMergeWarps; ++w) {
      sum += s_sum[w];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 o = s_acc[w][i][lane];
        acc[i].x += o.x; acc[i].y += o.y; acc[i].z += o.z; acc[i].w += o.w;
      }
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  uint2 *dst = reinterpret_cast<uint2 *>(p.out + size_t(row) * kDv);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(acc[i].x * inv, acc[i].y * inv);
    __nv_bfloat162 hi = __floats2bfloat162_rn(acc[i].z * inv, acc[i].w * inv);
    dst[lane + 32 * i] = make_uint2(*reinterpret_cast<uint32_t *>(&lo), *reinterpret_cast<uint32_t *>(&hi));
  }
  if (lane == 0) p.lse[row] = lse_out(p, merged_lse2(mref, sum));
}

// Chunks: the blocks of 128 rows that the pair kernel's schedule cut.  Pair c's record
// is that of the block it begins and others go on with: {pieces, first row, rows, place
// of its piece in its two slots}; half h of the block lies in the slots of "CTA"
// h * pairs + c.  At most a block a pair is cut, so the grid is one column of warps per
// pair, however many blocks there are.
__global__ void __launch_bounds__(kMergeWarps * 32, 7) chunk_merge_kernel(DecodeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  const int r = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);  // row within the block
  const int4 rec = info_ptr(p)[c];
  if (rec.x < 2 || rec.x > p.pairs - c || rec.z > 128 || r >= rec.z || rec.y < 0 ||
      (long long)rec.y + rec.z > (long long)p.chunk_tokens * p.q_heads)
    return;
  const int first = (r >> 6) * p.pairs + c;
  uint32_t pk[8];
  float lse2;
  merge_split_row(p, make_int4(first, rec.x, 2 * first + (rec.w & 1), 0), r & 63, pk, &lse2);
  const size_t row = size_t(rec.y) + r;
  store_row(p.out + row * kDv, pk);
  if (lane == 0) p.lse[row] = lse_out(p, lse2);
}

cudaError_t launch_chunk_merge(const DecodeParams &p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.pairs, 128 / kMergeWarps);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_merge_kernel, p);
}

cudaError_t launch_shared_merge(const DecodeParams &p, int grid, cudaStream_t stream) {
  const int rows = p.batch * p.heads;
  const bool wide = rows <= 7 * grid;  // a CTA per row still fits the device in one wave
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(wide ? rows : (rows + kMergeWarps - 1) / kMergeWarps);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int slots = pair_slots(p) + (p.pair_tails ? 0 : p.batch * p.head_groups + p.prefix_blocks + grid);
  return wide ? cudaLaunchKernelEx(&cfg, shared_merge_kernel<true>, p, slots)
              : cudaLaunchKernelEx(&cfg, shared_merge_kernel<false>, p, slots);
}

cudaError_t launch_split_merge(const DecodeParams &p, int grid, cudaStream_t stream) {
  const int V = p.batch * p.head_groups;
  if (V == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(V, (p.heads_per_group + kMergeWarps - 1) / kMergeWarps);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, split_merge_kernel, p, grid);
}

// The fused-mode merge: split merge and LSE combine in one launch
// (num_parts <= 8), a programmatic dependent of the decode kernel.
cudaError_t launch_dcp_merge_combine(const DecodeParams &p, int grid, cudaStream_t stream) {
  const long long ctas = (long long)p.req_batch * p.heads;
  if (ctas == 0) return cudaSuccess;
  if (p.num_parts < 1 || p.num_parts > kDcpMaxParts || ctas > 0x7fffffffLL)
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(32 * p.num_parts);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, dcp_merge_combine_kernel, p, grid);
}

}  // namespace mla
