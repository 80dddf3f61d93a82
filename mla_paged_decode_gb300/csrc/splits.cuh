// Split bookkeeping shared by the decode kernels: request walk, neutral outputs
// for requests a partition does not touch, split tickets and the split merge.
#pragma once

#include "common.cuh"

namespace mla {

struct SplitInfo {
  int nsplits;   // CTAs whose tile range meets the request
  int c_first;   // first of them
  int slot;      // this CTA's slot for the request
};

template <bool SHORT = false>
__device__ __forceinline__ SplitInfo split_info(const CtaRange &r, int v, long long pv,
                                                int tiles) {
  SplitInfo s;
  s.c_first = SHORT ? sched_owner_short(pv, r.total, r.g_eff) : sched_owner(pv, r.total, r.g_eff);
  int c_last = SHORT ? sched_owner_short(pv + tiles - 1, r.total, r.g_eff)
                     : sched_owner(pv + tiles - 1, r.total, r.g_eff);
  s.nsplits = c_last - s.c_first + 1;
  s.slot = 2 * int(blockIdx.x) + (v != r.v_begin ? 1 : 0);
  return s;
}

// Slots (of 64 rows) that the pair kernel's pieces take, before the others:
// one per CTA of a pair for every (pair, block).
__host__ __device__ __forceinline__ int pair_slots(const DecodeParams &p) {
  return 2 * (p.pair_blocks + p.pairs);
}
// What a merge may follow of a record {first CTA or -1, pieces, slot of the first
// piece}.  Every call rewrites the records that its merge reads, but for a call
// whose bounded wait gave up: what is then in them may be anything, so that the
// checks take no sum or product of two words in 32 bits.
//
// A split of the decode kernel's schedule: piece 0 in slot z, piece k > 0 in slot
// 2 (x + k), all below 2 * grid.
__host__ __device__ __forceinline__ bool is_split(int4 info, int grid) {
  return info.y > 1 && info.x >= 0 && (long long)info.x + info.y <= grid && info.z >= 0 && info.z < 2 * grid;
}
// Pieces of shared pages or tails: y runs of `stride` slots from slot z * stride on.
__host__ __device__ __forceinline__ bool has_pieces(int4 info, int stride, int slots) {
  return info.y > 0 && info.z >= 0 && ((long long)info.z + info.y) * stride <= slots;
}

__device__ __forceinline__ float *slot_lse_ptr(const DecodeParams &p) {
  return reinterpret_cast<float *>(p.ws + p.wl.slot_lse);
}
__device__ __forceinline__ float *slot_out_ptr(const DecodeParams &p) {
  return reinterpret_cast<float *>(p.ws + p.wl.slot_out);
}
__device__ __forceinline__ int4 *info_ptr(const DecodeParams &p) {
  return reinterpret_cast<int4 *>(p.ws + p.wl.info);
}
// Records of the pair kernel's blocks: after those of the other kernel's tails.
__device__ __forceinline__ int4 *pair_info_ptr(const DecodeParams &p) {
  return info_ptr(p) + (p.pair_tails ? 0 : p.batch * p.head_groups);
}
__device__ __forceinline__ int *error_word(const DecodeParams &p) {
  return reinterpret_cast<int *>(p.ws);
}

__device__ __forceinline__ float lse_out(const DecodeParams &p, float lse2) {
  return p.lse_base2 ? lse2 : lse2 * kLn2;
}

// Flags what is out of range in the inputs of virtual request v of a view:
// a request's length, a group's pages, a request outside its group.
__device__ __forceinline__ void check_view(const DecodeParams &p, int v, int *err) {
  if (p.view == kViewShared) {
    if (v < p.prefix_blocks) return;
    v -= p.prefix_blocks;
    if (v < p.batch) {
      const int g = group_of_request(p, v);
      const bool in = p.group_starts[g] <= v && v < p.group_starts[g + 1];
      if (!in || p.shared_pages[g] < 0 || p.shared_pages[g] > p.max_pages) atomicOr(err, kErrBadLen);
    }
  }
  checked_len(p, v % p.batch, err);
}

// The neutral pair (0, -inf) for every virtual request with no owned token,
// and its split record {-1, 0, 0} (no splits), so that every record is
// rewritten by each call and the merge reads no lengths.  Virtual request v
// is handled by CTA v mod gridDim.x.  Block-wide.
template <int MULTI = 0>
__device__ inline void write_empty_requests(const DecodeParams &p) {
  const int V = p.batch * p.head_groups;
  int *err = error_word(p);
  for (int v = blockIdx.x; v < V; v += gridDim.x) {
    int b = vreq_row(p, v), g = vreq_group(p, v);  // b: output row
    if (request_len<MULTI>(p, v, threadIdx.x == 0 ? err : nullptr) != 0) continue;
    if (threadIdx.x == 0) info_ptr(p)[v] = make_int4(-1, 0, 0, 0);
    int h0 = g * p.heads_per_group;
    int hn = min(p.heads_per_group, p.heads - h0);
    uint4 *dst = reinterpret_cast<uint4 *>(p.out + (size_t(b) * p.heads + h0) * kDv);
    for (int i = threadIdx.x; i < hn * kDv / 8; i += blockDim.x) dst[i] = make_uint4(0, 0, 0, 0);
    for (int i = threadIdx.x; i < hn; i += blockDim.x)
      p.lse[size_t(b) * p.heads + h0 + i] = -INFINITY;
  }
}

// The same for views, by one warp of the CTA, with the checks of the inputs.
template <int MULTI>
__device__ inline void write_empty_views(const DecodeParams &p, const int2 *groups) {
  const int lane = threadIdx.x & 31, V = virtual_requests<MULTI>(p);
  for (int v = blockIdx.x; v < V; v += gridDim.x) {
    if (lane == 0) check_view(p, v, error_word(p));
    const ViewReq r = view_req<MULTI>(p, v, groups);
    if (r.tiles != 0) continue;
    if (lane == 0) info_ptr(p)[v] = make_int4(-1, 0, 0, 0);
    if (MULTI == 4) continue;  // the merge writes every row
    uint4 *dst = reinterpret_cast<uint4 *>(p.out + size_t(r.row0) * kDv);
    for (int i = lane; i < r.rows * kDv / 8; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
    for (int i = lane; i < r.rows; i += 32) p.lse[size_t(r.row0) + i] = -INFINITY;
  }
  __syncwarp();
}

// Called (by one thread) in each CTA that worked on request v: the CTA that
// holds the request's first tile records where its splits are, for the merge
// kernel.  Every request with owned tokens gets a fresh record each call
// (and every other one the empty record of write_empty_requests).
__device__ __forceinline__ void record_split(const DecodeParams &p, int v, const SplitInfo &si) {
  if (int(blockIdx.x) == si.c_first) info_ptr(p)[v] = make_int4(si.c_first, si.nsplits, si.slot, 0);
}

}  // namespace mla
