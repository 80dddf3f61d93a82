// What the expanded prefill kernel and its host side share.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace mla {

constexpr int kNope = 128, kRope = 64, kDvx = 128;  // a head's score dims (own, shared) and value dims
constexpr int kExpRows = 512;                       // query tokens of a block

// Workspace: [0, 256) error word; a record a pair; two slots of 512 rows a pair (fp32
// LSEs, fp32 normalised outputs).
struct ExpandedLayout {
  size_t rec, lse, out, total;
};
__host__ __device__ constexpr ExpandedLayout expanded_layout(int pairs) {
  const size_t rec = 256, lse = align256(rec + 16 * size_t(pairs));
  const size_t out = align256(lse + sizeof(float) * 2 * pairs * kExpRows);
  return ExpandedLayout{rec, lse, out, align256(out + sizeof(float) * 2 * pairs * kExpRows * size_t(kDvx))};
}

struct ExpandedParams {
  __nv_bfloat16 *out;       // [q_tokens, heads, 128]
  float *lse;               // [q_tokens, heads]
  unsigned char *ws;
  const int32_t *q_starts;  // [batch + 1]
  const int32_t *k_starts;  // [batch + 1]
  int batch, heads, q_tokens, k_tokens, causal;
  int blocks;               // ids of 512-token blocks: q_tokens / 512 rounded down + batch
  int pairs;
  float score_scale_log2;
  int lse_base2;
};

struct ExpandedMaps {
  CUtensorMap q;       // 64 dims x 128 tokens of a head
  CUtensorMap k_nope;  // 64 dims x 64 tokens of a head
  CUtensorMap k_rope;  // 64 dims x 64 tokens
  CUtensorMap v;       // 64 dims x 128 tokens of a head
  CUtensorMap va;      // ... x 8
  CUtensorMap vr;      // ... x 1
};

cudaError_t launch_prefill_expanded(const ExpandedParams &p, const ExpandedMaps &m, cudaStream_t stream);

}  // namespace mla
