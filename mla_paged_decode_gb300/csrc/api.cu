// Host side of the C ABI declared in include/mla_decode.h: argument checks,
// workspace sizing, per-device facts, and kernel dispatch.  Nothing here
// allocates device memory or synchronises the host (except the explicit
// mla_decode_check_workspace).
#include "mla_decode.h"

#include <cuda.h>

#include <cmath>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "pages.cuh"
#include "pair_maps.cuh"
#include "prefill_expanded.cuh"

namespace mla {
cudaError_t launch_decode_simt(const DecodeParams &p, int grid, cudaStream_t stream);
cudaError_t launch_dcp_metadata(const int32_t *seq_lens, const int32_t *req_pool_indices,
                                const int32_t *req_to_token, int batch, int r2t_rows,
                                int r2t_width, int extra, int part_id, int num_parts,
                                int32_t *global_lens, int32_t *local_lens, int32_t *table,
                                int max_pages, int32_t pad, int32_t *error_word,
                                cudaStream_t stream);
cudaError_t launch_kv_append(const void *kv_new, void *kv_pages, const int32_t *block_table,
                             const int32_t *positions, int batch, int part_id, int num_parts,
                             int num_pages, int max_pages, int e4m3, float kv_scale,
                             int32_t *error_word, cudaStream_t stream);
cudaError_t launch_kv_chunk(bool read, void *cache, void *buffer, long long stride, const int32_t *block_table,
                            const int32_t *starts, const int32_t *positions, int rows, int batch, int part_id,
                            int num_parts, int num_pages, int max_pages, int e4m3, float kv_scale,
                            int32_t *error_word, cudaStream_t stream);
cudaError_t launch_decode_tc(const DecodeParams &p, int npv, int q_rows, int groups_per_page,
                             const CUtensorMap &tm_q, const CUtensorMap &tm_kv,
                             const CUtensorMap &tm_kvg, const CUtensorMap &tm_kvb, int grid,
                             cudaStream_t stream);
cudaError_t launch_decode_pair(const DecodeParams &p, const CUtensorMap &tm_q, const PairMaps &m,
                               cudaStream_t stream);
cudaError_t launch_lse_combine(const void *partials, const float *lses, int num_parts, void *out,
                               float *out_lse, int rows, int dim, int base2, cudaStream_t stream);
int combine_max_parts();
cudaError_t launch_pages_copy(const void *src_pool, void *dst_pool, const int32_t *src, const int32_t *dst,
                              int n, int src_pages, int dst_pages, int row_bytes, int32_t *error_word,
                              cudaStream_t stream);
cudaError_t launch_pages_fork(const PagesTable &t, void *pool, int row_bytes, const int32_t *parents,
                              const int32_t *children, int n, const PagesWorkspace &ws, int32_t *error_word,
                              cudaStream_t stream);
cudaError_t launch_pages_alloc(const PagesTable &t, const int32_t *new_lens, const PagesWorkspace &ws,
                               int32_t *error_word, cudaStream_t stream);
cudaError_t launch_pages_free(const PagesTable &t, const int32_t *new_lens, int window, int sinks,
                              int32_t *error_word, cudaStream_t stream);
cudaError_t launch_pages_compact(const PagesTable &t, void *pool, int row_bytes, int32_t *remap, int grid,
                                 const PagesWorkspace &ws, int32_t *error_word, cudaStream_t stream);
}  // namespace mla

namespace {

thread_local char g_cuda_error[256] = "";

int cuda_fail(cudaError_t e) {
  std::snprintf(g_cuda_error, sizeof(g_cuda_error), "%s: %s", cudaGetErrorName(e),
                cudaGetErrorString(e));
  return MLA_ERR_CUDA;
}

struct DeviceFacts {
  int sms = 0;
  int major = 0, minor = 0;
};

constexpr int kMaxDevices = 64;
DeviceFacts g_dev[kMaxDevices];
std::mutex g_dev_mu;

// Facts of the current device; status in *st.
DeviceFacts current_device(int *st, int *dev_out = nullptr) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) {
    *st = cuda_fail(e);
    return {};
  }
  if (dev_out) *dev_out = dev;
  if (dev < 0 || dev >= kMaxDevices) {
    *st = MLA_ERR_DEVICE;
    return {};
  }
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DeviceFacts &f = g_dev[dev];
  if (f.sms == 0) {
    int sms = 0, mj = 0, mn = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&mj, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&mn, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess) {
      *st = cuda_fail(e);
      return {};
    }
    f.sms = sms;
    f.major = mj;
    f.minor = mn;
  }
  *st = mla_arch_supported(f.major, f.minor) ? MLA_OK : MLA_ERR_DEVICE;
  return f;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// cuTensorMapEncodeTiled through the runtime's driver entry point (the
// library does not link the driver library directly).
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static EncodeTiled fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(f);
  });
  return fn;
}

int tensor_map_fail(const char *what, CUresult r) {
  std::snprintf(g_cuda_error, sizeof(g_cuda_error), "cuTensorMapEncodeTiled(%s) failed: %d", what,
                int(r));
  return MLA_ERR_CUDA;
}

constexpr int kTcHeadsPerGroup = 64;

// The tensor-core kernel reads exactly a partition's rows when they form whole
// 8-row groups of a page (P | 8), or through the strided gather below.
// Otherwise it gathers partition r mod g of g = gcd(P, 8) (g divides
// a page's 8 atoms) and, when g < P, drops the tokens other partitions own:
// it reads P / g times the partition's own bytes at the tensor-core rate,
// which beats the CUDA-core kernel while P / g stays small.
int gather_parts(int num_parts) {
  int g = 8, a = num_parts;
  while (a) { const int t = g % a; g = a; a = t; }
  return g;
}
constexpr int kMaxOwnerRatio = 16;  // P / gather_parts(P) served by the tensor cores

bool tensor_core_path(const mla_decode_desc *, int num_parts) {
  return num_parts >= 1 && num_parts / gather_parts(num_parts) <= kMaxOwnerRatio;
}

// P in {3, 5, 6, 7}: the tensor-core kernel gathers exactly the partition's
// rows, with a TMA traversal stride of P rows (at most 8), `strided_apg(P)`
// atoms of 8 rows per page, for bf16 and e4m3 caches and any q_len.  Other P
// not dividing 8 take the owner mask.
bool strided_path(const mla_decode_desc *, int num_parts) {
  return num_parts > 1 && num_parts < 8 && 8 % num_parts != 0;
}
int strided_apg(int num_parts) {
  const int rows = (mla::kPage + num_parts - 1) / num_parts;  // a partition's rows of a page, at most
  return (rows + 7) / 8;
}

// all partitions in one decode launch: P divides 8 (no owner mask), or the
// strided gather
bool fused_path(const mla_decode_desc *d, int num_parts) {
  return num_parts >= 1 && (8 % num_parts == 0 || strided_path(d, num_parts));
}

// Q as [rows, 576] bf16, one 64-column swizzled box of q_rows rows.
int make_q_map(EncodeTiled enc, const void *q, cuuint64_t rows, int q_rows, CUtensorMap *tm_q) {
  cuuint64_t dims[2] = {cuuint64_t(mla::kDqk), rows};
  cuuint64_t strides[1] = {cuuint64_t(mla::kDqk) * 2};
  cuuint32_t box[2] = {64, cuuint32_t(q_rows)};
  cuuint32_t es[2] = {1, 1};
  CUresult r = enc(tm_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(q), dims, strides,
                   box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MLA_OK : tensor_map_fail("q", r);
}

// Q (make_q_map);
// partition rows of a bf16 cache as a 5-D view (64 dims, 8 rows of stride P,
// 9 blocks of 64 dims, groups of 8 rows, partitions), one box = one page's
// owned rows; of an e4m3 cache as a 3-D view (576 bytes, rows of stride P,
// partitions), one swizzled box = 128 dims of one page's 64/P owned rows,
// with an unswizzled view of whole 576-byte rows for the L2 prefetch.  The
// strided gather's maps take an atom's rows through a traversal stride P.
// For one partition (`part_id`) the base is offset to its
// first row and the partition dimension is left off (4-D / 2-D maps, the
// faster boxes); for all P partitions (`all_parts`) it is added, with a stride
// of one row (5-D / 3-D maps, coordinate r).
int make_tensor_maps(const void *q, const void *kv, const mla_decode_desc *d, int q_rows, int part_id,
                     int num_parts, bool all_parts, bool strided, CUtensorMap *tm_q,
                     CUtensorMap *tm_kv, CUtensorMap *tm_kvg, CUtensorMap *tm_kvb) {
  EncodeTiled enc = encode_tiled();
  if (!enc) {
    std::snprintf(g_cuda_error, sizeof(g_cuda_error), "cuTensorMapEncodeTiled unavailable");
    return MLA_ERR_CUDA;
  }
  const cuuint64_t row = cuuint64_t(mla::kDqk) * 2;
  {
    const int st = make_q_map(enc, q, cuuint64_t(d->batch) * d->q_len * d->num_heads, q_rows, tm_q);
    if (st != MLA_OK) return st;
  }
  if (d->kv_dtype == MLA_KV_E4M3 && strided) {
    // (144 words of 4 fp8 values, 64 page rows, pages): one box is one atom,
    // raw rows c, c + P, ..., c + 7P of a page (traversal stride P), landing
    // as 8 consecutive 576-byte rows; rows past the page read as zeros
    const cuuint32_t P = cuuint32_t(num_parts);
    const cuuint64_t row8 = cuuint64_t(mla::kDqk);
    cuuint64_t dims[3] = {row8 / 4, cuuint64_t(mla::kPage), cuuint64_t(d->num_pages)};
    cuuint64_t strides[2] = {row8, cuuint64_t(mla::kPage) * row8};
    cuuint32_t box[3] = {cuuint32_t(row8 / 4), 8 * P, 1};
    cuuint32_t es[3] = {1, P, 1};
    CUresult r = enc(tm_kv, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void *>(kv), dims,
                     strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return tensor_map_fail("kv e4m3 strided", r);
    // block 4 of the kernel's loads (the box above serves the L2 prefetch):
    // (576 bytes, 64 page rows, pages), a box of dims 512..575 of an atom's
    // rows c, c + P, ..., c + 7P with the 64-byte swizzle
    cuuint64_t fdims[3] = {row8, cuuint64_t(mla::kPage), cuuint64_t(d->num_pages)};
    cuuint64_t fstrides[2] = {row8, cuuint64_t(mla::kPage) * row8};
    cuuint32_t fbox[3] = {64, 8 * P, 1};
    r = enc(tm_kvg, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(kv), fdims, fstrides, fbox, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return tensor_map_fail("kv e4m3 strided blocks", r);
    // blocks 0..3 of an atom in one box, landing [block][8 rows][128 B]:
    // (128 bytes, 64 page rows, 4 blocks, pages)
    cuuint64_t gdims[4] = {128, cuuint64_t(mla::kPage), 4, cuuint64_t(d->num_pages)};
    cuuint64_t gstrides[3] = {row8, 128, cuuint64_t(mla::kPage) * row8};
    cuuint32_t gbox[4] = {128, 8 * P, 4, 1};
    cuuint32_t ges[4] = {1, P, 1, 1};
    r = enc(tm_kvb, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(kv), gdims, gstrides, gbox, ges,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return tensor_map_fail("kv e4m3 strided grouped blocks", r);
  } else if (d->kv_dtype == MLA_KV_E4M3) {
    const cuuint64_t P = cuuint64_t(num_parts);
    const cuuint32_t R = cuuint32_t(mla::kPage / num_parts);
    const cuuint64_t row8 = cuuint64_t(mla::kDqk);
    const char *base = static_cast<const char *>(kv) + (all_parts ? 0 : size_t(part_id) * row8);
    cuuint64_t dims[3] = {row8 / 4, cuuint64_t(d->num_pages) * R, P};
    cuuint64_t strides[2] = {P * row8, row8};
    cuuint32_t box[3] = {cuuint32_t(row8 / 4), R, 1};
    cuuint32_t es[3] = {1, 1, 1};
    CUresult r = enc(tm_kv, CU_TENSOR_MAP_DATA_TYPE_UINT32, all_parts ? 3 : 2,
                     const_cast<char *>(base), dims,
                     strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return tensor_map_fail("kv e4m3", r);
    // block 4 of the kernel's loads (the box above serves the L2 prefetch):
    // (576 bytes, owned rows, partitions), a box of dims 512..575 of a page's
    // 64/P owned rows with the 64-byte swizzle
    cuuint64_t fdims[3] = {row8, cuuint64_t(d->num_pages) * R, P};
    cuuint64_t fstrides[2] = {P * row8, row8};
    cuuint32_t fbox[3] = {64, R, 1};
    r = enc(tm_kvg, CU_TENSOR_MAP_DATA_TYPE_UINT8, all_parts ? 3 : 2, const_cast<char *>(base), fdims,
            fstrides, fbox, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return tensor_map_fail("kv e4m3 blocks", r);
    {
      // blocks 0..3 of a page's owned atoms in one box, landing
      // [atom][block][8 rows][128 B]: (128 bytes, 8 rows, 4 blocks, 8-row
      // atoms, partitions)
      const cuuint64_t G = 8 / P;
      cuuint64_t gdims[5] = {128, 8, 4, cuuint64_t(d->num_pages) * G, P};
      cuuint64_t gstrides[4] = {P * row8, 128, 8 * P * row8, row8};
      cuuint32_t gbox[5] = {128, 8, 4, cuuint32_t(G), 1};
      cuuint32_t ges[5] = {1, 1, 1, 1, 1};
      r = enc(tm_kvb, CU_TENSOR_MAP_DATA_TYPE_UINT8, all_parts ? 5 : 4, const_cast<char *>(base), gdims,
              gstrides, gbox, ges, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
      if (r != CUDA_SUCCESS) return tensor_map_fail("kv e4m3 grouped blocks", r);
    }
  } else if (strided) {
    // (64 dims, 64 page rows, 9 blocks of 64 dims, pages): one box is one
    // atom, rows c, c + P, ..., c + 7P of a page (traversal stride P), which
    // lands as [9 blocks][8 rows][128 B]; rows past the page are out of
    // bounds and read as zeros.  The partition is in the row coordinate.
    const cuuint32_t P = cuuint32_t(num_parts);
    cuuint64_t dims[4] = {64, cuuint64_t(mla::kPage), cuuint64_t(mla::kDqk / 64),
                          cuuint64_t(d->num_pages)};
    cuuint64_t strides[3] = {row, 128, cuuint64_t(mla::kPage) * row};
    cuuint32_t box[4] = {64, 8 * P, cuuint32_t(mla::kDqk / 64), 1};
    cuuint32_t es[4] = {1, P, 1, 1};
    CUresult r = enc(tm_kv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(kv), dims,
                     strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return tensor_map_fail("kv strided", r);
    *tm_kvg = *tm_kv;  // unused: one column group
  } else {
    const cuuint64_t P = cuuint64_t(num_parts);
    const cuuint32_t G = cuuint32_t(8 / num_parts);
    const char *base = static_cast<const char *>(kv) + (all_parts ? 0 : size_t(part_id) * row);
    cuuint64_t dims[5] = {64, 8, cuuint64_t(mla::kDqk / 64), cuuint64_t(d->num_pages) * G, P};
    cuuint64_t strides[4] = {P * row, 128, 8 * P * row, row};
    cuuint32_t box[5] = {64, 8, cuuint32_t(mla::kDqk / 64), G, 1};
    cuuint32_t es[5] = {1, 1, 1, 1, 1};
    CUresult r = enc(tm_kv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, all_parts ? 5 : 4,
                     const_cast<char *>(base), dims,
                     strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return tensor_map_fail("kv", r);
    // one column group (3 of the 9 dim blocks) of a page's atoms: the
    // kernel's loads when a tile is one page (P = 1); the full-page box above
    // serves the L2 prefetch and the loads of P > 1
    box[2] = 3;
    r = enc(tm_kvg, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, all_parts ? 5 : 4, const_cast<char *>(base),
            dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return tensor_map_fail("kv column group", r);
  }
  if (d->kv_dtype != MLA_KV_E4M3) *tm_kvb = *tm_kv;  // unused: only e4m3 caches take grouped boxes
  return MLA_OK;
}

// The pair kernel's loads, on (128 bytes, 8 rows, dim blocks of 128 bytes, 8-row
// groups): one dim block of a page's 64 rows (K); the value dims of one CTA,
// four blocks of half a bf16 page or two of an e4m3 page (V).  The last 64 dims
// of an e4m3 page's rows come through tm_k4, 64 bytes a row.
int make_pair_maps(const void *kv, const mla_decode_desc *d, mla::PairMaps *m) {
  EncodeTiled enc = encode_tiled();
  if (!enc) {
    std::snprintf(g_cuda_error, sizeof(g_cuda_error), "cuTensorMapEncodeTiled unavailable");
    return MLA_ERR_CUDA;
  }
  const bool f8 = d->kv_dtype == MLA_KV_E4M3;
  const auto type = f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint32_t x = f8 ? 128 : 64;  // elements of a 128-byte row
  const cuuint64_t row = cuuint64_t(mla::kDqk) * (f8 ? 1 : 2);
  cuuint64_t dims[4] = {x, 8, cuuint64_t(f8 ? 4 : 9), cuuint64_t(d->num_pages) * 8};
  cuuint64_t strides[3] = {row, 128, 8 * row};
  cuuint32_t box_k[4] = {x, 8, 1, 8}, box_v[4] = {x, 8, f8 ? 2u : 4u, f8 ? 8u : 4u}, es[4] = {1, 1, 1, 1};
  cuuint32_t box_va[4] = {x, 8, f8 ? 2u : 4u, 1}, box_vr[4] = {x, 1, 1, 1};
  CUresult r = CUDA_SUCCESS;
  auto map = [&](CUtensorMap *tm, cuuint32_t *box) {
    if (r == CUDA_SUCCESS)
      r = enc(tm, type, 4, const_cast<void *>(kv), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  map(&m->k, box_k);
  map(&m->v, box_v);
  map(&m->va, box_va);
  map(&m->vr, box_vr);
  if (r != CUDA_SUCCESS) return tensor_map_fail("kv pair", r);
  m->k4 = m->k;
  if (f8) {
    cuuint64_t dims4[2] = {row, cuuint64_t(d->num_pages) * mla::kPage};
    cuuint64_t strides4[1] = {row};
    cuuint32_t box4[2] = {64, mla::kPage};
    r = enc(&m->k4, type, 2, const_cast<void *>(kv), dims4, strides4, box4, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return tensor_map_fail("kv pair rope", r);
  }
  return MLA_OK;
}

constexpr int kSimtHeadsPerGroup = 32;
// Query tokens per request: several (multi-token prediction / target verify)
// only on the tensor-core path; the CUDA-core kernel takes one.
constexpr int kMaxQLen = 16;

int check_desc(const mla_decode_desc *d) {
  if (!d) return MLA_ERR_NULL;
  if (d->batch < 0 || d->num_pages < 1 || d->max_pages_per_seq < 1) return MLA_ERR_SHAPE;
  if (d->q_len < 1 || d->q_len > kMaxQLen) return MLA_ERR_SHAPE;
  if (d->head_dim_qk != mla::kDqk || d->head_dim_v != mla::kDv) return MLA_ERR_SHAPE;
  if (d->page_size != mla::kPage) return MLA_ERR_SHAPE;
  if (d->num_heads < 1 || d->num_heads > 128) return MLA_ERR_SHAPE;
  if (d->kv_dtype != MLA_KV_BF16 && d->kv_dtype != MLA_KV_E4M3) return MLA_ERR_ARG;
  if (d->kv_dtype == MLA_KV_E4M3 && !(std::isfinite(d->kv_scale) && d->kv_scale > 0.f))
    return MLA_ERR_ARG;
  return MLA_OK;
}

// The fields of a decode descriptor that describe the cache itself.
int check_cache_desc(const mla_decode_desc *d) {
  if (!d) return MLA_ERR_NULL;
  if (d->batch < 0 || d->num_pages < 1 || d->max_pages_per_seq < 1) return MLA_ERR_SHAPE;
  if (d->head_dim_qk != mla::kDqk || d->page_size != mla::kPage) return MLA_ERR_SHAPE;
  if (d->kv_dtype != MLA_KV_BF16 && d->kv_dtype != MLA_KV_E4M3) return MLA_ERR_ARG;
  if (d->kv_dtype == MLA_KV_E4M3 && !(std::isfinite(d->kv_scale) && d->kv_scale > 0.f))
    return MLA_ERR_ARG;
  return MLA_OK;
}

int check_pages_desc(const mla_pages_desc *d) {
  if (!d) return MLA_ERR_NULL;
  if (d->num_requests < 0 || d->max_pages_per_seq < 1 || d->num_pages < 1) return MLA_ERR_SHAPE;
  if (d->head_dim_qk != mla::kDqk || d->page_size != mla::kPage) return MLA_ERR_SHAPE;
  if (d->kv_dtype != MLA_KV_BF16 && d->kv_dtype != MLA_KV_E4M3) return MLA_ERR_ARG;
  return MLA_OK;
}

int pages_row_bytes(const mla_pages_desc *d) { return mla::kDqk * (d->kv_dtype == MLA_KV_E4M3 ? 1 : 2); }

mla::PagesTable pages_table(int32_t *block_table, const int32_t *seq_lens, int32_t *ref_counts,
                            const mla_pages_desc *d) {
  return mla::PagesTable{block_table, const_cast<int32_t *>(seq_lens), ref_counts, d->num_requests,
                         d->max_pages_per_seq, d->num_pages};
}

// Rows of one request: q_len query tokens x num_heads heads.
int rows_of(const mla_decode_desc *d) { return d->q_len * d->num_heads; }

int head_groups_of(const mla_decode_desc *d) {
  return (rows_of(d) + kSimtHeadsPerGroup - 1) / kSimtHeadsPerGroup;
}

// Builds the decode parameters and enqueues the decode kernel and its split
// merge (arguments already validated).  `fused`: all num_parts partitions in
// one launch (tensor-core path only); out / lse are then [P, B, ...].
int enqueue_decode(const void *q, const void *kv_pages, const int32_t *block_table,
                   const int32_t *seq_lens, int part_id, int num_parts, bool fused,
                   float sm_scale, int lse_base, void *out, float *lse, const mla_decode_desc *d,
                   void *workspace, int grid, cudaStream_t s, void *comb_out = nullptr,
                   float *comb_lse = nullptr) {
  const bool tc = tensor_core_path(d, num_parts);
  if (fused && !fused_path(d, num_parts)) return MLA_ERR_ARG;
  if (d->q_len > 1 && !tc) return MLA_ERR_SHAPE;
  const int per_group = tc ? kTcHeadsPerGroup : kSimtHeadsPerGroup;
  const int rows = rows_of(d);
  const int groups = (rows + per_group - 1) / per_group;
  const int vbatch = fused ? num_parts * d->batch : d->batch;
  mla::DecodeParams p;
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.kv = kv_pages;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.lse = lse;
  p.ws = static_cast<unsigned char *>(workspace);
  p.wl = mla::workspace_layout(vbatch * groups, grid);
  p.batch = vbatch;
  p.heads = rows;
  p.head_groups = groups;
  p.heads_per_group = per_group;
  p.q_len = d->q_len;
  p.q_heads = d->num_heads;
  p.num_pages = d->num_pages;
  p.max_pages = d->max_pages_per_seq;
  p.part_id = fused ? 0 : part_id;
  p.num_parts = num_parts;
  const bool strided = tc && strided_path(d, num_parts);
  const int gp = tc && !strided ? gather_parts(num_parts) : num_parts;
  if (strided) {
    p.strided = 1;
    p.apg = strided_apg(num_parts);
    p.s_q63 = (mla::kPage - 1) / num_parts;
    p.s_r63 = (mla::kPage - 1) % num_parts;
    p.s_c64 = mla::kPage % num_parts;
  } else if (gp < num_parts) {  // owner mask over the gather of partition part_id mod gp of gp
    p.num_parts = gp;
    p.part_id = part_id % gp;
    p.own_parts = num_parts;
    p.own_part = part_id;
  }
  p.fused = fused ? 1 : 0;
  p.req_batch = d->batch;
  p.comb_out = static_cast<__nv_bfloat16 *>(comb_out);
  p.comb_lse = comb_lse;
  p.kv_e4m3 = d->kv_dtype == MLA_KV_E4M3;
  p.kv_scale = p.kv_e4m3 ? d->kv_scale : 1.f;
  p.score_scale_log2 = sm_scale * mla::kLog2e;
  p.lse_base2 = lse_base == MLA_LSE_BASE2;
  cudaError_t e;
  if (tc) {
    CUtensorMap tm_q, tm_kv, tm_kvg, tm_kvb;
    const int h = rows < kTcHeadsPerGroup ? rows : kTcHeadsPerGroup;
    int st = make_tensor_maps(q, kv_pages, d, h, p.part_id, p.num_parts, fused, strided, &tm_q,
                              &tm_kv, &tm_kvg, &tm_kvb);
    if (st != MLA_OK) return st;
    const int npv = ((h + 15) / 16) * 16;
    e = mla::launch_decode_tc(p, npv, h, strided ? 1 : 8 / p.num_parts, tm_q, tm_kv, tm_kvg, tm_kvb,
                              grid, s);
  } else {
    e = mla::launch_decode_simt(p, grid, s);
  }
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

// A view of the whole cache (one partition): see ViewReq.  `view` carries the
// view's own fields; everything else is filled in here.
int enqueue_view(mla::DecodeParams p, const void *q, const void *kv_pages, const int32_t *block_table,
                 const int32_t *seq_lens, float sm_scale, int lse_base, void *out, float *lse,
                 const mla_decode_desc *d, void *workspace, const mla::WorkspaceLayout &wl, int grid,
                 cudaStream_t s) {
  const int rows = rows_of(d);
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.kv = kv_pages;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.lse = lse;
  p.ws = static_cast<unsigned char *>(workspace);
  p.wl = wl;
  p.batch = p.req_batch = d->batch;
  p.heads = rows;
  p.head_groups = (rows + kTcHeadsPerGroup - 1) / kTcHeadsPerGroup;
  p.heads_per_group = kTcHeadsPerGroup;
  p.q_len = d->q_len;
  p.q_heads = d->num_heads;
  p.num_pages = d->num_pages;
  p.max_pages = d->max_pages_per_seq;
  p.part_id = 0;
  p.num_parts = 1;
  p.kv_e4m3 = d->kv_dtype == MLA_KV_E4M3;
  p.kv_scale = p.kv_e4m3 ? d->kv_scale : 1.f;
  p.score_scale_log2 = sm_scale * mla::kLog2e;
  p.lse_base2 = lse_base == MLA_LSE_BASE2;
  // blocks of the shared pages hold up to 64 rows whatever a request's rows
  const long long most = p.view == mla::kViewShared ? (long long)d->batch * rows : rows;
  const int h = int(most < kTcHeadsPerGroup ? most : kTcHeadsPerGroup);
  CUtensorMap tm_q, tm_kv, tm_kvg, tm_kvb;
  int st = make_tensor_maps(q, kv_pages, d, h, 0, 1, false, false, &tm_q, &tm_kv, &tm_kvg, &tm_kvb);
  if (st != MLA_OK) return st;
  if (p.pair_blocks) {
    mla::PairMaps maps;
    st = make_pair_maps(kv_pages, d, &maps);
    if (st != MLA_OK) return st;
    const cudaError_t e = mla::launch_decode_pair(p, tm_q, maps, s);
    if (e != cudaSuccess) return cuda_fail(e);
    if (p.view == mla::kViewWindow || p.pair_tails) return MLA_OK;
  }
  const cudaError_t e = mla::launch_decode_tc(p, (h + 15) / 16 * 16, h, 8, tm_q, tm_kv, tm_kvg, tm_kvb, grid, s);
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

// The checks of a view call's common arguments.
int check_view_call(const void *q, const void *kv_pages, const int32_t *block_table, const int32_t *seq_lens,
                    float sm_scale, int lse_base, const void *out, const float *lse,
                    const mla_decode_desc *d, const void *workspace) {
  if (lse_base != MLA_LSE_NATURAL && lse_base != MLA_LSE_BASE2) return MLA_ERR_ARG;
  if (!(std::isfinite(sm_scale) && sm_scale > 0.f)) return MLA_ERR_ARG;
  if ((long long)d->batch * rows_of(d) > (1LL << 30)) return MLA_ERR_SHAPE;
  if (d->batch == 0) return MLA_OK;
  if (!q || !kv_pages || !block_table || !seq_lens || !out || !lse || !workspace) return MLA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(kv_pages, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(workspace, 256))
    return MLA_ERR_ALIGN;
  return MLA_OK;
}

// Shared pages: blocks of `rows` rows of all groups (an upper bound known on
// the host), and the workspace: a record for every virtual request, and slots
// for every (virtual request, CTA) -- two for every (block, pair) -- enough
// for either kernel of the shared pages.
int shared_blocks(const mla_decode_desc *d, int num_groups, int rows) {
  return int((long long)d->batch * rows_of(d) / rows) + num_groups;
}
mla::WorkspaceLayout shared_layout(const mla_decode_desc *d, int num_groups, int grid) {
  const int groups = (rows_of(d) + kTcHeadsPerGroup - 1) / kTcHeadsPerGroup;
  const int v = shared_blocks(d, num_groups, 64) + d->batch * groups;
  // 2 (blocks of 128 rows + grid / 2) <= rows / 64 + 2 num_groups + grid, and
  // with the tails 2 batch * ceil(request rows / 128) <= batch * (groups + 1) more
  const int slots = v + num_groups + d->batch + 2 * grid;
  return mla::workspace_layout(v, (slots + 1) / 2);
}
// ... and, after all that, the groups' table.
size_t shared_workspace_bytes(const mla::WorkspaceLayout &wl, int num_groups) {
  return mla::align256(wl.total + sizeof(int2) * size_t(num_groups));
}
// The pair kernel takes windows of requests with more than one block of 64 rows
// in the other kernel; its start and end take 2 to 5 us longer on a bf16 cache,
// which rows x tokens in view (at most) have to make up for.  Measured, us a
// call in a graph, pair kernel / blocks of 64 rows, bf16, rows x requests, window:
// 128 x 8, 128 (0.1 M) 24.6 / 18.5; 192 x 8, 128 24.6 / 20.5; 128 x 32, 128 (0.5 M)
// 24.6 / 27.1; 65 x 32, 4096 60 / 74; 128 x 1, 4096 (0.5 M) 27.0 / 24.7; 192 x 8, 512
// (0.8 M) 24.6 / 22.6; 128 x 128, 512 64 / 69; 192 x 128, 4096 272 / 350; 512 x 128,
// 4096 507 / 796; e4m3: 22.5 / 28.1, 22.6 / 28.7, 22.6 / 34.8, 52 / 80, 26.6 / 34.2,
// 24.6 / 32.8, 65 / 90, 230 / 309, 429 / 748.
constexpr long long kWindowPairWork = 1LL << 19;
bool window_pair_path(const mla_decode_desc *d, int window, int sinks) {
  if (rows_of(d) <= kTcHeadsPerGroup) return false;
  const long long rows = (long long)d->batch * rows_of(d);
  const long long seen = (long long)window + sinks, most = (long long)d->max_pages_per_seq * mla::kPage;
  return d->kv_dtype == MLA_KV_E4M3 || rows * (seen < most ? seen : most) >= kWindowPairWork;
}
// The pair kernel takes the shared pages when the groups fill its blocks of 128
// rows on average and there is enough to multiply: it is a kernel more (9 to 13
// us), and nearly twice as fast in the long run.  Rows x tokens of the block
// table bound the work.  Measured, us a call in a graph, pair kernel / blocks of 64
// rows in the one kernel, 64 rows a request, 100 own tokens, bf16: 4096 rows x 1K
// shared tokens 47 / 33, 1024 x 8K 47 / 39, 256 x 32K 47 / 40, 512 x 32K 59 / 59, 4096 x
// 8K 82 / 101, 4096 x 32K 219 / 364; e4m3: 55 / 47, 57 / 47, 58 / 45, 64 / 59, 90 / 96,
// 202 / 275.  These tables were as wide as the work; only the device knows the
// tokens.  A table made for far longer requests sends short shared pages to the
// pair kernel too: 2,200 columns, 128 rows over 256 shared tokens and 100 own ones
// 32.5 / 18.4, over 4K 32.8 / 22.5, 1024 rows over 1K 36.9 / 22.6, over 8K 47 / 41;
// e4m3 45 / 29, 45 / 35, 50 / 35, 60 / 49.
constexpr long long kPairWork = 16LL << 20;
bool pair_path(const mla_decode_desc *d, int num_groups) {
  const long long rows = (long long)d->batch * rows_of(d);
  return rows >= 128LL * num_groups &&
         rows * mla::kPage >= kPairWork / d->max_pages_per_seq;
}
// Records of the chunks' blocks, one a pair, and two slots of 64 rows for each CTA.
mla::WorkspaceLayout chunk_layout(int sms) { return mla::workspace_layout(sms, sms); }

constexpr int kMaxGroups = 1 << 20;
constexpr int kMaxView = 1 << 30;
constexpr int kMaxChunkBatch = 1 << 20;

// The expanded prefill's loads: (dims, heads, tokens) of each tensor, 64 dims of `box`
// tokens of a head.  Without keys nothing is loaded through the maps of k and v, which
// then describe a row of q.
int make_expanded_maps(const void *q, const void *k_nope, const void *k_rope, const void *v,
                       const mla_expanded_desc *d, mla::ExpandedMaps *m) {
  EncodeTiled enc = encode_tiled();
  if (!enc) {
    std::snprintf(g_cuda_error, sizeof(g_cuda_error), "cuTensorMapEncodeTiled unavailable");
    return MLA_ERR_CUDA;
  }
  CUresult r = CUDA_SUCCESS;
  auto map = [&](CUtensorMap *tm, const void *base, int width, int heads, int64_t tokens, int64_t head_stride,
                 int64_t token_stride, int box_tokens) {
    const bool flat = heads == 0;  // (dims, tokens)
    cuuint64_t dims[3] = {cuuint64_t(width), cuuint64_t(flat ? tokens : heads), cuuint64_t(tokens)};
    cuuint64_t strides[2] = {cuuint64_t(flat ? token_stride : head_stride) * 2, cuuint64_t(token_stride) * 2};
    cuuint32_t box[3] = {64, flat ? cuuint32_t(box_tokens) : 1u, cuuint32_t(box_tokens)}, es[3] = {1, 1, 1};
    if (r == CUDA_SUCCESS)
      r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, flat ? 2 : 3, const_cast<void *>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  const int H = d->num_heads;
  map(&m->q, q, mla::kNope + mla::kRope, H, d->q_tokens, d->q_head_stride, d->q_token_stride, 128);
  if (d->k_tokens == 0) {
    m->k_nope = m->k_rope = m->v = m->va = m->vr = m->q;
  } else {
    map(&m->k_nope, k_nope, mla::kNope, H, d->k_tokens, d->k_head_stride, d->k_token_stride, 64);
    map(&m->k_rope, k_rope, mla::kRope, 0, d->k_tokens, 0, d->rope_token_stride, 64);
    map(&m->v, v, mla::kDvx, H, d->k_tokens, d->v_head_stride, d->v_token_stride, 128);
    map(&m->va, v, mla::kDvx, H, d->k_tokens, d->v_head_stride, d->v_token_stride, 8);
    map(&m->vr, v, mla::kDvx, H, d->k_tokens, d->v_head_stride, d->v_token_stride, 1);
  }
  return r == CUDA_SUCCESS ? MLA_OK : tensor_map_fail("expanded", r);
}

// kv_append_chunk and kv_read: `buffer` is the contiguous side.
int kv_chunk(bool read, void *kv_pages, void *buffer, int64_t stride, int rows, const int32_t *block_table,
             const int32_t *starts, const int32_t *positions, int part_id, int num_parts, const mla_decode_desc *d,
             int32_t *error_word, mla_stream_t stream) {
  int st = check_cache_desc(d);
  if (st != MLA_OK) return st;
  if (rows < 0 || stride < mla::kDqk || stride > (1LL << 40)) return MLA_ERR_SHAPE;
  if (num_parts < 1 || part_id < 0 || part_id >= num_parts) return MLA_ERR_PARTITION;
  if (d->batch == 0 || rows == 0) return MLA_OK;
  if (!buffer || !kv_pages || !block_table || !starts || !positions) return MLA_ERR_NULL;
  if (!aligned(buffer, 16) || stride % 8 != 0 || !aligned(kv_pages, 16) || !aligned(block_table, 4) ||
      !aligned(starts, 4) || !aligned(positions, 4) || !aligned(error_word, 4))
    return MLA_ERR_ALIGN;
  current_device(&st);
  if (st != MLA_OK) return st;
  const cudaError_t e = mla::launch_kv_chunk(read, kv_pages, buffer, stride, block_table, starts, positions, rows,
                                             d->batch, part_id, num_parts, d->num_pages, d->max_pages_per_seq,
                                             d->kv_dtype == MLA_KV_E4M3, d->kv_scale, error_word,
                                             reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

}  // namespace

namespace mla {
// The decode partial of one partition on a caller-chosen workspace and grid
// (arguments already validated): the path of the allocation-free entry point.
int enqueue_partial(const void *q, const void *kv_pages, const int32_t *block_table,
                    const int32_t *seq_lens, int part_id, int num_parts, float sm_scale,
                    int lse_base, void *out, float *lse, const mla_decode_desc *d,
                    void *workspace, int grid, cudaStream_t s) {
  return enqueue_decode(q, kv_pages, block_table, seq_lens, part_id, num_parts, false, sm_scale,
                        lse_base, out, lse, d, workspace, grid, s);
}
}  // namespace mla

extern "C" {

int mla_version(void) { return 100; }

// The kernels are built for sm_103a only (arch-specific tcgen05 and TMA
// forms): any other compute capability, sm_100 included, is refused.
int mla_arch_supported(int major, int minor) { return major == 10 && minor == 3 ? 1 : 0; }

const char *mla_status_string(int status) {
  switch (status) {
    case MLA_OK: return "ok";
    case MLA_ERR_NULL: return "a required pointer is NULL";
    case MLA_ERR_SHAPE: return "unsupported shape (q_len 1..16, and 1 off the tensor-core path: num_parts / gcd(num_parts, 8) > 16; Dqk 576, Dv 512, page 64, heads 1..128)";
    case MLA_ERR_PARTITION: return "bad partition (need num_parts >= 1 and 0 <= part_id < num_parts)";
    case MLA_ERR_ALIGN: return "misaligned pointer (16 B for tensors, 256 B for the workspace)";
    case MLA_ERR_WORKSPACE: return "workspace too small";
    case MLA_ERR_ARG: return "bad argument value";
    case MLA_ERR_CUDA: return "CUDA error (see mla_last_cuda_error)";
    case MLA_ERR_DEVICE: return "current device is not an sm_103 GPU";
    case MLA_ERR_BOUNDS: return "block-table entry or sequence length out of bounds";
    case MLA_ERR_TIMEOUT: return "a bounded wait inside the kernel gave up";
    default: return "unknown status";
  }
}

const char *mla_last_cuda_error(void) { return g_cuda_error; }

size_t mla_decode_workspace_size(const mla_decode_desc *d, int num_sms) {
  if (check_desc(d) != MLA_OK) return 0;
  if (num_sms <= 0) {
    int st = 0;
    DeviceFacts f = current_device(&st);
    if (f.sms <= 0) return 0;
    num_sms = f.sms;
  }
  const int virt = d->batch * head_groups_of(d);
  return mla::workspace_layout(virt, num_sms).total;
}

int mla_decode_partial(const void *q, const void *kv_pages, const int32_t *block_table,
                       const int32_t *seq_lens, int part_id, int num_parts, float sm_scale,
                       int lse_base, void *out, float *lse, const mla_decode_desc *d,
                       void *workspace, size_t workspace_bytes, mla_stream_t stream) {
  int st = check_desc(d);
  if (st != MLA_OK) return st;
  if (num_parts < 1 || part_id < 0 || part_id >= num_parts) return MLA_ERR_PARTITION;
  if (d->q_len > 1 && !tensor_core_path(d, num_parts)) return MLA_ERR_SHAPE;
  if (lse_base != MLA_LSE_NATURAL && lse_base != MLA_LSE_BASE2) return MLA_ERR_ARG;
  if (!std::isfinite(sm_scale)) return MLA_ERR_ARG;
  if (d->batch == 0) return MLA_OK;
  if (!q || !kv_pages || !block_table || !seq_lens || !out || !lse || !workspace)
    return MLA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(kv_pages, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(workspace, 256))
    return MLA_ERR_ALIGN;

  DeviceFacts f = current_device(&st);
  if (st != MLA_OK) return st;
  if (workspace_bytes < mla::workspace_layout(d->batch * head_groups_of(d), f.sms).total)
    return MLA_ERR_WORKSPACE;
  return enqueue_decode(q, kv_pages, block_table, seq_lens, part_id, num_parts, false, sm_scale,
                        lse_base, out, lse, d, workspace, f.sms,
                        reinterpret_cast<cudaStream_t>(stream));
}

size_t mla_decode_dcp_workspace_size(const mla_decode_desc *d, int num_parts, int num_sms) {
  if (check_desc(d) != MLA_OK || num_parts < 1) return 0;
  if (num_sms <= 0) {
    int st = 0;
    DeviceFacts f = current_device(&st);
    if (f.sms <= 0) return 0;
    num_sms = f.sms;
  }
  const long long virt = (long long)num_parts * d->batch * head_groups_of(d);
  if (virt > (1LL << 30)) return 0;
  return mla::workspace_layout(int(virt), num_sms).total;
}

int mla_decode_dcp(const void *q, const void *kv_pages, const int32_t *block_table,
                   const int32_t *seq_lens, int num_parts, float sm_scale, int lse_base,
                   void *partials, float *partial_lses, void *out, float *out_lse,
                   const mla_decode_desc *d, void *workspace, size_t workspace_bytes,
                   mla_stream_t stream) {
  int st = check_desc(d);
  if (st != MLA_OK) return st;
  if (num_parts < 1 || num_parts > mla::combine_max_parts()) return MLA_ERR_PARTITION;
  if (lse_base != MLA_LSE_NATURAL && lse_base != MLA_LSE_BASE2) return MLA_ERR_ARG;
  if (!std::isfinite(sm_scale)) return MLA_ERR_ARG;
  if (d->batch == 0) return MLA_OK;
  if ((long long)num_parts * d->batch * rows_of(d) > (1LL << 30)) return MLA_ERR_SHAPE;
  if (d->q_len > 1 && !tensor_core_path(d, num_parts)) return MLA_ERR_SHAPE;
  if (!q || !kv_pages || !block_table || !seq_lens || !partials || !partial_lses || !out ||
      !workspace)
    return MLA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(kv_pages, 16) || !aligned(partials, 16) ||
      !aligned(partial_lses, 4) || !aligned(out, 16) || !aligned(out_lse, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(workspace, 256))
    return MLA_ERR_ALIGN;
  DeviceFacts f = current_device(&st);
  if (st != MLA_OK) return st;
  if (workspace_bytes < mla_decode_dcp_workspace_size(d, num_parts, f.sms))
    return MLA_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const size_t rows = size_t(d->batch) * rows_of(d);
  if (num_parts > 1 && fused_path(d, num_parts)) {
    // every partition in one decode launch, then one kernel that merges the
    // splits and combines the partitions (one partition takes the loop below:
    // the single-partition kernel, whose tiles are one page each, and the
    // combine, then a copy)
    return enqueue_decode(q, kv_pages, block_table, seq_lens, 0, num_parts, true, sm_scale,
                          lse_base, partials, partial_lses, d, workspace, f.sms, s, out,
                          out_lse);
  } else {
    for (int r = 0; r < num_parts; ++r) {
      st = enqueue_decode(q, kv_pages, block_table, seq_lens, r, num_parts, false, sm_scale,
                          lse_base, static_cast<__nv_bfloat16 *>(partials) + r * rows * mla::kDv,
                          partial_lses + r * rows, d, workspace, f.sms, s);
      if (st != MLA_OK) return st;
    }
  }
  cudaError_t e = mla::launch_lse_combine(partials, partial_lses, num_parts, out, out_lse,
                                          int(rows), mla::kDv, lse_base == MLA_LSE_BASE2, s);
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

int mla_kv_append(const void *kv_new, void *kv_pages, const int32_t *block_table,
                  const int32_t *positions, int part_id, int num_parts,
                  const mla_decode_desc *d, int32_t *error_word, mla_stream_t stream) {
  int st = check_cache_desc(d);
  if (st != MLA_OK) return st;
  if (num_parts < 1 || part_id < 0 || part_id >= num_parts) return MLA_ERR_PARTITION;
  if (d->batch == 0) return MLA_OK;
  if (!kv_new || !kv_pages || !block_table || !positions) return MLA_ERR_NULL;
  if (!aligned(kv_new, 16) || !aligned(kv_pages, 16) || !aligned(block_table, 4) ||
      !aligned(positions, 4) || !aligned(error_word, 4))
    return MLA_ERR_ALIGN;
  current_device(&st);
  if (st != MLA_OK) return st;
  cudaError_t e = mla::launch_kv_append(kv_new, kv_pages, block_table, positions, d->batch,
                                        part_id, num_parts, d->num_pages, d->max_pages_per_seq,
                                        d->kv_dtype == MLA_KV_E4M3, d->kv_scale, error_word,
                                        reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

int mla_kv_append_chunk(const void *kv_new, int64_t row_stride, int num_rows, void *kv_pages,
                        const int32_t *block_table, const int32_t *chunk_starts, const int32_t *positions,
                        int part_id, int num_parts, const mla_decode_desc *d, int32_t *error_word,
                        mla_stream_t stream) {
  return kv_chunk(false, kv_pages, const_cast<void *>(kv_new), row_stride, num_rows, block_table, chunk_starts,
                  positions, part_id, num_parts, d, error_word, stream);
}

int mla_kv_read(const void *kv_pages, const int32_t *block_table, const int32_t *read_starts,
                const int32_t *positions, void *out, int64_t row_stride, int num_rows, const mla_decode_desc *d,
                int32_t *error_word, mla_stream_t stream) {
  return kv_chunk(true, const_cast<void *>(kv_pages), out, row_stride, num_rows, block_table, read_starts, positions,
                  0, 1, d, error_word, stream);
}

size_t mla_prefill_workspace_size(int num_sms) {
  if (num_sms <= 0) {
    int st = 0;
    DeviceFacts f = current_device(&st);
    if (f.sms <= 0) return 0;
    num_sms = f.sms;
  }
  const size_t chunk = chunk_layout(num_sms).total, expanded = mla::expanded_layout(num_sms / 2).total;
  return chunk > expanded ? chunk : expanded;
}

int mla_prefill_chunk(const void *q, int num_tokens, const void *kv_pages, const int32_t *block_table,
                      const int32_t *seq_lens, const int32_t *chunk_starts, float sm_scale, int lse_base, void *out,
                      float *lse, const mla_decode_desc *d, void *workspace, size_t workspace_bytes,
                      mla_stream_t stream) {
  int st = check_desc(d);
  if (st != MLA_OK) return st;
  if (num_tokens < 0 || (long long)num_tokens * d->num_heads > (1LL << 30) || d->batch > kMaxChunkBatch)
    return MLA_ERR_SHAPE;
  if (lse_base != MLA_LSE_NATURAL && lse_base != MLA_LSE_BASE2) return MLA_ERR_ARG;
  if (!(std::isfinite(sm_scale) && sm_scale > 0.f)) return MLA_ERR_ARG;
  if (d->batch == 0 || num_tokens == 0) return MLA_OK;
  if (!q || !kv_pages || !block_table || !seq_lens || !chunk_starts || !out || !lse || !workspace)
    return MLA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(kv_pages, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(chunk_starts, 4) || !aligned(workspace, 256))
    return MLA_ERR_ALIGN;
  const DeviceFacts f = current_device(&st);
  if (st != MLA_OK) return st;
  mla::DecodeParams p;
  p.wl = chunk_layout(f.sms);
  if (workspace_bytes < p.wl.total) return MLA_ERR_WORKSPACE;
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.kv = kv_pages;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.lse = lse;
  p.ws = static_cast<unsigned char *>(workspace);
  p.view = mla::kViewChunk;
  p.chunk_starts = chunk_starts;
  p.chunk_tokens = num_tokens;
  p.batch = p.req_batch = d->batch;
  p.heads = p.q_heads = d->num_heads;
  p.head_groups = 1;
  p.heads_per_group = kTcHeadsPerGroup;
  p.num_pages = d->num_pages;
  p.max_pages = d->max_pages_per_seq;
  p.part_id = 0;
  p.num_parts = 1;
  p.pairs = f.sms / 2;
  p.pair_blocks = int((long long)num_tokens * d->num_heads / 128) + d->batch;
  p.kv_e4m3 = d->kv_dtype == MLA_KV_E4M3;
  p.kv_scale = p.kv_e4m3 ? d->kv_scale : 1.f;
  p.score_scale_log2 = sm_scale * mla::kLog2e;
  p.lse_base2 = lse_base == MLA_LSE_BASE2;
  mla::PairMaps maps;
  st = make_pair_maps(kv_pages, d, &maps);
  if (st != MLA_OK) return st;
  CUtensorMap tm_q;
  st = make_q_map(encode_tiled(), q, cuuint64_t(num_tokens) * d->num_heads, 64, &tm_q);
  if (st != MLA_OK) return st;
  const cudaError_t e = mla::launch_decode_pair(p, tm_q, maps, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

int mla_prefill_expanded(const void *q, const void *k_nope, const void *k_rope, const void *v,
                         const int32_t *q_starts, const int32_t *k_starts, float sm_scale, int lse_base, void *out,
                         float *lse, const mla_expanded_desc *d, void *workspace, size_t workspace_bytes,
                         mla_stream_t stream) {
  if (!d) return MLA_ERR_NULL;
  if (d->batch < 0 || d->batch > kMaxChunkBatch || d->q_tokens < 0 || d->k_tokens < 0 || d->num_heads < 1 ||
      d->num_heads > 128 || (long long)d->q_tokens * d->num_heads > (1LL << 30) || d->k_tokens > (1 << 30))
    return MLA_ERR_SHAPE;
  if (lse_base != MLA_LSE_NATURAL && lse_base != MLA_LSE_BASE2) return MLA_ERR_ARG;
  if (!(std::isfinite(sm_scale) && sm_scale > 0.f)) return MLA_ERR_ARG;
  if (d->causal != 0 && d->causal != 1) return MLA_ERR_ARG;
  if (d->batch == 0 || d->q_tokens == 0) return MLA_OK;
  const bool keys = d->k_tokens > 0;
  if (!q || !q_starts || !k_starts || !out || !lse || !workspace || (keys && (!k_nope || !k_rope || !v)))
    return MLA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(q_starts, 4) || !aligned(k_starts, 4) ||
      !aligned(workspace, 256) || (keys && (!aligned(k_nope, 16) || !aligned(k_rope, 16) || !aligned(v, 16))))
    return MLA_ERR_ALIGN;
  const int64_t strides[7] = {d->q_token_stride, d->q_head_stride, d->k_token_stride, d->k_head_stride,
                              d->rope_token_stride, d->v_token_stride, d->v_head_stride};
  for (int i = keys ? 6 : 1; i >= 0; --i) {
    if (strides[i] <= 0 || strides[i] >= (1LL << 38)) return MLA_ERR_SHAPE;
    if (strides[i] % 8 != 0) return MLA_ERR_ALIGN;
  }
  int st = MLA_OK;
  const DeviceFacts f = current_device(&st);
  if (st != MLA_OK) return st;
  mla::ExpandedParams p;
  p.pairs = f.sms / 2;
  if (workspace_bytes < mla::expanded_layout(p.pairs).total) return MLA_ERR_WORKSPACE;
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.lse = lse;
  p.ws = static_cast<unsigned char *>(workspace);
  p.q_starts = q_starts;
  p.k_starts = k_starts;
  p.batch = d->batch;
  p.heads = d->num_heads;
  p.q_tokens = d->q_tokens;
  p.k_tokens = d->k_tokens;
  p.causal = d->causal;
  p.blocks = d->q_tokens / mla::kExpRows + d->batch;
  p.score_scale_log2 = sm_scale * mla::kLog2e;
  p.lse_base2 = lse_base == MLA_LSE_BASE2;
  mla::ExpandedMaps m;
  st = make_expanded_maps(q, keys ? k_nope : q, keys ? k_rope : q, keys ? v : q, d, &m);
  if (st != MLA_OK) return st;
  const cudaError_t e = mla::launch_prefill_expanded(p, m, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

int mla_dcp_local_metadata(const int32_t *seq_lens, const int32_t *req_pool_indices,
                           const int32_t *req_to_token, int part_id, int num_parts,
                           const mla_dcp_meta_desc *d, int32_t *global_lens,
                           int32_t *local_lens, int32_t *block_table, int32_t *error_word,
                           mla_stream_t stream) {
  if (!d) return MLA_ERR_NULL;
  if (num_parts < 1 || part_id < 0 || part_id >= num_parts) return MLA_ERR_PARTITION;
  if (d->batch < 0 || d->num_req_slots < 1 || d->req_to_token_width < 1 ||
      d->max_pages_per_seq < 1 || d->page_size != mla::kPage)
    return MLA_ERR_SHAPE;
  if (d->extra_tokens < 0) return MLA_ERR_ARG;
  if (d->batch == 0) return MLA_OK;
  if (!seq_lens || !req_pool_indices || !req_to_token || !global_lens || !local_lens ||
      !block_table)
    return MLA_ERR_NULL;
  if (!aligned(seq_lens, 4) || !aligned(req_pool_indices, 4) || !aligned(req_to_token, 4) ||
      !aligned(global_lens, 4) || !aligned(local_lens, 4) || !aligned(block_table, 4) ||
      !aligned(error_word, 4))
    return MLA_ERR_ALIGN;
  int st = 0;
  current_device(&st);
  if (st != MLA_OK) return st;
  cudaError_t e = mla::launch_dcp_metadata(
      seq_lens, req_pool_indices, req_to_token, d->batch, d->num_req_slots, d->req_to_token_width,
      d->extra_tokens, part_id, num_parts, global_lens, local_lens, block_table,
      d->max_pages_per_seq, d->pad_value, error_word, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

int mla_decode_check_workspace(void *workspace, mla_stream_t stream) {
  if (!workspace) return MLA_ERR_NULL;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int word = 0;
  cudaError_t e = cudaStreamSynchronize(s);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&word, workspace, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(workspace, 0, sizeof(int), s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e);
  if (word & mla::kErrTimeout) return MLA_ERR_TIMEOUT;
  return word ? MLA_ERR_BOUNDS : MLA_OK;
}

int mla_lse_combine(const void *partials, const float *lses, int num_parts, void *out,
                    const mla_combine_desc *d, mla_stream_t stream) {
  if (!d) return MLA_ERR_NULL;
  if (num_parts < 1 || num_parts > mla::combine_max_parts()) return MLA_ERR_PARTITION;
  if (d->num_tokens < 0 || d->num_heads < 1) return MLA_ERR_SHAPE;
  if (d->head_dim < 8 || d->head_dim > 1024 || d->head_dim % 8) return MLA_ERR_SHAPE;
  if (d->lse_base != MLA_LSE_NATURAL && d->lse_base != MLA_LSE_BASE2) return MLA_ERR_ARG;
  if (d->num_tokens == 0) return MLA_OK;
  if (!partials || !lses || !out) return MLA_ERR_NULL;
  if (!aligned(partials, 16) || !aligned(out, 16) || !aligned(lses, 4) ||
      (d->out_lse && !aligned(d->out_lse, 4)))
    return MLA_ERR_ALIGN;
  int st = 0;
  current_device(&st);
  if (st != MLA_OK) return st;
  const long long rows = (long long)d->num_tokens * d->num_heads;
  if (rows > (1LL << 30)) return MLA_ERR_SHAPE;
  cudaError_t e = mla::launch_lse_combine(partials, lses, num_parts, out, d->out_lse, int(rows),
                                          d->head_dim, d->lse_base == MLA_LSE_BASE2,
                                          reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

size_t mla_pages_workspace_size(int num_pages) {
  return num_pages < 1 ? 0 : mla::pages_workspace_bytes(num_pages);
}

int mla_pages_copy(const void *src_pages, void *dst_pages, const int32_t *src, const int32_t *dst, int n,
                   int dst_num_pages, const mla_pages_desc *d, int32_t *error_word, mla_stream_t stream) {
  int st = check_pages_desc(d);
  if (st != MLA_OK) return st;
  if (n < 0) return MLA_ERR_ARG;
  if (dst_num_pages < 1) return MLA_ERR_SHAPE;
  if (n == 0) return MLA_OK;
  if (!src_pages || !dst_pages || !src || !dst) return MLA_ERR_NULL;
  if (!aligned(src_pages, 16) || !aligned(dst_pages, 16) || !aligned(src, 4) || !aligned(dst, 4) ||
      !aligned(error_word, 4))
    return MLA_ERR_ALIGN;
  current_device(&st);
  if (st != MLA_OK) return st;
  cudaError_t e = mla::launch_pages_copy(src_pages, dst_pages, src, dst, n, d->num_pages, dst_num_pages,
                                         pages_row_bytes(d), error_word,
                                         reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

int mla_pages_fork(void *kv_pages, int32_t *block_table, int32_t *seq_lens, int32_t *ref_counts,
                   const int32_t *parents, const int32_t *children, int n, const mla_pages_desc *d,
                   void *workspace, size_t workspace_bytes, int32_t *error_word, mla_stream_t stream) {
  int st = check_pages_desc(d);
  if (st != MLA_OK) return st;
  if (n < 0 || n > mla::kMaxForks) return MLA_ERR_ARG;
  if (n == 0 || d->num_requests == 0) return MLA_OK;
  if (!kv_pages || !block_table || !seq_lens || !ref_counts || !parents || !children || !workspace)
    return MLA_ERR_NULL;
  if (!aligned(kv_pages, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(ref_counts, 4) || !aligned(parents, 4) || !aligned(children, 4) || !aligned(workspace, 256) ||
      !aligned(error_word, 4))
    return MLA_ERR_ALIGN;
  if (workspace_bytes < mla_pages_workspace_size(d->num_pages)) return MLA_ERR_WORKSPACE;
  current_device(&st);
  if (st != MLA_OK) return st;
  cudaError_t e = mla::launch_pages_fork(pages_table(block_table, seq_lens, ref_counts, d), kv_pages,
                                         pages_row_bytes(d), parents, children, n,
                                         mla::pages_workspace(workspace, d->num_pages), error_word,
                                         reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

int mla_pages_alloc(int32_t *block_table, const int32_t *seq_lens, int32_t *ref_counts,
                    const int32_t *new_lens, const mla_pages_desc *d, void *workspace,
                    size_t workspace_bytes, int32_t *error_word, mla_stream_t stream) {
  int st = check_pages_desc(d);
  if (st != MLA_OK) return st;
  if (d->num_requests == 0) return MLA_OK;
  if (!block_table || !seq_lens || !ref_counts || !new_lens || !workspace) return MLA_ERR_NULL;
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(ref_counts, 4) ||
      !aligned(new_lens, 4) || !aligned(workspace, 256) || !aligned(error_word, 4))
    return MLA_ERR_ALIGN;
  if (workspace_bytes < mla_pages_workspace_size(d->num_pages)) return MLA_ERR_WORKSPACE;
  current_device(&st);
  if (st != MLA_OK) return st;
  cudaError_t e = mla::launch_pages_alloc(pages_table(block_table, seq_lens, ref_counts, d), new_lens,
                                          mla::pages_workspace(workspace, d->num_pages), error_word,
                                          reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

int mla_pages_free(int32_t *block_table, int32_t *seq_lens, int32_t *ref_counts, const int32_t *new_lens,
                   int window, int sinks, const mla_pages_desc *d, int32_t *error_word,
                   mla_stream_t stream) {
  int st = check_pages_desc(d);
  if (st != MLA_OK) return st;
  if (window < 0 || sinks < 0) return MLA_ERR_ARG;
  if (d->num_requests == 0) return MLA_OK;
  if (!block_table || !seq_lens || !ref_counts || !new_lens) return MLA_ERR_NULL;
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(ref_counts, 4) ||
      !aligned(new_lens, 4) || !aligned(error_word, 4))
    return MLA_ERR_ALIGN;
  current_device(&st);
  if (st != MLA_OK) return st;
  cudaError_t e = mla::launch_pages_free(pages_table(block_table, seq_lens, ref_counts, d), new_lens, window,
                                         sinks, error_word, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

int mla_pages_compact(void *kv_pages, int32_t *block_table, int32_t *ref_counts, int32_t *remap,
                      const mla_pages_desc *d, void *workspace, size_t workspace_bytes,
                      int32_t *error_word, mla_stream_t stream) {
  int st = check_pages_desc(d);
  if (st != MLA_OK) return st;
  if (!kv_pages || (!block_table && d->num_requests > 0) || !ref_counts || !workspace) return MLA_ERR_NULL;
  if (!aligned(kv_pages, 16) || !aligned(block_table, 4) || !aligned(ref_counts, 4) || !aligned(remap, 4) ||
      !aligned(workspace, 256) || !aligned(error_word, 4))
    return MLA_ERR_ALIGN;
  if (workspace_bytes < mla_pages_workspace_size(d->num_pages)) return MLA_ERR_WORKSPACE;
  DeviceFacts f = current_device(&st);
  if (st != MLA_OK) return st;
  cudaError_t e = mla::launch_pages_compact(pages_table(block_table, nullptr, ref_counts, d), kv_pages,
                                            pages_row_bytes(d), remap, 4 * f.sms,
                                            mla::pages_workspace(workspace, d->num_pages), error_word,
                                            reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

int mla_decode_window(const void *q, const void *kv_pages, const int32_t *block_table,
                      const int32_t *seq_lens, int window, int sinks, float sm_scale, int lse_base,
                      void *out, float *lse, const mla_decode_desc *d, void *workspace,
                      size_t workspace_bytes, mla_stream_t stream) {
  int st = check_desc(d);
  if (st != MLA_OK) return st;
  if (window < 1 || sinks < 0) return MLA_ERR_ARG;
  st = check_view_call(q, kv_pages, block_table, seq_lens, sm_scale, lse_base, out, lse, d, workspace);
  if (st != MLA_OK || d->batch == 0) return st;
  DeviceFacts f = current_device(&st);
  if (st != MLA_OK) return st;
  const auto wl = mla::workspace_layout(d->batch * head_groups_of(d), f.sms);
  if (workspace_bytes < wl.total) return MLA_ERR_WORKSPACE;
  mla::DecodeParams p;
  p.view = mla::kViewWindow;
  if (window_pair_path(d, window, sinks)) {
    // (all pairs, not 16 pieces a block as below: capped, one request of 128 rows took
    // 34.9 us instead of 41.0 at a window of 16,000, 28.7 instead of 30.8 at 8,192, and
    // two or four requests the same or up to 4 us more)
    p.pair_blocks = d->batch * ((rows_of(d) + 127) / 128);
    p.pairs = f.sms / 2;
  }
  // (longer than any request: the kernel's sums with them stay in 32 bits)
  p.window = window < kMaxView ? window : kMaxView;
  p.sinks = sinks < kMaxView ? sinks : kMaxView;
  // Blocks of 64 rows: up to 16 pieces a block.  The merge takes a block's pieces one after another,
  // and one request cut across all CTAs waits longer for it than it gains.
  // Measured, us a call, 8 / 16 / 24 pieces / all CTAs, bf16, 64 rows: 1 request,
  // window 2000 21.3 / 20.2 / 20.5 / 25.5, 4096 27.0 / 23.4 / 22.3 / 37.0; 4
  // requests 22.9 / 21.1 / 22.4 / 26.0, 28.8 / 24.2 / 23.9 / 27.2; 16 rows, 4
  // requests 18.5 / 17.9 / 19.5 / 22.9; e4m3, 64 rows: 1 request, 4096 36.3 / 31.4 /
  // 31.8 / 44.7.
  const long long blocks = (long long)d->batch * ((rows_of(d) + kTcHeadsPerGroup - 1) / kTcHeadsPerGroup);
  const int grid = int(16 * blocks < f.sms ? 16 * blocks : f.sms);
  return enqueue_view(p, q, kv_pages, block_table, seq_lens, sm_scale, lse_base, out, lse, d, workspace, wl, grid,
                      reinterpret_cast<cudaStream_t>(stream));
}

size_t mla_decode_shared_workspace_size(const mla_decode_desc *d, int num_groups, int num_sms) {
  if (check_desc(d) != MLA_OK || num_groups < 1 || num_groups > kMaxGroups) return 0;
  if ((long long)d->batch * rows_of(d) > (1LL << 30)) return 0;
  if (num_sms <= 0) {
    int st = 0;
    DeviceFacts f = current_device(&st);
    if (f.sms <= 0) return 0;
    num_sms = f.sms;
  }
  return shared_workspace_bytes(shared_layout(d, num_groups, num_sms), num_groups);
}

int mla_decode_shared(const void *q, const void *kv_pages, const int32_t *block_table,
                      const int32_t *seq_lens, const int32_t *group_starts, const int32_t *shared_pages,
                      int num_groups, float sm_scale, int lse_base, void *out, float *lse,
                      const mla_decode_desc *d, void *workspace, size_t workspace_bytes,
                      mla_stream_t stream) {
  int st = check_desc(d);
  if (st != MLA_OK) return st;
  if (num_groups < 1 || num_groups > kMaxGroups) return MLA_ERR_ARG;
  st = check_view_call(q, kv_pages, block_table, seq_lens, sm_scale, lse_base, out, lse, d, workspace);
  if (st != MLA_OK || d->batch == 0) return st;
  if (!group_starts || !shared_pages) return MLA_ERR_NULL;
  if (!aligned(group_starts, 4) || !aligned(shared_pages, 4)) return MLA_ERR_ALIGN;
  DeviceFacts f = current_device(&st);
  if (st != MLA_OK) return st;
  const auto wl = shared_layout(d, num_groups, f.sms);
  if (workspace_bytes < shared_workspace_bytes(wl, num_groups)) return MLA_ERR_WORKSPACE;
  mla::DecodeParams p;
  p.view = mla::kViewShared;
  p.group_starts = group_starts;
  p.shared_pages = shared_pages;
  p.num_groups = num_groups;
  p.group_table = reinterpret_cast<int2 *>(static_cast<unsigned char *>(workspace) + wl.total);
  if (pair_path(d, num_groups)) {
    // the tails of requests with more than one block of 64 rows go along, a launch
    // less and the pair kernel's rate; us a call in a graph, tails along / in the other
    // kernel, bf16: 256 rows x 39 requests, 131 shared pages + 700 tokens 168 / 186, 128 x
    // 64, 128 + 1500 144 / 181, + 1 130 / 136, 512 x 32, 400 + 1 624 / 605, + 1500
    // 665 / 683; e4m3: 150 / 185, 135 / 178, 113 / 132, 553 / 537, 606 / 619
    if (rows_of(d) > kTcHeadsPerGroup) p.pair_tails = d->batch * ((rows_of(d) + 127) / 128);
    p.pair_blocks = shared_blocks(d, num_groups, 128) + p.pair_tails;
    p.pairs = f.sms / 2;
  } else {
    p.prefix_blocks = shared_blocks(d, num_groups, 64);
  }
  return enqueue_view(p, q, kv_pages, block_table, seq_lens, sm_scale, lse_base, out, lse, d, workspace, wl,
                      f.sms, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
