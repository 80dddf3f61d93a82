// Shared by the page operations' kernels and their host entries.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mla {

constexpr int kPagesChunk = 1024;  // pages whose free ones one CTA counts and lists

// Bits of a page operation's error word.
constexpr int kErrPagesEntry = 1;  // an index, length or table entry out of range
constexpr int kErrPagesFull = 2;   // no free page left for a fork or a request

struct PagesTable {
  int32_t *block_table;  // [rows, width], -1: no page
  int32_t *seq_lens;     // [rows]
  int32_t *ref_counts;   // [num_pages], 0: free
  int rows, width, num_pages;
};

__host__ __device__ constexpr int pages_chunks(int num_pages) {
  return int(((long long)num_pages + kPagesChunk - 1) / kPagesChunk);
}

// int32 arrays in the caller's workspace; every call writes what it reads.
struct PagesWorkspace {
  int32_t *totals;      // [64]: live pages, moves
  int32_t *chunk_free;  // [chunks]
  int32_t *free_list;   // [chunks][kPagesChunk]: a chunk's free ids, ascending
  int32_t *holes;       // the same memory, as one list (compaction)
  int32_t *movers;      // [num_pages], by rank among the live pages
  int32_t *rank;        // [num_pages]: a live page's rank, -1 for a free page
  int32_t *fork_count;  // the same memory as movers and rank: forks that need a page, by blocks
};
constexpr int kMaxForks = 1 << 19;  // what a one-chunk workspace's fork_count holds

constexpr size_t pages_workspace_bytes(int num_pages) {
  const size_t c = size_t(pages_chunks(num_pages));
  return 4 * (64 + (c + 63) / 64 * 64 + 3 * c * kPagesChunk);
}

inline PagesWorkspace pages_workspace(void *base, int num_pages) {
  const size_t c = size_t(pages_chunks(num_pages));
  int32_t *p = static_cast<int32_t *>(base);
  PagesWorkspace w;
  w.totals = p;
  w.chunk_free = p + 64;
  w.free_list = w.holes = w.chunk_free + (c + 63) / 64 * 64;
  w.movers = w.fork_count = w.free_list + c * kPagesChunk;
  w.rank = w.movers + c * kPagesChunk;
  return w;
}

}  // namespace mla
