// pool.cuh -- pages that sequences share: launch descriptions of the fork, reserve and compact kernels.
#pragma once

#include "cache.cuh"

namespace pisa {

struct PoolDev {
  unsigned char* pages;
  int32_t* table;  // [B, max_pages]
  int32_t* refs;   // [n_pages]: table entries that hold the page
  long long page_stride, page_bytes;
  int B, n_pages, max_pages;
  int page_shift;
};

struct PoolForkLaunch {
  PoolDev pool;
  const int32_t* parents;
  int32_t* lengths;
  int* status;  // may be nullptr
};

// The scratch of a reserve or a compaction: lists of whole numbers in the caller's workspace.
struct PoolScratch {
  int32_t* list_a;  // [n_pages]  reserve: fresh pages by rank;       compact: pages to move by rank
  int32_t* list_b;  // [n_pages]  reserve: the pages they replace, or -1;  compact: where they go
  int32_t* list_c;  // [n_pages]  compact: a page's new number
  int32_t* per_seq;  // [3 B]  reserve: rank of a sequence's first fresh page (or -1); copies (from, to)
  int32_t* counts;   // [2]  compact: pages in use, pages to move
};

struct PoolReserveLaunch {
  PoolDev pool;
  PoolScratch ws;
  const int32_t* lengths;
  const int32_t* counts;  // may be nullptr: T of every sequence
  int32_t* granted;
  int T;
  int* status;
};

struct PoolCompactLaunch {
  PoolDev pool;
  PoolScratch ws;
  int32_t* used;
};

constexpr int kForkMaxB = 32768;  // sequences of a fork: a column of the table lies in one CTA's shared memory

cudaError_t launch_pool_fork(const PoolForkLaunch& L, cudaStream_t s);
cudaError_t launch_pool_reserve(const PoolReserveLaunch& L, cudaStream_t s);
cudaError_t launch_pool_compact(const PoolCompactLaunch& L, cudaStream_t s);

}  // namespace pisa
