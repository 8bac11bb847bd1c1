// pool.cu -- pages that sequences share: forking and freeing sequences, reserving pages (a shared page
// that is about to be written is copied), and moving the pages in use to the front of the pool.
//
// All numbers are whole and every order is fixed (pages by their number, sequences by theirs, a sequence's
// entries by position), so that a call gives the same table however it is scheduled; atomics only count.
//
// What bounds it: copying pages (the memory, read and write: 356 MB moved in 54.4 us = 6.55 TB/s); planning is a few
// dependent loads and barriers.  Fork 1.6 us (16 sequences of 64 pages) to 7.3 (64 of 8192), reserve 5.6 (1200 pages)
// to 10.6 (530000), planning a compaction 5.3 to 33.7.
#include <climits>

#include <cooperative_groups.h>

#include "pool.cuh"

namespace pisa {

namespace cg = cooperative_groups;

// One cluster plans: it can hand sums around without another launch.  For small pools it has one CTA, whose barriers
// take less (plans_alone).
constexpr int kPlanCtas = 8;
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ bool is_page(const PoolDev& p, int x) { return x >= 0 && x < p.n_pages; }

// ------------------------------------------------------------------------------------------------- fork

// Row b becomes row parents[b] of the table as it was.  A CTA holds `cols` columns of all rows in shared
// memory, so that rows can be taken from one another in place; one more CTA does the same with the lengths.
__global__ void __launch_bounds__(512) pool_fork_kernel(PoolForkLaunch a, int cols_shift) {
  extern __shared__ int32_t fork_smem[];
  after_the_one_before();
  const PoolDev& p = a.pool;
  const int cols = 1 << cols_shift, c0 = blockIdx.x << cols_shift;
  if (c0 >= p.max_pages) {
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) fork_smem[b] = a.lengths[b];
    __syncthreads();
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
      const int q = a.parents[b];
      if (q >= p.B) set_status(a.status, PISA_ERR_DEVICE_BOUNDS);
      if (q < p.B && q != b) a.lengths[b] = q < 0 ? 0 : fork_smem[q];
    }
    return;
  }
  const int n = p.B << cols_shift;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int b = i >> cols_shift, c = c0 + (i & (cols - 1));
    fork_smem[i] = c < p.max_pages ? p.table[(long long)b * p.max_pages + c] : -1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int b = i >> cols_shift, x = i & (cols - 1), c = c0 + x;
    if (c >= p.max_pages) continue;
    const int q = a.parents[b];
    if (q >= p.B || q == b) continue;
    const int was = fork_smem[i], is = q < 0 ? -1 : fork_smem[(q << cols_shift) + x];
    if (is == was) continue;
    p.table[(long long)b * p.max_pages + c] = is;
    if (is_page(p, was)) atomicAdd(p.refs + was, -1);
    if (is_page(p, is)) atomicAdd(p.refs + is, 1);
  }
}

cudaError_t launch_pool_fork(const PoolForkLaunch& L, cudaStream_t s) {
  // Columns of a CTA: up to 32 (a row's 128 bytes), as few as spread the table over 64 CTAs (256 sequences of 28
  // pages: one CTA took 19.0 us), and no more than fit 96 KB.
  int shift = 0;
  while (shift < 5 && (L.pool.max_pages >> shift) > 64) ++shift;
  while (shift > 0 && ((long long)L.pool.B << shift) > 24576) --shift;
  const unsigned grid = (unsigned)((L.pool.max_pages + (1 << shift) - 1) >> shift) + 1;
  // (the attribute is set at the largest size, once on each device)
  const int need = L.pool.B << shift;
  if (need * 4 <= 48 * 1024) return launch_early<pool_fork_kernel>(grid, 512, need * 4, s, L, shift);
  return launch_early<pool_fork_kernel>(grid, 512, kForkMaxB * 4, s, L, shift);
}

// ------------------------------------------------------------------------------------- sums over the cluster

// (64 bits: what all sequences of a call ask for may be more than 2^31 pages)
struct PlanShared {
  long long warp[32];
  long long sum[2];  // of this CTA: read by the others
  int count[32];
};

// Sum of x over the threads before this one; total: over all.
__device__ __forceinline__ long long scan_block(long long x, PlanShared& sh, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(kFull, inc, d);
    if (lane >= d) inc += y;
  }
  __syncthreads();
  if (lane == 31) sh.warp[warp] = inc;
  __syncthreads();
  const long long w = sh.warp[lane];
  long long winc = w;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(kFull, winc, d);
    if (lane >= d) winc += y;
  }
  total = __shfl_sync(kFull, winc, 31);
  return inc - x + __shfl_sync(kFull, winc - w, warp);
}

// Pages of a slice whose reference count is zero (FREE) or not, counted.
template <bool FREE>
__device__ __forceinline__ long long count_pages(const PoolDev& p, int from, int to, PlanShared& sh) {
  int n = 0;
#pragma unroll 8
  for (int i = from + threadIdx.x; i < to; i += kPlanThreads) n += (p.refs[i] == 0) == FREE;
  long long total;
  scan_block(n, sh, total);
  return total;
}

template <int CTAS>
__device__ __forceinline__ void sync_cluster(cg::cluster_group& cluster) {
  if constexpr (CTAS == 1)
    __syncthreads();
  else
    cluster.sync();
}

// Calls f(page, held, rank) for the pages of a slice, rank being the number of free pages (FREE) or of held ones before
// it, `at` before the slice; ends when `at` has reached `most`.  8192 pages a turn, a warp 256 consecutive ones.
template <bool FREE, typename F>
__device__ __forceinline__ void each_page(const PoolDev& p, int from, int to, long long at, long long most,
                                          PlanShared& sh, F f) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int c = from; c < to && at < most; c += 8 * kPlanThreads) {
    const int first = c + 256 * warp + lane;
    int ref[8];
    unsigned mask[8];
    int n = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) ref[j] = first + 32 * j < to ? p.refs[first + 32 * j] : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      mask[j] = __ballot_sync(kFull, first + 32 * j < to && (ref[j] == 0) == FREE);
      n += __popc(mask[j]);
    }
    __syncthreads();
    if (lane == 0) sh.count[warp] = n;
    __syncthreads();
    const int other = sh.count[lane], total = __reduce_add_sync(kFull, other);
    long long before = at + __reduce_add_sync(kFull, lane < warp ? other : 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (first + 32 * j < to) f(first + 32 * j, ref[j] != 0, before + __popc(mask[j] & ((1u << lane) - 1u)));
      before += __popc(mask[j]);
    }
    at += total;
  }
}

// One number of each CTA of the cluster: the sum of those before this one, and of all.
template <int CTAS>
__device__ __forceinline__ long long before_in_cluster(cg::cluster_group& cluster, long long* mine, int rank,
                                                       long long& total) {
  long long before = 0;
  total = 0;
  for (int r = 0; r < CTAS; ++r) {
    const long long x = CTAS == 1 ? *mine : *cluster.map_shared_rank(mine, r);
    if (r < rank) before += x;
    total += x;
  }
  return before;
}

// ----------------------------------------------------------------------------------------------- reserve

// Tokens that sequence b gets, the table entries that they are written to, and whether they fit at all.
struct Wanted {
  int n, count, first, stop;
  bool fits;
};
__device__ __forceinline__ Wanted wanted(const PoolReserveLaunch& a, int b) {
  Wanted w;
  w.n = a.lengths[b];
  w.count = a.counts ? min(max(a.counts[b], 0), a.T) : a.T;
  const long long end = (long long)w.n + w.count;
  w.fits = w.n >= 0 && end <= (long long)a.pool.max_pages << a.pool.page_shift;
  w.first = w.fits ? w.n >> a.pool.page_shift : 0;
  w.stop = w.fits && w.count ? (int)((end + (1 << a.pool.page_shift) - 1) >> a.pool.page_shift) : w.first;
  return w;
}

// Eight lanes take a sequence, an entry each at a time: few entries at a decoding step, many at a prompt.
constexpr int kSeqLanes = 8;

// A missing or shared page is replaced by a fresh one; `old` is the page to copy and let go, or -1.
__device__ __forceinline__ bool takes_fresh(const PoolDev& p, int entry, int& old) {
  old = -1;
  if (!is_page(p, entry)) return true;
  if (p.refs[entry] <= 1) return false;
  old = entry;
  return true;
}

// Plans a reserve in one cluster:
//   1. each CTA counts the free pages of its eighth of the pool, and what its eighth of the sequences need;
//   2. from the others' sums it knows the ranks of its free pages and of its sequences' needs; a sequence is
//      served if it needs nothing, or all up to and with it need no more than there are;
//   3. it lists its free pages by rank, as far as they are needed;
//   4. its sequences take the pages of their ranks; 5. the pages that were replaced lose a reference (only now:
//      up to here whether a page is shared is read).
template <int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kPlanThreads) pool_reserve_kernel(PoolReserveLaunch a) {
  __shared__ PlanShared sh;
  after_the_one_before();
  cg::cluster_group cluster = cg::this_cluster();
  const PoolDev& p = a.pool;
  const int rank = (int)cluster.block_rank(), tid = threadIdx.x;
  const int lane = tid % kSeqLanes, group = tid / kSeqLanes;
  constexpr int kGroups = kPlanThreads / kSeqLanes;
  const unsigned lanes = 0xffu << (tid & 24);  // the group's lanes of its warp
  const int slice = (p.n_pages + CTAS - 1) / CTAS, part = (p.B + CTAS - 1) / CTAS;
  const int p0 = min(rank * slice, p.n_pages), p1 = min(p0 + slice, p.n_pages);
  const int b0 = min(rank * part, p.B), b1 = min(b0 + part, p.B);
  int32_t* at_of = a.ws.per_seq;
  int32_t* copy_from = a.ws.per_seq + p.B;
  int32_t* copy_to = a.ws.per_seq + 2LL * p.B;
  // 1.
  for (int b = b0 + group; b < b1; b += kGroups) {
    const Wanted w = wanted(a, b);
    const int32_t* row = p.table + (long long)b * p.max_pages;
    int need = 0, old;
    for (int e = w.first + lane; e < w.stop; e += kSeqLanes) need += takes_fresh(p, row[e], old);
#pragma unroll
    for (int d = 1; d < kSeqLanes; d <<= 1) need += __shfl_xor_sync(lanes, need, d);
    if (lane == 0) {
      at_of[b] = need;
      if (!w.fits) set_status(a.status, PISA_ERR_DEVICE_BOUNDS);
    }
  }
  const long long mine = count_pages<true>(p, p0, p1, sh);  // (its barriers order at_of for the block, too)
  long long needs = 0;
  for (int b = b0 + tid; b < b1; b += kPlanThreads) needs += at_of[b];
  long long need_here;
  scan_block(needs, sh, need_here);
  if (tid == 0) {
    sh.sum[0] = mine;
    sh.sum[1] = need_here;
  }
  sync_cluster<CTAS>(cluster);
  // 2.
  long long free_all, need_all;
  const long long at_page = before_in_cluster<CTAS>(cluster, &sh.sum[0], rank, free_all);
  long long at_need = before_in_cluster<CTAS>(cluster, &sh.sum[1], rank, need_all);
  for (int c = b0; c < b1; c += kPlanThreads) {
    const int b = c + tid, need = b < b1 ? at_of[b] : 0;
    long long total;
    const long long begin = at_need + scan_block(need, sh, total);
    if (b < b1) {
      const Wanted w = wanted(a, b);
      const bool served = w.fits && (need == 0 || begin + need <= free_all);
      at_of[b] = served ? (int)min(begin, (long long)p.n_pages) : -1;
      a.granted[b] = served ? w.count : 0;
      copy_to[b] = -1;
    }
    at_need += total;
  }
  // 3.
  const int list = (int)min(free_all, need_all);
  each_page<true>(p, p0, p1, at_page, list, sh, [&](int page, bool held, long long r) {
    if (held || r >= list) return;
    a.ws.list_a[r] = page;
    a.ws.list_b[r] = -1;
  });
  sync_cluster<CTAS>(cluster);  // (and what was written before it is there for all of the cluster)
  // 4.
  for (int b = b0 + group; b < b1; b += kGroups) {
    int r = at_of[b];
    if (r < 0) continue;
    const Wanted w = wanted(a, b);
    int32_t* row = p.table + (long long)b * p.max_pages;
    for (int c = w.first; c < w.stop; c += kSeqLanes) {
      const int e = c + lane;
      int old = -1;
      const bool take = e < w.stop && takes_fresh(p, row[e], old);
      const unsigned all = __ballot_sync(lanes, take) >> (tid & 24);
      if (take) {
        const int x = r + __popc(all & ((1u << lane) - 1u));
        const int page = a.ws.list_a[x];
        row[e] = page;
        p.refs[page] = 1;
        if (old >= 0) a.ws.list_b[x] = old;
        if (old >= 0 && e == w.first && (w.n & ((1 << p.page_shift) - 1))) {
          copy_from[b] = old;
          copy_to[b] = page;
        }
      }
      r += __popc(all);
    }
  }
  sync_cluster<CTAS>(cluster);
  // 5.
  for (int x = rank * kPlanThreads + tid; x < list; x += CTAS * kPlanThreads) {
    const int old = a.ws.list_b[x];
    if (old >= 0) atomicAdd(p.refs + old, -1);
  }
}

// Copies pages, 16 bytes a load, four of a thread at once: 16 KB a CTA and turn.
constexpr int kCopyThreads = 256, kCopyBytes = kCopyThreads * 16 * 4;

__device__ __forceinline__ void copy_piece(const PoolDev& p, int from, int to, long long at) {
  const unsigned char* src = p.pages + from * p.page_stride + at;
  unsigned char* dst = p.pages + to * p.page_stride + at;
  const long long left = p.page_bytes - at;
  uint4 x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long o = (i * kCopyThreads + threadIdx.x) * 16;
    if (o < left) x[i] = *reinterpret_cast<const uint4*>(src + o);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long o = (i * kCopyThreads + threadIdx.x) * 16;
    if (o < left) *reinterpret_cast<uint4*>(dst + o) = x[i];
  }
}

__global__ void __launch_bounds__(kCopyThreads) pool_copy_kernel(PoolDev p, const int32_t* from, const int32_t* to,
                                                                 int pieces) {
  after_the_one_before();
  const long long jobs = (long long)p.B * pieces;
  for (long long j = blockIdx.x; j < jobs; j += gridDim.x) {
    const int b = (int)(j / pieces);
    const int dst = to[b];
    if (dst >= 0) copy_piece(p, from[b], dst, (j - (long long)b * pieces) * kCopyBytes);
  }
}

// Whether one CTA plans.  One CTA / a cluster of eight, us: reserve of 16 sequences, 1200 pages 5.7 / 8.6, 64 and 2300
// 6.4 / 8.7, 256 and 8000 8.9 / 8.9; compact 5.0 / 7.1, 5.8 / 7.3, 9.9 / 7.3.
static bool plans_alone(const PoolDev& p) { return p.n_pages <= 4096 && p.B <= 256; }

static unsigned copy_grid(long long jobs) { return (unsigned)(jobs < 152 * 8 ? jobs : 152 * 8); }

cudaError_t launch_pool_reserve(const PoolReserveLaunch& L, cudaStream_t s) {
  cudaError_t e = plans_alone(L.pool) ? launch_early<pool_reserve_kernel<1>>(1, kPlanThreads, 0, s, L)
                                      : launch_early<pool_reserve_kernel<kPlanCtas>>(kPlanCtas, kPlanThreads, 0, s, L);
  if (e != cudaSuccess) return e;
  const int pieces = (int)((L.pool.page_bytes + kCopyBytes - 1) / kCopyBytes);
  return launch_early<pool_copy_kernel>(copy_grid((long long)L.pool.B * pieces), kCopyThreads, 0, s, L.pool,
                                        (const int32_t*)(L.ws.per_seq + L.pool.B),
                                        (const int32_t*)(L.ws.per_seq + 2LL * L.pool.B), pieces);
}

// ----------------------------------------------------------------------------------------------- compact

// Plans a compaction in one cluster.  U pages are in use; the i-th of those at U and behind moves to the i-th
// free place before U.  With h(p) the pages in use before p: a free place p < U has rank p - h(p), a page p >= U
// in use has rank h(p) - h(U).
template <int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kPlanThreads) pool_compact_kernel(PoolCompactLaunch a) {
  __shared__ PlanShared sh;
  after_the_one_before();
  cg::cluster_group cluster = cg::this_cluster();
  const PoolDev& p = a.pool;
  const int rank = (int)cluster.block_rank(), tid = threadIdx.x;
  const int slice = (p.n_pages + CTAS - 1) / CTAS;
  const int p0 = min(rank * slice, p.n_pages), p1 = min(p0 + slice, p.n_pages);
  const long long mine = count_pages<false>(p, p0, p1, sh);
  if (tid == 0) sh.sum[0] = mine;
  sync_cluster<CTAS>(cluster);
  long long used_all;
  const int h = (int)before_in_cluster<CTAS>(cluster, &sh.sum[0], rank, used_all);
  const int used = (int)used_all;
  const long long below = count_pages<false>(p, p0, max(p0, min(p1, used)), sh);
  if (tid == 0) sh.sum[1] = below;
  sync_cluster<CTAS>(cluster);
  long long below_all;
  before_in_cluster<CTAS>(cluster, &sh.sum[1], rank, below_all);
  const int h_used = (int)below_all;
  const int moves = used - h_used;
  each_page<false>(p, p0, p1, h, LLONG_MAX, sh, [&](int page, bool held, long long before) {
    if (page < used) {
      if (!held) a.ws.list_b[page - before] = page;
    } else {
      if (held) a.ws.list_a[before - h_used] = page;
      a.ws.list_c[page] = page;
    }
  });
  if (rank == 0 && tid == 0) {
    a.ws.counts[0] = used;
    a.ws.counts[1] = moves;
    *a.used = used;
  }
  sync_cluster<CTAS>(cluster);
  for (int x = rank * kPlanThreads + tid; x < moves; x += CTAS * kPlanThreads) {
    const int from = a.ws.list_a[x], to = a.ws.list_b[x];
    a.ws.list_c[from] = to;
    p.refs[to] = p.refs[from];
    p.refs[from] = 0;
  }
  sync_cluster<CTAS>(cluster);  // (no CTA leaves while another may still read its sums)
}

// Moves the pages and renames them in the table.  (Pages come from behind U and go before it: no order among them.)
__global__ void __launch_bounds__(kCopyThreads) pool_move_kernel(PoolCompactLaunch a, int pieces) {
  after_the_one_before();
  const PoolDev& p = a.pool;
  const int used = a.ws.counts[0];
  const long long jobs = (long long)a.ws.counts[1] * pieces;
  const long long entries = (long long)p.B * p.max_pages;
  for (long long i = (long long)blockIdx.x * kCopyThreads + threadIdx.x; i < entries;
       i += (long long)gridDim.x * kCopyThreads) {
    const int x = p.table[i];
    if (x >= used && x < p.n_pages) {
      const int y = a.ws.list_c[x];
      if (y != x) p.table[i] = y;
    }
  }
  for (long long j = blockIdx.x; j < jobs; j += gridDim.x) {
    const int x = (int)(j / pieces);
    copy_piece(p, a.ws.list_a[x], a.ws.list_b[x], (j - (long long)x * pieces) * kCopyBytes);
  }
}

cudaError_t launch_pool_compact(const PoolCompactLaunch& L, cudaStream_t s) {
  cudaError_t e = plans_alone(L.pool) ? launch_early<pool_compact_kernel<1>>(1, kPlanThreads, 0, s, L)
                                      : launch_early<pool_compact_kernel<kPlanCtas>>(kPlanCtas, kPlanThreads, 0, s, L);
  if (e != cudaSuccess) return e;
  const int pieces = (int)((L.pool.page_bytes + kCopyBytes - 1) / kCopyBytes);
  const long long jobs = (long long)(L.pool.n_pages / 2) * pieces;  // at most half of the pages move
  const long long entries = ((long long)L.pool.B * L.pool.max_pages + kCopyThreads - 1) / kCopyThreads;
  return launch_early<pool_move_kernel>(copy_grid(jobs > entries ? jobs : entries), kCopyThreads, 0, s, L, pieces);
}

}  // namespace pisa
