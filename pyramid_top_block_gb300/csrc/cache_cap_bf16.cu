// cache_cap_bf16.cu -- attention over a paged cache of bf16 pages with capped scores (cache_attend.cuh).
#include "cache_attend.cuh"

namespace pisa {

cudaError_t launch_cache_cap_bf16(const CacheAttendLaunch& L, cudaStream_t s) {
  return launch_attend_k<PISA_CACHE_BF16, kCapped>(L, s);
}

}  // namespace pisa
