// cache_attend_bf16.cu -- attention over a paged cache of bf16 pages (cache_attend.cuh).
#include "cache_attend.cuh"

namespace pisa {

size_t cache_part_bytes() { return part_bytes(); }

cudaError_t launch_cache_attend_bf16(const CacheAttendLaunch& L, cudaStream_t s) {
  return launch_attend_k<PISA_CACHE_BF16>(L, s);
}

}  // namespace pisa
