// cache_attend_e2m1.cu -- attention over a paged cache of 4-bit pages (cache_attend.cuh).
#include "cache_attend.cuh"

namespace pisa {

cudaError_t launch_cache_attend_e2m1(const CacheAttendLaunch& L, cudaStream_t s) {
  return launch_attend_k<PISA_CACHE_E2M1>(L, s);
}

}  // namespace pisa
