// cache_window_bf16.cu -- attention over a paged cache of bf16 pages with a window (cache_attend.cuh).
#include "cache_attend.cuh"

namespace pisa {

cudaError_t launch_cache_window_bf16(const CacheAttendLaunch& L, cudaStream_t s) {
  return launch_attend_k<PISA_CACHE_BF16, kWindow>(L, s);
}

}  // namespace pisa
