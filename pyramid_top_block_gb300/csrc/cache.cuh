// cache.cuh -- the paged KV cache: page layout, its 4-bit format and the launch
// descriptions shared by the append, attention and read kernels.
//
// A page holds `page_size` = 16 .. 256 tokens of every KV head, head-major, in records of
// U = min(page_size, 64) tokens: one record is one contiguous run of bytes holding K and V
// of U tokens of one head, so a leaf block (64 tokens) is 64 / U records and a kernel's
// loads are contiguous for any number of heads.
//   bf16 record : K [U, 64], V [U, 64] bf16                           (256 U bytes)
//   e2m1 record : K codes [U, 32], K scales [U, 4], V codes [U, 32],
//                 V scales [U, 4] bytes                                (72 U bytes)
// A code byte holds dims 2 i (low nibble) and 2 i + 1 as e2m1; a scale byte is the e4m3
// factor of 16 dims.  The value is code * scale * 2^exp with one exponent per cache for K
// and one for V.  code * scale has six significant bits, so it is exact in fp16 and bf16.
#pragma once

#include <atomic>

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "api.cuh"
#include "scores.cuh"

namespace pisa {

constexpr int kCacheMaxT = 16;      // queries of one sequence in an attention call
constexpr int kCacheMaxSel = 64;    // blocks a query may list

struct CacheDev {
  unsigned char* pages;
  const int32_t* table;
  long long page_stride;
  int B, Hkv, n_pages, max_pages;
  int page_shift;  // log2 of the page size
  int rec_shift;   // log2 of U
  int kind;
  int k_exp, v_exp;
};

constexpr int kRowBf16 = 256, kRowE2m1 = 72;  // bytes of one token's K and V of one head

// Byte offset of the record holding position p (of a sequence whose page there is `page`).
__host__ __device__ __forceinline__ long long cache_record(const CacheDev& c, int row_bytes, long long page, int kv,
                                                           long long p) {
  const int parts = c.page_shift - c.rec_shift;  // log2 of the records of a page and head
  const int rec = (int)(p & ((1 << c.page_shift) - 1)) >> c.rec_shift;
  return page * c.page_stride + ((long long)((kv << parts) + rec) << c.rec_shift) * row_bytes;
}

__device__ __forceinline__ float exp2i(int e) {  // 2^e, -126 <= e <= 127
  return __int_as_float((e + 127) << 23);
}

// Eight e2m1 codes of a word as four fp16 pairs (dims 2 i and 2 i + 1 of byte i); exact.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&d)[4]) {
  asm("{ .reg .b8 a, b, c, e;\n mov.b32 {a, b, c, e}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, e; }"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(w));
}

// Two e4m3 bytes (the low 16 bits) as an fp16 pair; exact.
__device__ __forceinline__ uint32_t e4m3x2(uint32_t v) {
  uint32_t d;
  asm("{ .reg .b16 a, b;\n mov.b32 {a, b}, %1;\n cvt.rn.f16x2.e4m3x2 %0, a; }" : "=r"(d) : "r"(v));
  return d;
}

__device__ __forceinline__ uint32_t hmul2u(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Rows of 64 bf16 of a [B, T, H, 64] tensor; strides in elements.
struct RowsDev {
  __nv_bfloat16* data;
  long long sb, st, sh;
};

struct CacheAppendLaunch {
  CacheDev cache;
  RowsDev q, k, v, q_out, k_out;  // q, q_out and k_out may be absent (data == nullptr)
  int T, Hq;
  const int32_t* start;
  const int32_t* counts;  // may be nullptr: T of every sequence
  const float* rotary;    // [n_rot, rot]: cosines, then sines
  long long n_rot;
  int rot, interleaved;
  const int32_t* positions;  // [n_axes, B, T], or nullptr: a token turns by its position in the cache
  int n_axes;
  unsigned long long axis_of;  // the axis of pair i: bits 2 i and 2 i + 1
  int* status;  // may be nullptr
};

struct CacheReadLaunch {
  CacheDev cache;
  RowsDev k_out, v_out;  // either may be absent
  int T;
  const int32_t* start;
  const int32_t* counts;
  int* status;
};

struct CacheAttendLaunch {
  CacheDev cache;
  RowsDev q;
  int T, Hq, G;
  const int32_t* lengths;
  const int32_t* idx;  // nullptr: every token
  int Ksel;
  void* out;
  int out_f32;
  int* status;
  float* part;  // partial results (see cache_attend.cuh)
  ScoreDev score;  // (of the scored forms only)
};

// The launch is programmatic: a kernel may start while the one before it in the stream ends,
// and touches memory only after this.  Its loads are plain ones: a read-only load (ld.global.nc)
// promises that nothing writes the memory while the kernel lives, which begins before the one before
// has ended, and the compiler may move it ahead of the wait.
__device__ __forceinline__ void after_the_one_before() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launches a kernel that may start while the one before it in the stream ends.
template <auto kernel, typename... Args>
static cudaError_t launch_early(dim3 grid, int threads, int smem, cudaStream_t s, Args... args) {
  if (smem > 48 * 1024) {
    // the attribute belongs to the device: set once on each of the first 64 (on others at every call)
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (!(done.load(std::memory_order_acquire) & bit)) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      done.fetch_or(bit, std::memory_order_release);
    }
  }
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t launch_cache_append(const CacheAppendLaunch& L, cudaStream_t s);
cudaError_t launch_cache_read(const CacheReadLaunch& L, cudaStream_t s);
cudaError_t launch_cache_attend_bf16(const CacheAttendLaunch& L, cudaStream_t s);
cudaError_t launch_cache_attend_e2m1(const CacheAttendLaunch& L, cudaStream_t s);
cudaError_t launch_cache_window_bf16(const CacheAttendLaunch& L, cudaStream_t s);
cudaError_t launch_cache_window_e2m1(const CacheAttendLaunch& L, cudaStream_t s);
cudaError_t launch_cache_bias_bf16(const CacheAttendLaunch& L, cudaStream_t s);
cudaError_t launch_cache_bias_e2m1(const CacheAttendLaunch& L, cudaStream_t s);
cudaError_t launch_cache_cap_bf16(const CacheAttendLaunch& L, cudaStream_t s);
cudaError_t launch_cache_cap_e2m1(const CacheAttendLaunch& L, cudaStream_t s);
size_t cache_part_bytes();

}  // namespace pisa
