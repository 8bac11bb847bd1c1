// cache_prompt.cu -- attention of a prompt's tokens over the paged cache, a row (token and head) a thread.
#include "cache_prompt.cuh"

#include <climits>

namespace pisa {

constexpr int kPromptRows = 128, kPromptKeys = 32;

template <int KIND>
__global__ void __launch_bounds__(kPromptRows) cache_prompt_kernel(CachePromptLaunch a) {
  __shared__ float sk[kPromptKeys][kD], sv[kPromptKeys][kD];
  __shared__ int bad[kPromptKeys];
  __shared__ int range[2];
  after_the_one_before();
  const int kv = blockIdx.y, b = blockIdx.z, count = prompt_count(a, b);
  const int r = blockIdx.x * kPromptRows + threadIdx.x, t = r / a.G, head = kv * a.G + r % a.G;
  const bool there = t < count;
  bool over = false;
  Span s = {0, 0, 0};
  if (there) s = span_of(a, b, t, count, over);
  if (over) set_status(a.status, PISA_ERR_DEVICE_BOUNDS);
  if (threadIdx.x == 0) {
    range[0] = INT_MAX;
    range[1] = 0;
  }
  __syncthreads();
  if (s.lo < s.hi) {
    atomicMin(&range[0], s.lo);
    atomicMax(&range[1], s.hi);
  }
  float q[kD], o[kD];
#pragma unroll
  for (int i = 0; i < kD; ++i) q[i] = o[i] = 0.f;
  if (there) {
    const uint4* p = reinterpret_cast<const uint4*>(a.q.data + b * a.q.sb + (long long)t * a.q.st + head * a.q.sh);
#pragma unroll
    for (int i = 0; i < 8; ++i) unpack8(p[i], q + 8 * i);
  }
  const float slope = a.score.slopes && there ? a.score.slopes[head] : 0.f;
  float m = -INFINITY, l = 0.f;
  __syncthreads();
  const int end = range[1];
  for (int k0 = range[0]; k0 < end; k0 += kPromptKeys) {
    __syncthreads();
    {  // four threads a token, 16 dims each
      const int key = threadIdx.x >> 2, c = threadIdx.x & 3, p = k0 + key;
      int page = -1;
      if (p < end) page = a.cache.table[(long long)b * a.cache.max_pages + (p >> a.cache.page_shift)];
      const bool ok = page >= 0 && page < a.cache.n_pages;
      if (c == 0) bad[key] = p < end && !ok;
      const int U = 1 << a.cache.rec_shift, u = p & (U - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float* dst = (h ? sv : sk)[key] + 16 * c;
        if (!ok) {
          for (int i = 0; i < 16; ++i) dst[i] = 0.f;
        } else if (KIND == PISA_CACHE_BF16) {
          const uint4* x = reinterpret_cast<const uint4*>(a.cache.pages + cache_record(a.cache, kRowBf16, page, kv, p) +
                                                          h * U * 128 + u * 128 + 32 * c);
          unpack8(x[0], dst);
          unpack8(x[1], dst + 8);
        } else {
          const unsigned char* rec = a.cache.pages + cache_record(a.cache, kRowE2m1, page, kv, p) + h * 36 * U;
          const uint32_t f = e4m3x2(rec[32 * U + 4 * u + c]);
          const float scale =
              __low2float(*reinterpret_cast<const __half2*>(&f)) * exp2i(h ? a.cache.v_exp : a.cache.k_exp);
          for (int w = 0; w < 2; ++w) {
            uint32_t d[4];
            e2m1x8(*reinterpret_cast<const uint32_t*>(rec + 32 * u + 8 * c + 4 * w), d);
            for (int i = 0; i < 4; ++i) {
              const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&d[i]));
              dst[8 * w + 2 * i] = v.x * scale;
              dst[8 * w + 2 * i + 1] = v.y * scale;
            }
          }
        }
      }
    }
    __syncthreads();
    for (int key = 0; key < kPromptKeys; ++key) {
      const int p = k0 + key;
      if (p < s.lo || p >= s.hi) continue;
      if (bad[key]) {
        l = __int_as_float(0x7fc00000);
        set_status(a.status, PISA_ERR_DEVICE_BOUNDS);
        continue;
      }
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < kD; ++i) x = fmaf(q[i], sk[key][i], x);
      x *= kScale;
      if (a.score.cap > 0.f) x = a.score.cap * tanhf(x * a.score.inv_cap);
      x -= slope * fabsf((float)(s.pos - p));
      if (x == -INFINITY) continue;
      const float n = fmaxf(m, x), f = expf(m - n), w = expf(x - n);
      l = l * f + w;
      m = n;
#pragma unroll
      for (int i = 0; i < kD; ++i) o[i] = fmaf(w, sv[key][i], o[i] * f);
    }
  }
  if (!there) return;
  const float f = l == 0.f ? 0.f : 1.f / l;
  __nv_bfloat16* dst = a.out + (((long long)b * a.T + t) * a.Hq + head) * kD;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = l == 0.f ? 0.f : o[8 * i + k] * f;
    *reinterpret_cast<uint4*>(dst + 8 * i) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                        pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

cudaError_t launch_cache_prompt(const CachePromptLaunch& L, cudaStream_t s) {
  const dim3 grid((unsigned)(((long long)L.T * L.G + kPromptRows - 1) / kPromptRows), L.cache.Hkv, L.cache.B);
  if (L.cache.kind == PISA_CACHE_BF16) return launch_early<cache_prompt_kernel<PISA_CACHE_BF16>>(grid, kPromptRows, 0, s, L);
  return launch_early<cache_prompt_kernel<PISA_CACHE_E2M1>>(grid, kPromptRows, 0, s, L);
}

}  // namespace pisa
