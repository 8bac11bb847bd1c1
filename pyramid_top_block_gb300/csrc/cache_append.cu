// cache_append.cu -- new queries and keys are rotated by their positions, keys and values go
// into the pages of a paged cache; and the way back, cached tokens as dense bf16 rows.
//
// Rotation of a pair (a, b) at a position with cosine c and sine s:
//   a' = a c - b s,  b' = b c + a s
// Eight lanes hold one row of 64 (16 bytes each), a warp four rows.  In the split-halves
// order the other member of a pair is rot/2 dims away, which is a whole number of lanes, so
// it comes by shuffle; in the interleaved order it is the neighbouring element.
//
// Both kernels only move rows: the bound is the bytes of the rows in and out.
#include "cache.cuh"

namespace pisa {

constexpr int kAppWarps = 8;
constexpr int kAppIter = 4;  // groups of four rows a warp takes at most, their loads issued together

// Two rotated elements x c + p s (p the pair's other member, s signed), as the bf16 values
// that the 64-bit sum rounds to (by way of 32 bits).  In 32 bits the sum is off by at most
// (|p s| + |r|) 2^-24 (and 2^-149 among the subnormal); where every value within twice that
// rounds to the same bf16 that is the answer, else the sum is taken in 64 bits (both
// products are exact there).  So a key has the same bits however it was appended, which
// matters where it is quantised next.
__device__ __forceinline__ uint32_t rotate2(float x0, float p0, float c0, float s0, float x1, float p1, float c1,
                                            float s1) {
  const float m0 = p0 * s0, m1 = p1 * s1;
  const float r0 = fmaf(x0, c0, m0), r1 = fmaf(x1, c1, m1);
  const float e0 = fmaf(fabsf(m0) + fabsf(r0), 0x1p-23f, 0x1p-147f);
  const float e1 = fmaf(fabsf(m1) + fabsf(r1), 0x1p-23f, 0x1p-147f);
  uint32_t lo = pack_bf16x2(r0 - e0, r1 - e1);
  if (lo != pack_bf16x2(r0 + e0, r1 + e1)) {
    const double d0 = (double)x0 * (double)c0 + (double)p0 * (double)s0;
    const double d1 = (double)x1 * (double)c1 + (double)p1 * (double)s1;
    lo = pack_bf16x2((float)d0, (float)d1);
  }
  return lo;
}

// The 4-bit form of a row: this lane's 8 of 64 values (bf16 pairs w) and, with the
// neighbouring lane's, the scale of their 16.  Steps, each exact or rounded once:
//   top = largest |x| (compared as integers, so that an infinity or a NaN is the largest)
//   scale = e4m3(top 2^-exp / 6), to nearest even, at most 448; code = e2m1(x 2^-exp / scale)
// x is a bf16 (8 bits) and a border between two codes times the scale has at most 7, so a
// quotient that is not on a border is at least 2^-10 from it (borders lie in [1/4, 5], and
// so does any quotient near one).  x times the rounded reciprocal is off by 2^-21 there at
// most; rounding it to a multiple of 2^-11 (by adding 1.5 * 2^12) puts the quotients that are
// on a border exactly there and moves no other one across, so the conversion's
// ties-to-even rule decides them.
__device__ __forceinline__ void quantise8(const uint32_t (&w)[4], int exp, uint32_t& codes, uint32_t& scale) {
  uint32_t t = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                        __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
  t = max(t & 0xffffu, t >> 16);
  t = max(t, __shfl_xor_sync(kFull, t, 1));
  const float down = exp2i(-exp);
  const float s = __fdiv_rn(__uint_as_float(t << 16) * down, 6.f);
  scale = __nv_cvt_float_to_fp8(s, __NV_SATFINITE, __NV_E4M3);
  const float sv = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)scale, __NV_E4M3)));
  const float inv = sv > 0.f ? __frcp_rn(sv) : 0.f;
  constexpr float kSnap = 6144.f;  // 1.5 * 2^12: sums near it are multiples of 2^-11
  codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = __uint_as_float(w[i] << 16) * down * inv, b = __uint_as_float(w[i] & 0xffff0000u) * down * inv;
    a = (a + kSnap) - kSnap;
    b = (b + kSnap) - kSnap;
    uint32_t c;
    asm("{ .reg .b8 x;\n cvt.rn.satfinite.e2m1x2.f32 x, %2, %1;\n cvt.u32.u8 %0, x; }" : "=r"(c) : "f"(a), "f"(b));
    codes |= c << (8 * i);
  }
  if (t >= 0x7f80u) {  // an infinity or a NaN among the 16: the block stands for NaNs
    scale = 0x7f;
    codes = 0;
  }
}

template <int KIND>
__global__ void __launch_bounds__(kAppWarps * 32) cache_append_kernel(CacheAppendLaunch a, int parts, int per) {
  const int lane = threadIdx.x & 31, sub = lane >> 3, c = lane & 7;
  const unsigned job = blockIdx.x * kAppWarps + (threadIdx.x >> 5);
  const unsigned tok = job / parts, part = job % parts;
  if (tok >= (unsigned)a.cache.B * a.T) return;
  const int b = tok / a.T, t = tok % a.T;
  const int Hkv = a.cache.Hkv, Hq = a.q.data ? a.Hq : 0;
  const int rows = Hq + 2 * Hkv, r0 = part * per * 4 + sub;
  const long long p = (long long)a.start[b] + t;
  const bool counted = a.counts == nullptr || t < a.counts[b];
  // the rows of this warp (their addresses do not depend on the position)
  uint4 x[kAppIter];
#pragma unroll
  for (int i = 0; i < kAppIter; ++i) {
    const int r = r0 + 4 * i;
    if (i < per && r < rows) {
      const RowsDev& src = r < Hq ? a.q : r < Hq + Hkv ? a.k : a.v;
      const int h = r < Hq ? r : r < Hq + Hkv ? r - Hq : r - Hq - Hkv;
      x[i] = *reinterpret_cast<const uint4*>(src.data + b * src.sb + t * src.st + h * src.sh + 8 * c);
    } else {
      x[i] = make_uint4(0, 0, 0, 0);
    }
  }
  if (!counted) return;
  const long long cap = (long long)a.cache.max_pages << a.cache.page_shift;
  bool ok = p >= 0 && p < cap && (a.rot == 0 || p < a.n_rot);
  int page = -1;
  if (ok) {
    page = a.cache.table[(long long)b * a.cache.max_pages + (p >> a.cache.page_shift)];
    ok = page >= 0 && page < a.cache.n_pages;
  }
  if (!ok) {  // the token is left out
    if (lane == 0) set_status(a.status, PISA_ERR_DEVICE_BOUNDS);
    return;
  }
  // this lane's cosines and signed sines, for pairs of elements (8 c + e, its partner)
  const int half = a.rot >> 4;  // lanes of one half of the rotated dims (split-halves order)
  const bool turned = c < 2 * half;
  float cs[8], sn[8];
  int from = lane;  // lane of the partner elements
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cs[e] = 1.f;
    sn[e] = 0.f;
  }
  if (turned) {
    const float* row = a.rotary + p * a.rot;
    if (a.interleaved) {
      const float4 u = *reinterpret_cast<const float4*>(row + 4 * c);
      const float4 v = *reinterpret_cast<const float4*>(row + (a.rot >> 1) + 4 * c);
      const float uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        cs[e] = uu[e >> 1];
        sn[e] = (e & 1) ? vv[e >> 1] : -vv[e >> 1];
      }
    } else {
      const bool low = c < half;
      from = low ? lane + half : lane - half;
      const float4* u = reinterpret_cast<const float4*>(row + 8 * (low ? c : c - half));
      const float4* v = reinterpret_cast<const float4*>(row + (a.rot >> 1) + 8 * (low ? c : c - half));
      const float4 u0 = u[0], u1 = u[1], v0 = v[0], v1 = v[1];
      const float uu[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
      const float vv[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        cs[e] = uu[e];
        sn[e] = low ? -vv[e] : vv[e];
      }
    }
  }
  const int U = 1 << a.cache.rec_shift, u = (int)(p & (U - 1));
#pragma unroll
  for (int i = 0; i < kAppIter; ++i) {
    if (i >= per) break;
    const int r = r0 + 4 * i;
    uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, o[4];
    if (a.interleaved) {
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = (w[k] >> 16) | (w[k] << 16);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = __shfl_sync(kFull, w[k], from);
    }
    const bool is_v = r >= Hq + Hkv;
    if (turned && !is_v) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = rotate2(__uint_as_float(w[k] << 16), __uint_as_float(o[k] << 16), cs[2 * k], sn[2 * k],
                       __uint_as_float(w[k] & 0xffff0000u), __uint_as_float(o[k] & 0xffff0000u), cs[2 * k + 1],
                       sn[2 * k + 1]);
    }
    const uint4 y = make_uint4(w[0], w[1], w[2], w[3]);
    if (r < Hq) {
      if (a.q_out.data)
        *reinterpret_cast<uint4*>(a.q_out.data + b * a.q_out.sb + t * a.q_out.st + r * a.q_out.sh + 8 * c) = y;
    } else if (r < Hq + Hkv && a.k_out.data) {
      *reinterpret_cast<uint4*>(a.k_out.data + b * a.k_out.sb + t * a.k_out.st + (r - Hq) * a.k_out.sh + 8 * c) = y;
    }
    const int kv = is_v ? r - Hq - Hkv : r - Hq;
    if (KIND == PISA_CACHE_BF16) {
      if (r >= Hq && r < rows) {
        unsigned char* rec = a.cache.pages + cache_record(a.cache, kRowBf16, page, kv, p) + (is_v ? U * 128 : 0);
        *reinterpret_cast<uint4*>(rec + u * 128 + 16 * c) = y;
      }
    } else if (__any_sync(kFull, r >= Hq && r < rows)) {
      uint32_t codes, scale;
      quantise8(w, is_v ? a.cache.v_exp : a.cache.k_exp, codes, scale);
      if (r >= Hq && r < rows) {
        unsigned char* rec = a.cache.pages + cache_record(a.cache, kRowE2m1, page, kv, p) + (is_v ? U * 36 : 0);
        *reinterpret_cast<uint32_t*>(rec + u * 32 + 4 * c) = codes;
        if (!(c & 1)) rec[U * 32 + u * 4 + (c >> 1)] = (unsigned char)scale;
      }
    }
  }
}

// One thread per 8 dims of one token's K and V of one head; tokens run fastest over groups of
// eight lanes, as they lie in a record.
template <int KIND>
__global__ void __launch_bounds__(256) cache_read_kernel(CacheReadLaunch a, int tok_groups) {
  const int lane = threadIdx.x & 31, c = lane & 7;
  const unsigned job = blockIdx.x * 8 + (threadIdx.x >> 5);  // (b, group of 4 tokens, kv), kv fastest
  const int Hkv = a.cache.Hkv;
  const unsigned kv = job % Hkv, bg = job / Hkv;
  const unsigned b = bg / tok_groups;
  const int t = (int)(bg % tok_groups) * 4 + (lane >> 3);
  if (b >= (unsigned)a.cache.B || t >= a.T) return;
  if (a.counts && t >= a.counts[b]) return;
  const long long p = (long long)a.start[b] + t;
  const long long cap = (long long)a.cache.max_pages << a.cache.page_shift;
  int page = -1;
  if (p >= 0 && p < cap) page = a.cache.table[(long long)b * a.cache.max_pages + (p >> a.cache.page_shift)];
  if (page < 0 || page >= a.cache.n_pages) {
    if (c == 0) set_status(a.status, PISA_ERR_DEVICE_BOUNDS);
    return;
  }
  const int U = 1 << a.cache.rec_shift, u = (int)(p & (U - 1));
  uint4 y[2];
  if (KIND == PISA_CACHE_BF16) {
    const unsigned char* rec = a.cache.pages + cache_record(a.cache, kRowBf16, page, kv, p) + u * 128 + 16 * c;
    y[0] = *reinterpret_cast<const uint4*>(rec);
    y[1] = *reinterpret_cast<const uint4*>(rec + U * 128);
  } else {
    const unsigned char* rec = a.cache.pages + cache_record(a.cache, kRowE2m1, page, kv, p);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(rec + i * 36 * U + u * 32 + 4 * c);
      const uint32_t s = e4m3x2(rec[i * 36 * U + 32 * U + u * 4 + (c >> 1)]);
      const float f = __low2float(*reinterpret_cast<const __half2*>(&s)) * exp2i(i ? a.cache.v_exp : a.cache.k_exp);
      uint32_t d[4], o[4];
      e2m1x8(w, d);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&d[k]));
        o[k] = pack_bf16x2(v.x * f, v.y * f);
      }
      y[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  const RowsDev* dst[2] = {&a.k_out, &a.v_out};
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (dst[i]->data)
      *reinterpret_cast<uint4*>(dst[i]->data + b * dst[i]->sb + t * dst[i]->st + kv * dst[i]->sh + 8 * c) = y[i];
}

cudaError_t launch_cache_append(const CacheAppendLaunch& L, cudaStream_t s) {
  const int rows = (L.q.data ? L.Hq : 0) + 2 * L.cache.Hkv;
  const int groups = (rows + 3) / 4;
  const int parts = (groups + kAppIter - 1) / kAppIter, per = (groups + parts - 1) / parts;
  const long long jobs = (long long)L.cache.B * L.T * parts;
  const unsigned blocks = (unsigned)((jobs + kAppWarps - 1) / kAppWarps);
  if (L.cache.kind == PISA_CACHE_BF16)
    cache_append_kernel<PISA_CACHE_BF16><<<blocks, kAppWarps * 32, 0, s>>>(L, parts, per);
  else
    cache_append_kernel<PISA_CACHE_E2M1><<<blocks, kAppWarps * 32, 0, s>>>(L, parts, per);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheReadLaunch& L, cudaStream_t s) {
  const int tok_groups = (L.T + 3) / 4;
  const long long jobs = (long long)L.cache.B * tok_groups * L.cache.Hkv;
  const unsigned blocks = (unsigned)((jobs + 7) / 8);
  if (L.cache.kind == PISA_CACHE_BF16)
    cache_read_kernel<PISA_CACHE_BF16><<<blocks, 256, 0, s>>>(L, tok_groups);
  else
    cache_read_kernel<PISA_CACHE_E2M1><<<blocks, 256, 0, s>>>(L, tok_groups);
  note_launch();
  return cudaGetLastError();
}

}  // namespace pisa
