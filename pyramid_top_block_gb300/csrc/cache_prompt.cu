// cache_prompt.cu -- attention of a prompt's tokens over the paged cache on the tensor cores.
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = exp(x_j - m),   x_j = score(q . k_j) (scores.cuh)
// over the tokens lo <= j < hi of each row's own span, in one pass with a running reference m and sum per row.
//
// Rows are (token, head) pairs of one KV head, heads fastest, so that a head group shares its keys.  A CTA takes
// 256 rows, two tiles of 128, over tiles of 128 keys: S = Q K^T (tcgen05, operands from shared memory) -> registers,
// a row a thread -> weights, back to tensor memory as the left operand of O += P V.  While one row tile's weights are
// computed the tensor core works for the other; keys and values are read from L2 once for both.
//   warps 0 .. 7   softmax, four for each row tile
//   warps 8 .. 11  pages -> shared memory (bf16: asynchronous copies; 4 bits: through registers, as fp16)
//   warp 12        issues the matrix instructions
// Tensor memory, for each row tile: S 128 columns, P 64, O 64; both together all 512.
#include "cache_prompt.cuh"

#include <climits>

namespace pisa {

constexpr int kRowsTile = 128, kRowsCta = 256, kKeys = 128;
constexpr int kSoftWarps = 8, kLoadWarps = 4, kPromptThreads = (kSoftWarps + kLoadWarps + 1) * 32;
constexpr int kPStages = 5;
constexpr int kTileBytes = kKeys * kD * 2;  // keys or values of a tile: rows of 128 bytes, 128-byte swizzle
constexpr int kPromptSmem = 2 * kTileBytes + kPStages * 2 * kTileBytes + 1024;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -0x1.fffffep127f;  // the reference of a row that has seen no logit above minus infinity
constexpr float kFar = 0x1p20f;            // references from which on differences are taken in two steps

// Weights enter the product with V in the pages' type: bf16, or fp16 for 4-bit pages, where they are held
// times 2^10 (weights down to 2^-24 of the reference keep all 11 bits).  A bf16 weight is off by up to 2^-8 of itself,
// as the bf16 result is of its own size; a second part would take half as much again of the tensor core.
template <int KIND>
struct PCfg {
  static constexpr float kShift = KIND == PISA_CACHE_BF16 ? 0.f : 10.f;
  static constexpr float kTop = kShift + (KIND == PISA_CACHE_BF16 ? 20.f : 5.f);  // how far a logit may pass m
  static constexpr uint32_t kType = KIND == PISA_CACHE_BF16 ? 1u : 0u;
  // fp32 accumulator, A and B of the type; the second has B with its columns (dims) contiguous
  static constexpr uint32_t kIdescS = (1u << 4) | (kType << 7) | (kType << 10) | ((kKeys >> 3) << 17) | ((kRowsTile >> 4) << 24);
  static constexpr uint32_t kIdescO =
      (1u << 4) | (kType << 7) | (kType << 10) | (1u << 16) | ((kD >> 3) << 17) | ((kRowsTile >> 4) << 24);
};

// Values [128 keys][64 dims], rows of 128 bytes with 128-byte swizzle, as a B operand whose N dimension (dims) is
// contiguous: eight keys are 1024 bytes (both strides, as N has one block of 64).
__device__ __forceinline__ uint64_t umma_desc_mn128(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3fff) | (64ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

struct PromptShared {
  uint64_t full[kPStages], empty[kPStages];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2], drain;
  uint32_t tmem;
  int abort, odd, bad;
  int lo_min, lo_max, hi_min, hi_max;  // of the rows that see anything
  float factor[kRowsCta];              // 4-bit pages: the rows' logit factors
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// What of a CTA's rows a warp needs to know.
struct PromptUnit {
  int b, kv, r0;   // rows r0 .. r0 + 255 of (b, kv)
  int i0, i1;      // key tiles
  // whether some row does not see some key of the tile
  __device__ __forceinline__ bool mixed(const PromptShared& sh, int tile) const {
    return tile * kKeys < sh.lo_max || (tile + 1) * kKeys > sh.hi_min;
  }
};

// ------------------------------------------------------------------------------------------------ loading

// Where the 16-key pieces of a warp's 32 keys lie, for 16 tiles ahead: lane l has piece l & 1 of tile first + l / 2.
// -1: no row sees any of it, or its page is out of range (noted); its keys and values become zeros.
struct Pieces {
  long long off;
  int first;
};

template <int KIND>
__device__ __forceinline__ void look(const CachePromptLaunch& a, const PromptUnit& u, PromptShared& sh, int warp, int lane,
                                     int tile, Pieces& p) {
  p.first = tile;
  p.off = -1;
  const int key = (tile + (lane >> 1)) * kKeys + 32 * warp + 16 * (lane & 1);
  if (tile + (lane >> 1) < u.i1 && key < sh.hi_max && key + 16 > sh.lo_min) {
    const int page = a.cache.table[(long long)u.b * a.cache.max_pages + (key >> a.cache.page_shift)];
    if (page >= 0 && page < a.cache.n_pages)
      p.off = cache_record(a.cache, KIND == PISA_CACHE_BF16 ? kRowBf16 : kRowE2m1, page, u.kv, key);
    else
      sh.bad = 1;
  }
}

// A bf16 tile's values that this thread copied: those that are not finite become zeros, since 0 times them is
// not zero; the rows that do see them get them at the end (odd_values).
__device__ __forceinline__ void scrub(PromptShared& sh, unsigned char* v, int tile, int warp, int lane) {
  const int sub = lane >> 3, ch = lane & 7;
  bool odd = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int row = 32 * warp + 4 * j + sub;
    uint4* at = reinterpret_cast<uint4*>(v + row * 128 + ((ch ^ (row & 7)) << 4));
    uint4 x = *at;
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((w[i] & 0x7f80u) == 0x7f80u) {
        w[i] &= 0xffff0000u;
        any = true;
      }
      if ((w[i] & 0x7f800000u) == 0x7f800000u) {
        w[i] &= 0xffffu;
        any = true;
      }
    }
    if (any) {
      *at = make_uint4(w[0], w[1], w[2], w[3]);
      const int key = tile * kKeys + row;
      odd = odd || (key >= sh.lo_min && key < sh.hi_max);
    }
  }
  if (odd) sh.odd = 1;
}

// Tiles of bf16 pages: copied ahead by two tiles, then handed over.
__device__ __forceinline__ bool load_bf16(const CachePromptLaunch& a, const PromptUnit& u, PromptShared& sh,
                                          unsigned char* stages, unsigned kt, int warp, int lane) {
  constexpr int kAhead = 2;
  const int sub = lane >> 3, ch = lane & 7, U = 1 << a.cache.rec_shift, n = u.i1 - u.i0;
  Pieces p;
  bool ok = true;
  for (int x = 0; x < n + kAhead && ok; ++x) {
    if (x < n) {
      const unsigned k = kt + x, st = k % kPStages;
      if (k >= kPStages) ok = mbar_wait(&sh.empty[st], (k / kPStages - 1) & 1, &sh.abort);
      ok = __all_sync(kFull, ok);
      if (!ok) break;
      const int tile = u.i0 + x;
      if (x % 16 == 0) look<PISA_CACHE_BF16>(a, u, sh, warp, lane, tile, p);
      const uint32_t base = smem_u32(stages) + st * 2 * kTileBytes;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int key = 4 * j + sub, row = 32 * warp + key;  // (of the tile)
        const long long off = __shfl_sync(kFull, p.off, ((x % 16) << 1) | (j >> 2));
        const int in = (tile * kKeys + row) & (U - 1);  // row of its record
        const unsigned char* src = a.cache.pages + (off < 0 ? 0 : off + in * 128 + ch * 16);
        const uint32_t dst = base + row * 128 + ((ch ^ (row & 7)) << 4);
        cp16(dst, src, off >= 0);
        cp16(dst + kTileBytes, off < 0 ? src : src + U * 128, off >= 0);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (x >= kAhead) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
      const unsigned st = (kt + x - kAhead) % kPStages;
      const int tile = u.i0 + x - kAhead;
      if (u.mixed(sh, tile)) scrub(sh, stages + st * 2 * kTileBytes + kTileBytes, tile, warp, lane);
      fence_async_proxy();
      mbar_arrive(&sh.full[st]);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  return ok;
}

// 16 dims of a token: 8 bytes of codes and a scale, as 16 fp16.
__device__ __forceinline__ void dequant16(uint32_t c0, uint32_t c1, uint32_t scale, uint4& x, uint4& y) {
  const uint32_t s2 = e4m3x2(scale | scale << 8);
  uint32_t d[4];
  e2m1x8(c0, d);
  x = make_uint4(hmul2u(d[0], s2), hmul2u(d[1], s2), hmul2u(d[2], s2), hmul2u(d[3], s2));
  e2m1x8(c1, d);
  y = make_uint4(hmul2u(d[0], s2), hmul2u(d[1], s2), hmul2u(d[2], s2), hmul2u(d[3], s2));
}

// Tiles of 4-bit pages: a token a thread, the next tile's words on their way meanwhile.
__device__ __forceinline__ bool load_e2m1(const CachePromptLaunch& a, const PromptUnit& u, PromptShared& sh,
                                          unsigned char* stages, unsigned kt, int warp, int lane) {
  const int U = 1 << a.cache.rec_shift, n = u.i1 - u.i0, row = 32 * warp + lane;
  Pieces p;
  uint4 k0, k1, v0, v1;
  uint32_t ks, vs;
  auto fetch = [&](int x) {
    if (x % 16 == 0) look<PISA_CACHE_E2M1>(a, u, sh, warp, lane, u.i0 + x, p);
    const long long off = __shfl_sync(kFull, p.off, ((x % 16) << 1) | (lane >> 4));
    k0 = k1 = v0 = v1 = make_uint4(0, 0, 0, 0);
    ks = vs = 0;
    if (off >= 0) {
      const int in = ((u.i0 + x) * kKeys + row) & (U - 1);
      const unsigned char* r = a.cache.pages + off;
      const uint4* kc = reinterpret_cast<const uint4*>(r + in * 32);
      const uint4* vc = reinterpret_cast<const uint4*>(r + 36 * U + in * 32);
      k0 = kc[0];
      k1 = kc[1];
      ks = *reinterpret_cast<const uint32_t*>(r + 32 * U + in * 4);
      v0 = vc[0];
      v1 = vc[1];
      vs = *reinterpret_cast<const uint32_t*>(r + 68 * U + in * 4);
    }
  };
  bool ok = true;
  fetch(0);
  for (int x = 0; x < n; ++x) {
    const unsigned k = kt + x, st = k % kPStages;
    if (k >= kPStages) ok = mbar_wait(&sh.empty[st], (k / kPStages - 1) & 1, &sh.abort);
    ok = __all_sync(kFull, ok);
    if (!ok) break;
    const int tile = u.i0 + x;
    if (u.mixed(sh, tile)) {  // NaN blocks of values that not all rows see become zeros (see scrub)
      uint32_t keep = 0xffffffffu;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((vs >> (8 * i) & 0x7fu) == 0x7fu) keep &= ~(0xffu << (8 * i));
      if (keep != 0xffffffffu) {
        vs &= keep;
        const int key = tile * kKeys + row;
        if (key >= sh.lo_min && key < sh.hi_max) sh.odd = 1;
      }
    }
    unsigned char* kd = stages + st * 2 * kTileBytes + row * 128;
    const uint32_t w[2][8] = {{k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w},
                              {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w}};
    const uint32_t sc[2] = {ks, vs};
    uint4 y[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) dequant16(w[h][2 * i], w[h][2 * i + 1], sc[h] >> (8 * i) & 0xffu, y[h][2 * i], y[h][2 * i + 1]);
    if (x + 1 < n) fetch(x + 1);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(kd + h * kTileBytes + ((i ^ (row & 7)) << 4)) = y[h][i];
    fence_async_proxy();
    mbar_arrive(&sh.full[st]);
  }
  return ok;
}

// ------------------------------------------------------------------------------------------------ the MMA warp

template <int KIND>
__device__ __forceinline__ bool multiply(const PromptUnit& u, PromptShared& sh, const unsigned char* q,
                                         const unsigned char* stages, unsigned kt, int lane, bool& issued) {
  const int n = u.i1 - u.i0;
  const uint32_t tmem = sh.tmem;
  bool ok = true;
  for (int x = 0; x <= n && ok; ++x) {
    const unsigned k = kt + x, st = k % kPStages, before = (k - 1) % kPStages;
    if (x < n) ok = mbar_wait(&sh.full[st], (k / kPStages) & 1, &sh.abort);
#pragma unroll
    for (int X = 0; X < 2; ++X) {
      if (x < n) {  // S = Q K^T
        if (k > 0) ok = ok && mbar_wait(&sh.s_free[X], (k - 1) & 1, &sh.abort);
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const uint64_t da = umma_desc_sw128(q + X * kTileBytes);
          const uint64_t db = umma_desc_sw128(stages + st * 2 * kTileBytes);
#pragma unroll
          for (int i = 0; i < 4; ++i)  // (16 dims are 32 bytes, 2 in the descriptor's units)
            umma_ss(tmem + 256 * X, da + 2 * i, db + 2 * i, PCfg<KIND>::kIdescS, i);
          umma_commit(&sh.s_full[X]);
        }
        issued = true;
        __syncwarp();
      }
      if (x > 0) {  // O += P V of the tile before
        ok = __all_sync(kFull, mbar_wait(&sh.p_full[X], (k - 1) & 1, &sh.abort));
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const uint64_t db = umma_desc_mn128(smem_u32(stages + before * 2 * kTileBytes + kTileBytes));
#pragma unroll
          for (int i = 0; i < 8; ++i)  // (16 keys are 2048 bytes of V and 8 columns of P)
            umma_ts(tmem + 256 * X + 192, tmem + 256 * X + 128 + 8 * i, db + 128 * i, PCfg<KIND>::kIdescO,
                    x > 1 || i > 0);
          umma_commit(&sh.pv_done[X]);
          if (X == 1) umma_commit(&sh.empty[before]);
        }
        __syncwarp();
      }
    }
  }
  return ok;
}

// ------------------------------------------------------------------------------------------------ softmax

struct PromptRow {
  int lo, hi, pos;  // the row's span (empty where lo >= hi) and position
  int head, t;
  bool there;       // whether the row exists
  float f;          // logit factor
  float m, l;       // reference and sum of weights
  float slope, dref;  // bias by distance, base 2, relative to the nearest token that is seen
  CapRow cap;
};

__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 64 products of a row, of the keys from key0 on, as the logits that the softmax takes with factor ff.
template <bool SCORED>
__device__ __forceinline__ void logits(const CachePromptLaunch& a, const PromptRow& r, int key0, bool whole, bool two_step,
                                       float (&v)[64]) {
  if constexpr (SCORED) {
    if (a.score.cap > 0.f) {
      float b = 0.f;
#pragma unroll
      for (int i = 0; i < 64; i += 2) b = max3f(b, fabsf(v[i]), fabsf(v[i + 1]));
      if (__any_sync(kFull, b * r.cap.to_y > 1.f)) {
        const float top = a.score.cap * kLog2e;
#pragma unroll
        for (int i = 0; i < 64; ++i) v[i] = cap_any(v[i], r.cap, top);
      } else {
#pragma unroll
        for (int i = 0; i < 64; i += 2) cap_small(v[i], v[i + 1], r.cap);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 64; ++i) v[i] *= r.f;
    }
    if (a.score.slopes) {  // -slope (|p - j| - |p - nearest|): whole numbers, exact up to 2^24
      const float d0 = (float)(key0 - r.pos);
#pragma unroll
      for (int i = 0; i < 64; ++i) v[i] = fmaf(-r.slope, fabsf(d0 + (float)i) - r.dref, v[i]);
    }
  } else if (two_step) {
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = __fmul_rn(v[i], r.f);
  }
  if (!whole) {
    const int from = r.lo - key0, to = r.hi - key0;
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = i >= from && i < to ? v[i] : -INFINITY;
  }
}

__device__ __forceinline__ float max64(const float (&v)[64]) {
  float b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
  for (int i = 0; i < 64; i += 4) {
    b0 = max3f(b0, v[i], v[i + 1]);
    b1 = max3f(b1, v[i + 2], v[i + 3]);
  }
  return fmaxf(b0, b1);
}

__device__ __forceinline__ void load64(uint32_t taddr, float (&v)[64]) {
  uint32_t w[64];
  tmem_ld64_now(taddr, w);
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(w[i]);
}

// The softmax of one key tile for the warp's 32 rows.  s: the S columns of the warp's lanes.
template <int KIND, bool SCORED>
__device__ __forceinline__ bool soften(const CachePromptLaunch& a, PromptShared& sh, PromptRow& r, uint32_t s, int X,
                                       int lane, int tile, unsigned k, bool first, bool& two_step) {
  using C = PCfg<KIND>;
  const int key0 = tile * kKeys;
  // (rows that see nothing do not matter: they get zeros at the end, or do not exist)
  const bool whole = __all_sync(kFull, r.lo >= r.hi || (r.lo <= key0 && r.hi >= key0 + kKeys));
  bool ok = __all_sync(kFull, mbar_wait(&sh.s_full[X], k & 1, &sh.abort));
  if (!ok) return false;
  tc_fence_after();
  bool waited = k == 0;  // for the product before, which reads P and writes O
  const auto wait_pv = [&] {
    if (!waited) {
      ok = __all_sync(kFull, mbar_wait(&sh.pv_done[X], (k - 1) & 1, &sh.abort));
      tc_fence_after();
      waited = true;
    }
    return ok;
  };
  const auto factor = [&] { return SCORED || two_step ? 1.f : r.f; };
  bool scan = first;
  float sum;
  while (true) {
    if (scan) {  // a new reference: the largest logit, less the shift
      float b = -INFINITY;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        float v[64];
        load64(s + 64 * h, v);
        logits<SCORED>(a, r, key0 + 64 * h, whole, two_step, v);
        b = fmaxf(b, max64(v));
      }
      const float t = __fmul_rn(b, factor());
      const float n = fmaxf(r.m, fabsf(t) < 16.f * kFar ? t - C::kShift : t);
      const float f = ex2_approx(r.m - n);
      r.m = n;
      r.l *= f;
      if (!SCORED) two_step = two_step || __any_sync(kFull, fabsf(n) >= kFar && n != kNone);
      if (!first) {  // what O holds has the old reference
        if (!wait_pv()) return false;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t o[32];
          tmem_ld32_now(s + 192 + 32 * h, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          tmem_st32(s + 192 + 32 * h, o);
        }
        tmem_st_wait();
      }
    }
    sum = 0.f;
    bool again = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[64];
      load64(s + 64 * h, v);
      logits<SCORED>(a, r, key0 + 64 * h, whole, two_step, v);
      const float ff = factor();
      if (!scan && __any_sync(kFull, max64(v) * ff > r.m + C::kTop)) {
        again = true;
        break;
      }
      if (h == 1) {  // S is in registers: the next product may overwrite it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.s_free[X]);
      }
      const unsigned long long f2 = f2_pack(ff, ff), m2 = f2_pack(-r.m, -r.m);
      unsigned long long s0 = 0, s1 = 0;
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float x, y;
        f2_unpack(f2_fma(f2_pack(v[2 * i], v[2 * i + 1]), f2, m2), x, y);
        x = ex2_approx(x);
        y = ex2_approx(y);
        if (i & 1)
          s1 = f2_add(s1, f2_pack(x, y));
        else
          s0 = f2_add(s0, f2_pack(x, y));
        w[i] = KIND == PISA_CACHE_BF16 ? pack_bf16x2(x, y) : pack_f16x2(x, y);
      }
      float x, y;
      f2_unpack(f2_add(s0, s1), x, y);
      sum += x + y;
      if (!wait_pv()) return false;
      tmem_st32(s + 128 + 32 * h, w);
    }
    if (!again) break;
    scan = true;
  }
  r.l += sum;
  tmem_st_wait();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(&sh.p_full[X]);
  return true;
}

// Values that scrub took out, of tokens that this row sees, in dims d0 .. d0 + 31 (an infinity, or a NaN, whatever
// the weight).
template <int KIND>
__device__ __forceinline__ void odd_values(const CachePromptLaunch& a, const PromptUnit& u, const PromptShared& sh,
                                           const PromptRow& r, int d0, float (&o)[32]) {
  const int U = 1 << a.cache.rec_shift;
  for (int tile = u.i0; tile < u.i1; ++tile) {
    if (!u.mixed(sh, tile)) continue;
    for (int key = max(tile * kKeys, r.lo); key < min((tile + 1) * kKeys, r.hi); ++key) {
      const int page = a.cache.table[(long long)u.b * a.cache.max_pages + (key >> a.cache.page_shift)];
      if (page < 0 || page >= a.cache.n_pages) continue;
      const int in = key & (U - 1);
      if (KIND == PISA_CACHE_BF16) {
        const unsigned char* v = a.cache.pages + cache_record(a.cache, kRowBf16, page, u.kv, key) + U * 128 + in * 128 + 2 * d0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 x = reinterpret_cast<const uint4*>(v)[i];
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if ((w[j] & 0x7f80u) == 0x7f80u) o[8 * i + 2 * j] += __uint_as_float(w[j] << 16);
            if ((w[j] & 0x7f800000u) == 0x7f800000u) o[8 * i + 2 * j + 1] += __uint_as_float(w[j] & 0xffff0000u);
          }
        }
      } else {
        const unsigned char* s = a.cache.pages + cache_record(a.cache, kRowE2m1, page, u.kv, key) + 68 * U + in * 4 + d0 / 16;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if ((s[i / 16] & 0x7f) == 0x7f) o[i] = __int_as_float(0x7fc00000);
      }
    }
  }
}

// Whether the row sees a token in a page out of range, among tiles i0 .. i1 - 1.
__device__ __forceinline__ bool sees_bad(const CachePromptLaunch& a, const PromptUnit& u, const PromptRow& r) {
  const int from = max(r.lo, u.i0 * kKeys), to = min(r.hi, u.i1 * kKeys);
  if (from >= to) return false;
  for (int e = from >> a.cache.page_shift; e <= (to - 1) >> a.cache.page_shift; ++e) {
    const int page = a.cache.table[(long long)u.b * a.cache.max_pages + e];
    if (page < 0 || page >= a.cache.n_pages) return true;
  }
  return false;
}

__device__ __forceinline__ void write_row(const CachePromptLaunch& a, const PromptUnit& u, const PromptRow& r, int d0,
                                          const float (&o)[32]) {
  if (!r.there) return;
  const float f = r.l == 0.f ? 0.f : exp2i(a.cache.kind == PISA_CACHE_E2M1 ? a.cache.v_exp : 0) / r.l;
  uint4* dst = reinterpret_cast<uint4*>(a.out + (((long long)u.b * a.T + r.t) * a.Hq + r.head) * kD + d0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = r.l == 0.f ? 0u : pack_bf16x2(o[8 * i + 2 * j] * f, o[8 * i + 2 * j + 1] * f);
    dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ------------------------------------------------------------------------------------------------ the kernel

// The queries of the CTA's rows as two swizzled operands, by the softmax warps: eight threads a row.  4-bit pages:
// as fp16, the row scaled by a power of two so that its largest element lies in [1, 2) (cache_attend.cuh, make_q).
template <int KIND, bool SCORED>
__device__ __forceinline__ void stage_queries(const CachePromptLaunch& a, const PromptUnit& u, PromptShared& sh,
                                              unsigned char* q, int count, int g_shift) {
  const int ch = threadIdx.x & 7;
#pragma unroll 4
  for (int it = 0; it < 8; ++it) {
    const int row = it * 32 + (threadIdx.x >> 3), r = u.r0 + row, t = r >> g_shift;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (t < count) {
      const int head = u.kv * a.G + (r & (a.G - 1));
      x = *reinterpret_cast<const uint4*>(a.q.data + u.b * a.q.sb + (long long)t * a.q.st + head * a.q.sh + 8 * ch);
    }
    if (KIND == PISA_CACHE_E2M1) {
      uint32_t w[4] = {x.x, x.y, x.z, x.w}, m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
      m = max(m & 0xffffu, m >> 16);
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) m = max(m, __shfl_xor_sync(kFull, m, d));
      const int e = max(min((int)(m >> 7) - 127, 126), -100);
      const float down = exp2i(-e);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = pack_f16x2(__uint_as_float(w[i] << 16) * down, __uint_as_float(w[i] & 0xffff0000u) * down);
      x = make_uint4(w[0], w[1], w[2], w[3]);
      constexpr float kFactor = SCORED ? kScale : kScale * kLog2e;
      if (ch == 0) sh.factor[row] = fminf(kFactor * exp2i(e) * exp2i(a.cache.k_exp), 0x1.fffffep127f);
    }
    *reinterpret_cast<uint4*>(q + row * 128 + ((ch ^ (row & 7)) << 4)) = x;
  }
}

template <int KIND, bool SCORED>
__global__ void __launch_bounds__(kPromptThreads, 1) cache_prompt_kernel(CachePromptLaunch a, int g_shift, int row_tiles) {
  extern __shared__ unsigned char prompt_smem[];
  __shared__ PromptShared sh;
  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  unsigned char* q = prompt_smem + ((1024 - (smem_u32(prompt_smem) & 1023)) & 1023);
  unsigned char* stages = q + 2 * kTileBytes;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPStages; ++i) {
      mbar_init(&sh.full[i], kLoadWarps * 32);
      mbar_init(&sh.empty[i], 1);
    }
    for (int X = 0; X < 2; ++X) {
      mbar_init(&sh.s_full[X], 1);
      mbar_init(&sh.s_free[X], 4);
      mbar_init(&sh.p_full[X], 4);
      mbar_init(&sh.pv_done[X], 1);
    }
    mbar_init(&sh.drain, 1);
    mbar_fence_init();
    sh.abort = sh.odd = sh.bad = 0;
    sh.lo_min = sh.hi_min = INT_MAX;
    sh.lo_max = sh.hi_max = 0;
  }
  after_the_one_before();
  if (warp == kSoftWarps + kLoadWarps) tmem_alloc<512>(&sh.tmem);  // (held by no kernel that waits for another one)
  // the longest row tiles first
  PromptUnit u;
  const int heads = a.cache.B * a.cache.Hkv, bk = blockIdx.x % heads;
  u.b = bk / a.cache.Hkv;
  u.kv = bk % a.cache.Hkv;
  u.r0 = (row_tiles - 1 - (int)(blockIdx.x / heads)) * kRowsCta;
  const int count = prompt_count(a, u.b);
  PromptRow r{};
  if (warp < kSoftWarps) {
    const int row = u.r0 + threadIdx.x;
    r.t = row >> g_shift;
    r.head = u.kv * a.G + (row & (a.G - 1));
    r.there = r.t < count;
    if (r.there) {
      bool over;
      const Span s = span_of(a, u.b, r.t, count, over);
      if (over) set_status(a.status, PISA_ERR_DEVICE_BOUNDS);
      r.lo = s.lo;
      r.hi = s.hi;
      r.pos = s.pos;
    }
  }
  __syncthreads();
  if (warp < kSoftWarps) {
    const bool sees = r.lo < r.hi;
    const int lo_min = __reduce_min_sync(kFull, sees ? r.lo : INT_MAX), lo_max = __reduce_max_sync(kFull, sees ? r.lo : 0);
    const int hi_min = __reduce_min_sync(kFull, sees ? r.hi : INT_MAX), hi_max = __reduce_max_sync(kFull, sees ? r.hi : 0);
    if (lane == 0) {
      atomicMin(&sh.lo_min, lo_min);
      atomicMax(&sh.lo_max, lo_max);
      atomicMin(&sh.hi_min, hi_min);
      atomicMax(&sh.hi_max, hi_max);
    }
    stage_queries<KIND, SCORED>(a, u, sh, q, count, g_shift);
    fence_async_proxy();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  u.i0 = sh.lo_min < sh.hi_max ? sh.lo_min / kKeys : 0;
  u.i1 = sh.lo_min < sh.hi_max ? (sh.hi_max + kKeys - 1) / kKeys : 0;
  const unsigned kt = 0;
  bool ok = true, issued = false;
  if (warp < kSoftWarps) {
    const int X = warp >> 2, n = u.i1 - u.i0;
    const uint32_t s = sh.tmem + 256 * X + ((uint32_t)(warp & 3) << 21);  // (lanes 32 (warp & 3) .. of the tile's columns)
    r.f = KIND == PISA_CACHE_E2M1 ? sh.factor[threadIdx.x] : SCORED ? kScale : kScale * kLog2e;
    r.m = kNone;
    if (SCORED) {
      r.cap = CapRow{r.f * a.score.inv_cap, r.f * kLog2e};
      r.f *= kLog2e;
      if (a.score.slopes && r.there) {
        r.slope = a.score.slopes[r.head] * kLog2e;
        r.dref = (float)abs(r.pos - max(min(r.pos, r.hi - 1), r.lo));
      }
    }
    bool two_step = false;
    for (int x = 0; x < n && ok; ++x)
      ok = soften<KIND, SCORED>(a, sh, r, s, X, lane, u.i0 + x, kt + x, x == 0, two_step);
    if (ok && n > 0) ok = __all_sync(kFull, mbar_wait(&sh.pv_done[X], (kt + n - 1) & 1, &sh.abort));
    if (ok) {
      tc_fence_after();
      if (r.lo >= r.hi) r.l = 0.f;  // (its weights were never masked: see soften)
      if (sh.bad && sees_bad(a, u, r)) {
        r.l = __int_as_float(0x7fc00000);
        set_status(a.status, PISA_ERR_DEVICE_BOUNDS);
      }
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        float o[32];
        if (n > 0) {
          uint32_t w[32];
          tmem_ld32_now(s + 192 + 32 * h, w);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(w[i]);
          if (sh.odd) odd_values<KIND>(a, u, sh, r, 32 * h, o);
        }
        write_row(a, u, r, 32 * h, o);
      }
      tc_fence_before();
    }
  } else if (warp < kSoftWarps + kLoadWarps) {
    if (u.i0 < u.i1) {
      if (KIND == PISA_CACHE_BF16)
        ok = load_bf16(a, u, sh, stages, kt, warp - kSoftWarps, lane);
      else
        ok = load_e2m1(a, u, sh, stages, kt, warp - kSoftWarps, lane);
    }
  } else if (u.i0 < u.i1) {
    ok = multiply<KIND>(u, sh, q, stages, kt, lane, issued);
  }
  if (!ok && lane == 0) {  // a wait ran out: the others give up, too
    *const_cast<volatile int*>(&sh.abort) = 1;
    set_status(a.status, PISA_ERR_DEVICE_TIMEOUT);
  }
  if (!ok && issued) {  // (the MMA warp: its products end before tensor memory is given back)
    if (lane == 0) {
      umma_commit(&sh.drain);
      mbar_wait(&sh.drain, 0, nullptr);
    }
    __syncwarp();
  }
  __syncthreads();
  if (warp == kSoftWarps + kLoadWarps) tmem_dealloc<512>(sh.tmem);
}

template <int KIND, bool SCORED>
static cudaError_t launch_prompt(const CachePromptLaunch& L, cudaStream_t s) {
  int g_shift = 0;
  while ((1 << g_shift) < L.G) ++g_shift;
  const int row_tiles = (int)(((long long)L.T * L.G + kRowsCta - 1) / kRowsCta);
  const long long units = (long long)row_tiles * L.cache.B * L.cache.Hkv;
  return launch_early<cache_prompt_kernel<KIND, SCORED>>((unsigned)units, kPromptThreads, kPromptSmem, s, L, g_shift,
                                                         row_tiles);
}

cudaError_t launch_cache_prompt(const CachePromptLaunch& L, cudaStream_t s) {
  const bool scored = L.score.cap > 0.f || L.score.slopes;
  if (L.cache.kind == PISA_CACHE_BF16)
    return scored ? launch_prompt<PISA_CACHE_BF16, true>(L, s) : launch_prompt<PISA_CACHE_BF16, false>(L, s);
  return scored ? launch_prompt<PISA_CACHE_E2M1, true>(L, s) : launch_prompt<PISA_CACHE_E2M1, false>(L, s);
}

}  // namespace pisa
