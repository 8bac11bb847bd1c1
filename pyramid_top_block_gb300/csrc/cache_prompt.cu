// cache_prompt.cu -- attention of a prompt's tokens over the paged cache on the tensor cores.
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = exp(x_j - m),   x_j = score(q . k_j) (scores.cuh)
// over the tokens lo <= j < hi of each row's own span, in one pass with a running reference m and sum per row.
//
// Rows are (token, head) pairs of one KV head, heads fastest, so that a head group shares its keys.  A CTA takes
// 256 rows, two tiles of 128, over tiles of 128 keys: S = Q K^T (tcgen05, operands from shared memory) -> registers,
// a row a thread -> weights, back to tensor memory as the left operand of O += P V.  While one row tile's weights
// are computed the tensor core works for the other; keys and values are read from L2 once for both.
//   warps 0 .. 7    softmax, four for each row tile
//   warps 8, 9      pages -> shared memory, every second tile each (bf16: by TMA; 4 bits: through registers, as fp16)
//   warps 10, 11    issue the matrix instructions: one S = Q K^T, the other O += P V
// Tensor memory, for each row tile: S 128 columns, P 64, O 64; both together all 512.
//
// What bounds it: a step of 256 rows and 128 keys takes the tensor core 1552 clocks (the product with V has 64 columns,
// and takes as long as with 128) and the exponentials 1024, and each row tile waits for its product, takes its scores
// into registers, weighs them and hands the weights back: about 2000 clocks.  32 heads on 2, bf16 (4-bit) pages: 32768
// tokens 3.51 ms = 1.25 PFLOP/s (3.81 ms), 2048 at 131072 1.68 ms = 1.30 PFLOP/s (1.82), 1216 at 16384 132 us (142),
// capped 170 to 180, with slopes 161; a library's bf16 product of matrices reaches 1.90 PFLOP/s.
#include "cache_prompt.cuh"

#include <climits>
#include <mutex>
#include <type_traits>

#include <cudaTypedefs.h>

namespace pisa {

// Where there are few row tiles of a CTA (units) for their length, the key tiles of all units form one stream that is
// cut into runs of equal length, one for each SM, and where a unit ends: a CTA takes a piece, the longest first.  Units
// in several pieces leave partial results, which a last kernel joins (takes_stream says when).  (A CTA for a run, with
// a loop over its pieces, was slower: the loop costs the softmax the registers that hold its scores, 138 -> 233 us for
// 1216 tokens at 16384.)
constexpr int kRuns = kPromptRuns, kMaxUnits = kPromptUnits;
// places of the stream that a unit counts beside its tiles: what its begin and end cost
constexpr int kUnitEnd = 4;
constexpr int kMinRun = 4;             // places that a run has at least
constexpr int kPartRow = 66;           // a partial result, for each of 256 rows: O [64], reference, sum of weights
constexpr int kRowsTile = 128, kRowsCta = 256, kKeys = 128;
constexpr int kSoftWarps = 8, kLoadWarps = 2, kPromptThreads = (kSoftWarps + kLoadWarps + 2) * 32;
constexpr int kTileBytes = kKeys * kD * 2;  // keys or values of a tile: rows of 128 bytes, 128-byte swizzle
constexpr int kRawBytes = kKeys * kRowE2m1;  // a tile as 4-bit pages hold it
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
  static constexpr int kStages = KIND == PISA_CACHE_BF16 ? 5 : 4;  // tiles of keys and values in shared memory
  static constexpr int kSmem =
      1024 + (2 + 2 * kStages) * kTileBytes + (KIND == PISA_CACHE_BF16 ? 0 : 2 * kLoadWarps * kRawBytes);
  static constexpr uint32_t kType = KIND == PISA_CACHE_BF16 ? 1u : 0u;
  // fp32 accumulator, A and B of the type; the second has B with its columns (dims) contiguous
  static constexpr uint32_t kIdescS =
      (1u << 4) | (kType << 7) | (kType << 10) | ((kKeys >> 3) << 17) | ((kRowsTile >> 4) << 24);
  static constexpr uint32_t kIdescO =
      (1u << 4) | (kType << 7) | (kType << 10) | (1u << 16) | ((kD >> 3) << 17) | ((kRowsTile >> 4) << 24);
};

// Values [128 keys][64 dims], rows of 128 bytes with 128-byte swizzle, as a B operand whose N dimension (dims) is
// contiguous: eight keys are 1024 bytes (both strides, as N has one block of 64).
__device__ __forceinline__ uint64_t umma_desc_mn128(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3fff) | (64ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// Key tiles go from the last to the first: where a bias by distance grows towards a row's own position, the first
// tile then has the largest logits, and the reference stays.
struct PromptUnit {
  int b, kv, r0;   // rows r0 .. r0 + 255 of (b, kv)
  int i0, i1;      // key tiles that this CTA takes
  __device__ __forceinline__ unsigned n() const { return i1 - i0; }
  __device__ __forceinline__ int tile(int k) const { return i1 - 1 - k; }  // the k-th
};

// What a loading warp has asked for.
struct Asked {
  unsigned count;   // waits on its own landing barrier (bf16), raw buffers (4 bits)
  unsigned stages;  // bf16: bit i: stage i, bit 8 + i: the parity of the phase in which that lands
};

struct PromptShared {
  uint64_t full[5], empty[5];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2], drain[2];
  uint64_t landed[kLoadWarps][2];  // (bf16: the first; 4 bits: of each raw buffer)
  uint32_t tmem;
  int abort, odd, bad;
  int lo_min, lo_max, hi_min, hi_max;  // of the rows that see anything
  Asked asked[kLoadWarps];
  // what the softmax needs at its end alone (its registers are full of scores)
  PromptUnit unit;
  int slot;
  float factor[kRowsCta];              // 4-bit pages: the rows' logit factors
};

// Whether some row of the CTA does not see some key of the tile.
__device__ __forceinline__ bool mixed_tile(const PromptShared& sh, int tile) {
  return tile * kKeys < sh.lo_max || (tile + 1) * kKeys > sh.hi_min;
}

// ------------------------------------------------------------------------------------------------ loading

// A loading warp takes every second tile, whole.  The pages of its tiles' records, four tiles ahead: lane l has record
// l % 8 (of 8, 4 or 2) of the tile number first + 2 (l / 8).  n_pages: no row sees any of it, or its page is out of
// range (noted); its keys and values become zeros.
__device__ __forceinline__ int look(const CachePromptLaunch& a, const PromptUnit& u, PromptShared& sh, int lane,
                                    int first) {
  const int tile = u.tile(first + kLoadWarps * (lane >> 3)), U = 1 << a.cache.rec_shift;
  const int key = tile * kKeys + U * (lane & 7);
  if (U * (lane & 7) >= kKeys || tile < u.i0 || key >= sh.hi_max || key + U <= sh.lo_min) return a.cache.n_pages;
  const int page = a.cache.table[(long long)u.b * a.cache.max_pages + (key >> a.cache.page_shift)];
  if (page >= 0 && page < a.cache.n_pages) return page;
  sh.bad = 1;
  return a.cache.n_pages;
}

// A bf16 tile's values: those that are not finite become zeros, since 0 times them is not zero; the rows that do see
// them get them at the end (odd_values).
__device__ __forceinline__ void scrub(PromptShared& sh, unsigned char* v, int tile, int lane) {
  const int sub = lane >> 3, ch = lane & 7;
  const auto at = [&](int j) {
    const int row = 4 * j + sub;
    return reinterpret_cast<uint4*>(v + row * 128 + ((ch ^ (row & 7)) << 4));
  };
  // an exponent of all ones carries into the sign's place
  const auto test = [](uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
  uint32_t some = 0;  // bit j: something in this lane's row number j
#pragma unroll 8
  for (int j = 0; j < kKeys / 4; ++j) {
    const uint4 x = *at(j);
    if (test(x.x) | test(x.y) | test(x.z) | test(x.w)) some |= 1u << j;
  }
  for (; some; some &= some - 1) {
    const int j = __ffs(some) - 1, key = tile * kKeys + 4 * j + sub;
    const uint4 x = *at(j);
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
      if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0xffffu;
    }
    *at(j) = make_uint4(w[0], w[1], w[2], w[3]);
    if (key >= sh.lo_min && key < sh.hi_max) sh.odd = 1;
  }
}

// Whether no row sees the key.  (In a scored call's mixed tile such keys become zeros: no row's logits count them, but
// the largest product of a tile chooses how scores are computed.)
__device__ __forceinline__ bool is_scored(const CachePromptLaunch& a) { return a.score.cap > 0.f || a.score.slopes; }
__device__ __forceinline__ bool unseen(const PromptShared& sh, int key) { return key < sh.lo_min || key >= sh.hi_max; }

// 16 dims of a token: 8 bytes of codes and a scale, as 16 fp16.
__device__ __forceinline__ void dequant16(uint32_t c0, uint32_t c1, uint32_t scale, uint4& x, uint4& y) {
  const uint32_t s2 = e4m3x2(scale | scale << 8);
  uint32_t d[4];
  e2m1x8(c0, d);
  x = make_uint4(hmul2u(d[0], s2), hmul2u(d[1], s2), hmul2u(d[2], s2), hmul2u(d[3], s2));
  e2m1x8(c1, d);
  y = make_uint4(hmul2u(d[0], s2), hmul2u(d[1], s2), hmul2u(d[2], s2), hmul2u(d[3], s2));
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// bf16 pages by TMA.
__device__ __forceinline__ bool load_bf16(const CachePromptLaunch& a, const CUtensorMap* map, const PromptUnit& u,
                                          PromptShared& sh, unsigned char* stages, int warp, int lane) {
  constexpr unsigned kPStages = PCfg<PISA_CACHE_BF16>::kStages;
  Asked asked = {0, 0};
  const int rs = a.cache.rec_shift;
  int page = 0, mine = 0;
  for (unsigned k = warp; k < u.n(); k += kLoadWarps, ++mine) {
    const unsigned st = k % kPStages;
    const int tile = u.tile(k);
    if (mine % 4 == 0) page = look(a, u, sh, lane, k);
    const bool ok = k < kPStages || mbar_wait(&sh.empty[st], (k / kPStages - 1) & 1, &sh.abort);
    if (!__all_sync(kFull, ok)) return false;
    unsigned char* stage = stages + st * 2 * kTileBytes;
    const bool mixed = mixed_tile(sh, tile);
    // lane 2 i + h: the keys (h = 0) or values of record i; a page number of n_pages lies outside the map and gives
    // zeros
    uint64_t* bar = mixed ? &sh.landed[warp][0] : &sh.full[st];
    if (lane == 0) mbar_expect_tx(bar, 2 * kTileBytes);
    __syncwarp();
    const int i = lane >> 1, h = lane & 1, from = __shfl_sync(kFull, page, ((mine % 4) * 8 + i) & 31);
    if (i < kKeys >> rs) {
      const int key = tile * kKeys + (i << rs), rec = (key & ((1 << a.cache.page_shift) - 1)) >> rs;
      tma_load_4d(stage + h * kTileBytes + (i << rs) * 128, map, 0, 0,
                  (((u.kv << (a.cache.page_shift - rs)) + rec) << 1) + h, from, bar);
    }
    if (mixed) {
      if (!__all_sync(kFull, mbar_wait(bar, asked.count & 1, &sh.abort))) {
        mbar_wait(bar, asked.count & 1, nullptr);  // (given up; the copies land first)
        return false;
      }
      ++asked.count;
      scrub(sh, stage + kTileBytes, tile, lane);
      if (is_scored(a)) {
#pragma unroll 4
        for (int j = lane; j < kKeys * 8; j += 32)
          if (unseen(sh, tile * kKeys + (j >> 3))) reinterpret_cast<uint4*>(stage)[j] = make_uint4(0, 0, 0, 0);
      }
      fence_async_proxy();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.full[st]);
    }
    asked.stages = (asked.stages & ~(0x100u << st)) | (1u << st) | (((k / kPStages) & 1) << (8 + st));
    if (lane == 0) sh.asked[warp] = asked;
  }
  return true;
}

// 4-bit pages: records by bulk copies into one of the warp's two raw buffers, a tile ahead; from there as fp16 into the
// stage, a token a lane.
__device__ __forceinline__ bool load_e2m1(const CachePromptLaunch& a, const PromptUnit& u, PromptShared& sh,
                                          unsigned char* stages, unsigned char* raw, int warp, int lane) {
  constexpr unsigned kPStages = PCfg<PISA_CACHE_E2M1>::kStages;
  const int rs = a.cache.rec_shift, U = 1 << rs;
  const uint32_t rec_bytes = U * kRowE2m1;
  int page = 0, page_next = 0;
  // asks for the records of the warp's tile number x
  const auto ask = [&](int x) {
    const int k = warp + kLoadWarps * x, tile = u.tile(k);
    if (x % 4 == 0) page_next = look(a, u, sh, lane, k);
    const int from = __shfl_sync(kFull, page_next, ((x % 4) * 8 + lane) & 31);
    const bool there = lane < kKeys >> rs && from < a.cache.n_pages;
    const uint32_t bytes = __popc(__ballot_sync(kFull, there)) * rec_bytes;
    uint64_t* bar = &sh.landed[warp][x & 1];
    if (lane == 0) mbar_expect_tx(bar, bytes);
    __syncwarp();
    if (there)
      bulk_load(raw + (x & 1) * kRawBytes + lane * rec_bytes,
                a.cache.pages + cache_record(a.cache, kRowE2m1, from, u.kv, tile * kKeys + (lane << rs)), rec_bytes,
                bar);
    if (lane == 0) sh.asked[warp].count = x + 1;
  };
  int x = 0;
  if (warp < (int)u.n()) ask(0);
  for (unsigned k = warp; k < u.n(); k += kLoadWarps, ++x) {
    const unsigned st = k % kPStages;
    const int tile = u.tile(k);
    if (x % 4 == 0) page = page_next;
    if (k + kLoadWarps < u.n()) ask(x + 1);
    bool ok = k < kPStages || mbar_wait(&sh.empty[st], (k / kPStages - 1) & 1, &sh.abort);
    ok = ok && mbar_wait(&sh.landed[warp][x & 1], (x >> 1) & 1, &sh.abort);
    if (!__all_sync(kFull, ok)) return false;
    const bool mixed = mixed_tile(sh, tile);
    unsigned char* stage = stages + st * 2 * kTileBytes;
#pragma unroll 2
    for (int j = 0; j < 4; ++j) {
      const int row = 32 * j + lane, rec = row >> rs, in = row & (U - 1);
      const bool there = __shfl_sync(kFull, page, ((x % 4) * 8 + rec) & 31) < a.cache.n_pages;
      const unsigned char* r = raw + (x & 1) * kRawBytes + rec * rec_bytes;
      const uint4 c[2][2] = {{reinterpret_cast<const uint4*>(r + in * 32)[0],
                              reinterpret_cast<const uint4*>(r + in * 32)[1]},
                             {reinterpret_cast<const uint4*>(r + 36 * U + in * 32)[0],
                              reinterpret_cast<const uint4*>(r + 36 * U + in * 32)[1]}};
      // (a scale of zero makes zeros of whatever the codes are)
      uint32_t sc[2] = {there ? *reinterpret_cast<const uint32_t*>(r + 32 * U + in * 4) : 0u,
                        there ? *reinterpret_cast<const uint32_t*>(r + 68 * U + in * 4) : 0u};
      if (mixed) {  // NaN blocks of values that not all rows see become zeros (see scrub)
        if (is_scored(a) && unseen(sh, tile * kKeys + row)) sc[0] = 0u;
        uint32_t keep = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((sc[1] >> (8 * i) & 0x7fu) == 0x7fu) keep &= ~(0xffu << (8 * i));
        if (keep != 0xffffffffu) {
          sc[1] &= keep;
          const int key = tile * kKeys + row;
          if (key >= sh.lo_min && key < sh.hi_max) sh.odd = 1;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w[8] = {c[h][0].x, c[h][0].y, c[h][0].z, c[h][0].w, c[h][1].x, c[h][1].y, c[h][1].z, c[h][1].w};
        unsigned char* at = stage + h * kTileBytes + row * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 y, z;
          dequant16(w[2 * i], w[2 * i + 1], sc[h] >> (8 * i) & 0xffu, y, z);
          *reinterpret_cast<uint4*>(at + (((2 * i) ^ (row & 7)) << 4)) = y;
          *reinterpret_cast<uint4*>(at + (((2 * i + 1) ^ (row & 7)) << 4)) = z;
        }
      }
    }
    fence_async_proxy();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.full[st]);
  }
  return true;
}

// ------------------------------------------------------------------------------------------------ the MMA warps

// One thread issues the S products of both row tiles, another one the products with V: issuing takes as long as the
// products themselves, so that one thread for both would hold the next S back behind a product with V.
template <int KIND>
__device__ __forceinline__ bool multiply_s(const PromptUnit& u, PromptShared& sh, const unsigned char* q,
                                           const unsigned char* stages) {
  constexpr unsigned kPStages = PCfg<KIND>::kStages;
  const uint64_t dq = umma_desc_sw128(q);
  for (unsigned k = 0; k < u.n(); ++k) {
    const unsigned st = k % kPStages;
    if (!mbar_wait(&sh.full[st], (k / kPStages) & 1, &sh.abort)) return false;
    const uint64_t dk = umma_desc_sw128(stages + st * 2 * kTileBytes);
#pragma unroll
    for (int X = 0; X < 2; ++X) {
      if (k > 0 && !mbar_wait(&sh.s_free[X], (k - 1) & 1, &sh.abort)) return false;
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < 4; ++i)  // (16 dims are 32 bytes; descriptors count in 16)
        umma_ss(sh.tmem + 256 * X, dq + X * (kTileBytes / 16) + 2 * i, dk + 2 * i, PCfg<KIND>::kIdescS, i);
      umma_commit(&sh.s_full[X]);
    }
  }
  return true;
}

template <int KIND>
__device__ __forceinline__ bool multiply_v(const PromptUnit& u, PromptShared& sh, const unsigned char* stages) {
  constexpr unsigned kPStages = PCfg<KIND>::kStages;
  for (unsigned k = 0; k < u.n(); ++k) {
    const unsigned st = k % kPStages;
    if (!mbar_wait(&sh.full[st], (k / kPStages) & 1, &sh.abort)) return false;
    const uint64_t dv = umma_desc_mn128(smem_u32(stages + st * 2 * kTileBytes + kTileBytes));
#pragma unroll
    for (int X = 0; X < 2; ++X) {
      const uint32_t t = sh.tmem + 256 * X;
      if (!mbar_wait(&sh.p_full[X], k & 1, &sh.abort)) return false;
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < 8; ++i)  // (16 keys are 2048 bytes of V and 8 columns of P)
        umma_ts(t + 192, t + 128 + 8 * i, dv + 128 * i, PCfg<KIND>::kIdescO, k > 0 || i > 0);
      umma_commit(&sh.pv_done[X]);
    }
    umma_commit(&sh.empty[st]);  // (S of this tile is long done: its weights are here)
  }
  return true;
}

// ------------------------------------------------------------------------------------------------ softmax

struct PromptRow {
  int lo, hi;       // the row's span (empty where lo >= hi)
  float f;          // logit factor
  float m, l;       // reference and sum of weights
  // scored:
  CapRow cap;
  float slope;      // bias by distance, base 2
  int pos;          // the row's position
  // Biases are relative to the one of this token, as far before the position as the token in sight that is nearest to
  // it, or with a negative slope farthest from it: the row's largest one.
  int zero;
};

__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A new reference for the warp's rows, given each row's largest logit b: O and the sums of weights follow.  Returns
// false if the wait for the product before, which writes O, ran out.
template <int KIND>
__device__ __forceinline__ bool refer(PromptShared& sh, PromptRow& r, uint32_t s, int X, unsigned k, float b) {
  // (a step of 32 bits is too coarse for the shift from 2^24 on; nothing that it is for is left there)
  const float n = fmaxf(r.m, fabsf(b) < 16.f * kFar ? b - PCfg<KIND>::kShift : b);
  const float f = ex2_approx(r.m - n);
  if (k > 0) {
    if (!__all_sync(kFull, mbar_wait(&sh.pv_done[X], (k - 1) & 1, &sh.abort))) return false;
    tc_fence_after();
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      uint32_t o[32];
      tmem_ld32_now(s + 192 + 32 * h, o);
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
      tmem_st32(s + 192 + 32 * h, o);
    }
  }
  r.m = n;
  r.l *= f;
  return true;
}

template <int KIND>
__device__ __forceinline__ uint32_t pack_weights(float x, float y) {
  return KIND == PISA_CACHE_BF16 ? pack_bf16x2(x, y) : pack_f16x2(x, y);
}

// The softmax of one key tile, the k-th, for the warp's 32 rows, plain scores.  s: the tensor memory columns of the row
// tile at the warp's lanes.
template <int KIND>
__device__ __forceinline__ bool soften(PromptShared& sh, PromptRow& r, uint32_t s, int X, int lane, int tile,
                                       unsigned k, bool& two_step) {
  const int key0 = tile * kKeys;
  // (rows that see nothing do not matter: they get zeros at the end, or do not exist)
  const bool whole = __all_sync(kFull, r.lo >= r.hi || (r.lo <= key0 && r.hi >= key0 + kKeys));
  if (!__all_sync(kFull, mbar_wait(&sh.s_full[X], k & 1, &sh.abort))) return false;
  tc_fence_after();
  float v[kKeys], b;
  tmem_ld128_top<false>(s, v, b);
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(&sh.s_free[X]);  // S is in registers: the next product may overwrite it
  float ff = two_step ? 1.f : r.f;
  if (two_step || !whole) {
    if (two_step) {
#pragma unroll
      for (int i = 0; i < kKeys; ++i) v[i] = __fmul_rn(v[i], r.f);
    }
    if (!whole) {
      const int from = r.lo - key0, to = r.hi - key0;
#pragma unroll
      for (int i = 0; i < kKeys; ++i) v[i] = i >= from && i < to ? v[i] : -INFINITY;
    }
    float b1 = b = -INFINITY;
#pragma unroll
    for (int i = 0; i < kKeys; i += 4) {
      b = max3f(b, v[i], v[i + 1]);
      b1 = max3f(b1, v[i + 2], v[i + 3]);
    }
    b = fmaxf(b, b1);
  }
  b = __fmul_rn(b, ff);
  bool waited = k == 0;  // for the product before, which reads P and writes O
  // A row's reference m is set anew only when a logit passes it by more than kTop, so that few tiles rescale O.
  if (__any_sync(kFull, b > r.m + PCfg<KIND>::kTop)) {
    if (!refer<KIND>(sh, r, s, X, k, b)) return false;
    waited = true;
    // Below, a logit less m is an exact product less a rounded one: 2^-24 of m, no error as all weights of the row have
    // it, until it overflows a weight.  From kFar on the products are rounded first.
    if (!two_step && __any_sync(kFull, fabsf(r.m) >= kFar && r.m != kNone)) {
      two_step = true;
#pragma unroll
      for (int i = 0; i < kKeys; ++i) v[i] = __fmul_rn(v[i], r.f);
      ff = 1.f;
    }
  }
  const unsigned long long f2 = f2_pack(ff, ff), m2 = f2_pack(-r.m, -r.m);
  unsigned long long s0 = 0, s1 = 0;
  uint32_t w[32];
#pragma unroll
  for (int i = 0; i < kKeys / 2; ++i) {
    float x, y;
    f2_unpack(f2_fma(f2_pack(v[2 * i], v[2 * i + 1]), f2, m2), x, y);
    x = ex2_approx(x);
    y = ex2_approx(y);
    if (i & 1)
      s1 = f2_add(s1, f2_pack(x, y));
    else
      s0 = f2_add(s0, f2_pack(x, y));
    w[i & 31] = pack_weights<KIND>(x, y);
    // stored half a tile at a time (the product before may still read the last weights when the first are ready)
    if (i == 31 && !waited) {
      if (!__all_sync(kFull, mbar_wait(&sh.pv_done[X], (k - 1) & 1, &sh.abort))) return false;
      tc_fence_after();
    }
    if ((i & 31) == 31) tmem_st32(s + 128 + (i & 32), w);
  }
  float x, y;
  f2_unpack(f2_add(s0, s1), x, y);
  r.l += x + y;
  tmem_st_wait();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(&sh.p_full[X]);
  return true;
}

// The same for scores that are not plain products.  What bounds it is the arithmetic units: two packed operations take
// four clocks a scheduler, so that a cap's short polynomial (5 a pair) and the sums take 1536 for the two warps' rows,
// next to 1024 of the exponentials.  So both stand in one block, where one unit works beside the other (apart: 240
// instead of 208 us for 1216 tokens at 16384), and the row's factors are in the polynomial's coefficients (7 a pair:
// 231).
// The usual tile (whole, within the short polynomial or a line, no new reference) comes from the registers that
// its maximum came with (read once more: 208 instead of 182 us, with slopes 173 instead of 161).  The rest is a loop
// over 64 columns, which reads S again: the longer forms unrolled over all 128 do not fit the instruction cache.  (A
// shorter polynomial up to a quarter of the cap: 168 instead of 177 us where it is enough, 321 instead of 269 where all
// forms take turns.)
// a kernel for each: with all forms in one the usual ones have fewer registers (231 instead of 211 us)
enum PromptMode {
  kPromptPlain,
  kPromptCapped,  // a cap of kCapExp or less
  kPromptBias,
  kPromptEither,  // a larger cap, or a cap and a bias
};
enum ScoreForm {
  kCapHalf,     // capped, |score| at most half the cap: a short polynomial
  kCapWhole,    // capped, |score| at most the cap: a longer one
  kCapFar,      // capped at kCapExp or less: exponentials
  kCapAny,      // capped at more: either, and a choice
  kCapFarBias,  // the last two with a bias
  kCapAnyBias,
  kLine,        // a bias, where no row of the warp sees a later token than its own: a line
  kCapLine,     // kCapHalf with such a bias
  kBias,        // a bias
};

// Products of a row, of the keys from key0 on, as logits less a reference (m2: minus the reference, twice).
template <ScoreForm FORM>
struct Logits {
  static constexpr bool kAny = FORM == kCapAny || FORM == kCapAnyBias;
  static constexpr bool kFarther = FORM == kCapFar || FORM == kCapFarBias || kAny;
  static constexpr bool kAway = FORM == kCapFarBias || FORM == kCapAnyBias || FORM == kBias;
  static constexpr bool kHalf = FORM == kCapHalf || FORM == kCapLine, kStraight = FORM == kLine || FORM == kCapLine;
  static constexpr int n = kHalf ? TanhHalf::n : FORM == kCapWhole || kAny ? Tanh::n : 1;
  unsigned long long f, two, top2, c, p[n];
  float top1, slope, d0, least;

  __device__ __forceinline__ Logits(const CachePromptLaunch& a, const PromptRow& r, int key0, unsigned long long m2) {
    const float top = a.score.cap * kLog2e;
    c = m2;
    if constexpr (kHalf) {
      const CapPoly q = cap_poly(r.cap);
#pragma unroll
      for (int i = 0; i < n; ++i) p[i] = f2_pack(q.c[i], q.c[i]);
    } else if constexpr (FORM == kCapWhole || kAny) {
      constexpr Tanh k;
      f = f2_pack(r.cap.to_y, r.cap.to_y);
#pragma unroll
      for (int i = 0; i < n; ++i) p[i] = f2_pack(top * k.c[i], top * k.c[i]);
    } else if constexpr (FORM == kLine || FORM == kBias) {
      f = f2_pack(r.f, r.f);
    }
    if constexpr (kFarther) {
      const float x = 2.f * kLog2e * r.cap.to_y;
      two = f2_pack(x, x);
      top2 = f2_pack(-2.f * top, -2.f * top);
      c = f2_add(m2, f2_pack(top, top));
    }
    if constexpr (kStraight) {
      const float bias = r.slope * (float)(key0 - r.zero);  // of the first key
      slope = r.slope;
      c = f2_add(m2, f2_pack(bias, bias));
    }
    if constexpr (kAway) {
      // -slope (|j - p| - (p - zero)): whole numbers, exact up to 2^24.  Both distances less what all keys of the tile
      // have of the second, so that they are small where their difference is.
      const int d = key0 - r.pos, away = r.pos - r.zero, both = min(max(max(d, 1 - kKeys - d), 0), away);
      slope = -r.slope;
      d0 = (float)(d < 0 ? d + both : d - both);
      least = (float)(away - both);
    }
    if constexpr (kAny || kAway) c = m2;
    top1 = top;
  }

  // those of the keys key0 + i and the next
  __device__ __forceinline__ unsigned long long operator()(int i, float v, float w) const {
    const unsigned long long x = f2_pack(v, w);
    unsigned long long z = 0;
    unsigned long long add = c;
    if constexpr (kStraight) add = f2_fma(f2_pack(slope, slope), f2_pack((float)i, (float)(i + 1)), c);
    if constexpr (FORM == kLine) z = f2_fma(x, f, add);
    if constexpr (FORM == kBias) z = f2_mul(x, f);
    if constexpr (kFarther) {  // (as cap_exp; the reference in its last step where nothing else follows)
      float e, g;
      f2_unpack(f2_mul(x, two), e, g);
      f2_unpack(f2_add(f2_pack(ex2_approx(e), ex2_approx(g)), f2_pack(1.f, 1.f)), e, g);
      z = f2_fma(f2_pack(rcp_approx(e), rcp_approx(g)), top2, FORM == kCapFar ? c : f2_pack(top1, top1));
    }
    if constexpr (kHalf || FORM == kCapWhole || kAny) {
      const unsigned long long y = kHalf ? x : f2_mul(x, f), u = f2_mul(y, y);
      unsigned long long q = p[n - 1];
#pragma unroll
      for (int j = n - 2; j >= 0; --j) q = f2_fma(q, u, p[j]);
      if constexpr (kAny) {
        float y0, y1, z0, z1, q0, q1;
        f2_unpack(y, y0, y1);
        f2_unpack(z, z0, z1);
        f2_unpack(f2_mul(y, q), q0, q1);
        z = f2_pack(fabsf(y0) <= 1.f ? q0 : z0, fabsf(y1) <= 1.f ? q1 : z1);
      } else {
        z = f2_fma(y, q, add);
      }
    }
    if constexpr (kAway) {
      float z0, z1;
      f2_unpack(z, z0, z1);
      z = f2_pack(fmaf(slope, fabsf(d0 + (float)i) - least, z0), fmaf(slope, fabsf(d0 + (float)(i + 1)) - least, z1));
    }
    if constexpr (kAny || kAway) z = f2_add(z, c);
    return z;
  }
};

// The form as a constant, to use.
template <ScoreForm FORM, typename Use>
__device__ __forceinline__ void use_form(const Use& use) {
  use(std::integral_constant<ScoreForm, FORM>());
}
template <PromptMode MODE, typename Use>
__device__ __forceinline__ void with_form(ScoreForm form, const Use& use) {
  if constexpr (MODE == kPromptBias) {
    if (form == kLine) return use_form<kLine>(use);
    return use_form<kBias>(use);
  } else {
    if (form == kCapHalf) return use_form<kCapHalf>(use);
    if (form == kCapWhole) return use_form<kCapWhole>(use);
    if constexpr (MODE == kPromptCapped) return use_form<kCapFar>(use);
    if (form == kCapAny) return use_form<kCapAny>(use);
    if (form == kCapLine) return use_form<kCapLine>(use);
    if (form == kCapFarBias) return use_form<kCapFarBias>(use);
    return use_form<kCapAnyBias>(use);
  }
}

// 64 of them, masked.
template <PromptMode MODE>
__device__ __forceinline__ void logits64(const CachePromptLaunch& a, const PromptRow& r, ScoreForm form, bool whole,
                                         int key0, unsigned long long m2, float (&v)[64]) {
  with_form<MODE>(form, [&](auto f) {
    const Logits<f()> logits(a, r, key0, m2);
#pragma unroll
    for (int i = 0; i < 64; i += 2) f2_unpack(logits(i, v[i], v[i + 1]), v[i], v[i + 1]);
  });
  if (!whole) {
    const int from = r.lo - key0, to = r.hi - key0;
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = i >= from && i < to ? v[i] : -INFINITY;
  }
}

// The sum of a tile's weights, and the weights of 64 products at a time.
template <int KIND>
struct Weights {
  unsigned long long s0 = 0, s1 = 0;
  uint32_t w[32];
  __device__ __forceinline__ void operator()(int i, unsigned long long logits) {  // of the keys 2 i and 2 i + 1
    float x, y;
    f2_unpack(logits, x, y);
    x = ex2_approx(x);
    y = ex2_approx(y);
    if (i & 1)
      s1 = f2_add(s1, f2_pack(x, y));
    else
      s0 = f2_add(s0, f2_pack(x, y));
    w[i & 31] = pack_weights<KIND>(x, y);
  }
};

template <int KIND, PromptMode MODE>
__device__ __forceinline__ bool soften_scored(const CachePromptLaunch& a, PromptShared& sh, PromptRow& r, uint32_t s,
                                              int X, int lane, int tile, unsigned k) {
  const int key0 = tile * kKeys;
  const bool whole = __all_sync(kFull, r.lo >= r.hi || (r.lo <= key0 && r.hi >= key0 + kKeys));
  constexpr bool cap = MODE != kPromptBias;
  const bool slopes = MODE == kPromptBias || (MODE == kPromptEither && a.score.slopes);
  if (!__all_sync(kFull, mbar_wait(&sh.s_full[X], k & 1, &sh.abort))) return false;
  tc_fence_after();
  float all[kKeys], size;  // the products, and the largest one's magnitude
  tmem_ld128_top<true>(s, all, size);
  const bool in_range = r.cap.to_y <= kCapMost && (KIND == PISA_CACHE_E2M1 || r.cap.to_y >= kCapLeast);
  const bool half = cap && !__any_sync(kFull, !in_range || size * r.cap.to_y > 0.5f);
  // at least the row's largest logit (a cap makes none larger)
  float b = size * r.f;
  if (cap && !half) b = cap_any(size, r.cap, a.score.cap * kLog2e);
  bool line = false;
  if (slopes) {
    const int d0 = key0 - r.pos, d1 = d0 + kKeys - 1, near = max(max(d0, -d1), 0), most = max(abs(d0), abs(d1));
    const float top = r.slope * (float)(r.pos - r.zero - (r.slope > 0.f ? near : most));  // the tile's largest bias
    const float span = fabsf(r.slope) * (float)(kKeys - 1);
    // (rows that see no later tokens than their own: such are masked; from kFar on, an exact logit less a rounded
    // reference may be far from zero for the largest, see soften, and so it is below -kFar, where the reference is of a
    // piece of far tiles alone)
    line = !__any_sync(kFull, b >= kFar || fabsf(top) + span >= kFar || (d1 > 0 && r.hi > r.pos + 1));
    b += top;
  }
  ScoreForm form = line ? kLine : kBias;
  if (cap && slopes)
    form = half && line ? kCapLine : a.score.cap <= kCapExp ? kCapFarBias : kCapAnyBias;
  else if (half)
    form = kCapHalf;
  else if (cap && !__any_sync(kFull, size * r.cap.to_y > 1.f))
    form = kCapWhole;
  else if (cap)
    form = a.score.cap <= kCapExp ? kCapFar : kCapAny;
  bool waited = k == 0;
  const bool over = __any_sync(kFull, b > r.m + PCfg<KIND>::kTop);
  Weights<KIND> weigh;
  const auto store = [&](int h) {
    if (!waited) {
      if (!__all_sync(kFull, mbar_wait(&sh.pv_done[X], (k - 1) & 1, &sh.abort))) return false;
      tc_fence_after();
      waited = true;
    }
    tmem_st32(s + 128 + 32 * h, weigh.w);
    return true;
  };
  const auto release = [&] {  // S is in registers: the next product may overwrite it
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.s_free[X]);
  };
  // The usual tile; false: a wait ran out.
  const auto at_once = [&](auto f) {
    release();
    const Logits<f()> logits(a, r, key0, f2_pack(-r.m, -r.m));
#pragma unroll
    for (int i = 0; i < kKeys / 2; ++i) {
      weigh(i, logits(2 * i, all[2 * i], all[2 * i + 1]));
      if ((i & 31) == 31 && !store(i >> 5)) return false;
    }
    return true;
  };
  constexpr ScoreForm kUsual = MODE == kPromptBias ? kLine : MODE == kPromptCapped ? kCapHalf : kCapLine;
  using Usual = std::integral_constant<ScoreForm, kUsual>;
  if (whole && !over && form == Usual()) {
    if (!at_once(Usual())) return false;
  } else if (MODE == kPromptEither && whole && !over && form == kCapHalf) {
    if (!at_once(std::integral_constant<ScoreForm, kCapHalf>())) return false;
  } else {
    if (over) {
      b = -INFINITY;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        float v[64];
        tmem_ld64_now(s + 64 * h, v);
        logits64<MODE>(a, r, form, whole, key0 + 64 * h, 0, v);
#pragma unroll
        for (int i = 0; i < 64; i += 2) b = max3f(b, v[i], v[i + 1]);
      }
      if (__any_sync(kFull, b > r.m + PCfg<KIND>::kTop)) {
        if (!refer<KIND>(sh, r, s, X, k, b)) return false;
        waited = true;
      }
    }
    const unsigned long long m2 = f2_pack(-r.m, -r.m);
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      float v[64];
      tmem_ld64_now(s + 64 * h, v);
      if (h == 1) release();
      if (whole) {
        with_form<MODE>(form, [&](auto f) {
          const Logits<f()> logits(a, r, key0 + 64 * h, m2);
#pragma unroll
          for (int i = 0; i < 32; ++i) weigh(i, logits(2 * i, v[2 * i], v[2 * i + 1]));
        });
      } else {
        logits64<MODE>(a, r, form, whole, key0 + 64 * h, m2, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) weigh(i, f2_pack(v[2 * i], v[2 * i + 1]));
      }
      if (!store(h)) return false;
    }
  }
  float x, y;
  f2_unpack(f2_add(weigh.s0, weigh.s1), x, y);
  r.l += x + y;
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
    if (!mixed_tile(sh, tile)) continue;
    for (int key = max(tile * kKeys, r.lo); key < min((tile + 1) * kKeys, r.hi); ++key) {
      const int page = a.cache.table[(long long)u.b * a.cache.max_pages + (key >> a.cache.page_shift)];
      if (page < 0 || page >= a.cache.n_pages) continue;
      const int in = key & (U - 1);
      if (KIND == PISA_CACHE_BF16) {
        const unsigned char* v = a.cache.pages + cache_record(a.cache, kRowBf16, page, u.kv, key) + U * 128 + in * 128;
        v += 2 * d0;
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
        const unsigned char* s = a.cache.pages + cache_record(a.cache, kRowE2m1, page, u.kv, key) + 68 * U + in * 4;
        s += d0 / 16;
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

__device__ __forceinline__ void write_row(const CachePromptLaunch& a, const PromptUnit& u, int t, int head, float l,
                                          int d0, const float (&o)[32]) {
  const float f = l == 0.f ? 0.f : exp2i(a.cache.kind == PISA_CACHE_E2M1 ? a.cache.v_exp : 0) / l;
  uint4* dst = reinterpret_cast<uint4*>(a.out + (((long long)u.b * a.T + t) * a.Hq + head) * kD + d0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = l == 0.f ? 0u : pack_bf16x2(o[8 * i + 2 * j] * f, o[8 * i + 2 * j + 1] * f);
    dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ------------------------------------------------------------------------------------------------ the kernel

// The queries of the CTA's rows, by the softmax warps, eight threads a row and eight rows a thread ..
__device__ __forceinline__ void fetch_queries(const CachePromptLaunch& a, const PromptUnit& u, int count, int g_shift,
                                              uint4 (&x)[8]) {
  const int ch = threadIdx.x & 7;
#pragma unroll
  for (int it = 0; it < 8; ++it) {
    const int r = u.r0 + it * 32 + (threadIdx.x >> 3), t = r >> g_shift;
    x[it] = make_uint4(0, 0, 0, 0);
    if (t < count) {
      const int head = u.kv * a.G + (r & (a.G - 1));
      x[it] = *reinterpret_cast<const uint4*>(a.q.data + u.b * a.q.sb + (long long)t * a.q.st + head * a.q.sh + 8 * ch);
    }
  }
}

// .. as two swizzled operands.  4-bit pages: as fp16, the row scaled by a power of two so that its largest element lies
// in [1, 2) (cache_attend.cuh, make_q).
template <int KIND, PromptMode MODE>
__device__ __forceinline__ void stage_queries(const CachePromptLaunch& a, PromptShared& sh, unsigned char* q,
                                              const uint4 (&x)[8]) {
  const int ch = threadIdx.x & 7;
#pragma unroll
  for (int it = 0; it < 8; ++it) {
    const int row = it * 32 + (threadIdx.x >> 3);
    uint4 y = x[it];
    if (KIND == PISA_CACHE_E2M1) {
      uint32_t w[4] = {y.x, y.y, y.z, y.w}, m = 0;
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
      y = make_uint4(w[0], w[1], w[2], w[3]);
      constexpr float kFactor = MODE != kPromptPlain ? kScale : kScale * kLog2e;
      if (ch == 0) sh.factor[row] = fminf(kFactor * exp2i(e) * exp2i(a.cache.k_exp), 0x1.fffffep127f);
    }
    *reinterpret_cast<uint4*>(q + row * 128 + ((ch ^ (row & 7)) << 4)) = y;
  }
}

// Unit number x: the row tile and (sequence, KV head) that it is.
__device__ __forceinline__ void set_unit(const CachePromptLaunch& a, int x, int row_tiles, PromptUnit& u) {
  const int bk = x / row_tiles;
  u.b = bk / a.cache.Hkv;
  u.kv = bk - u.b * a.cache.Hkv;
  u.r0 = (x - bk * row_tiles) * kRowsCta;
}

// Key tiles of a unit whose rows see the tokens lo .. hi - 1 together.
__device__ __forceinline__ int tiles_of(int lo, int hi) { return lo < hi ? (hi + kKeys - 1) / kKeys - lo / kKeys : 0; }

// The stream form: key tiles of each unit, a warp a unit, where the spans are listed.
__global__ void __launch_bounds__(256) cache_prompt_tiles_kernel(CachePromptLaunch a, int g_shift, int row_tiles,
                                                                 int units) {
  after_the_one_before();
  const int x = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (x >= units) return;
  PromptUnit u;
  set_unit(a, x, row_tiles, u);
  const int count = prompt_count(a, u.b);
  int lo = INT_MAX, hi = 0;
  for (int t = (u.r0 >> g_shift) + lane; t < count && t <= (u.r0 + kRowsCta - 1) >> g_shift; t += 32) {
    bool over;
    const Span s = span_of(a, u.b, t, count, over);
    if (s.lo < s.hi) {
      lo = min(lo, s.lo);
      hi = max(hi, s.hi);
    }
  }
  lo = __reduce_min_sync(kFull, lo);
  hi = __reduce_max_sync(kFull, hi);
  if (lane == 0) a.plan.tiles[x] = tiles_of(lo, hi);
}

// The stream form's plan, by one CTA: the pieces in order of length, and for each run the unit that begins in it and
// goes on.  Unit x has the places from place[x] on, its tiles and kUnitEnd more; run r those from r per on.  A piece
// begins where a unit or a run does.
__global__ void __launch_bounds__(1024) cache_prompt_plan_kernel(CachePromptLaunch a, int g_shift, int row_tiles,
                                                                 int units) {
  constexpr int kBuckets = 256;
  __shared__ int place[kMaxUnits + 1], bucket[kBuckets], sums[32];
  after_the_one_before();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // places, by three scans of consecutive units a thread
  constexpr int kEach = (kMaxUnits + 1023) / 1024;
  int own[kEach], sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int x = tid * kEach + i;
    own[i] = 0;
    if (x < units) {
      int n;
      if (a.first || a.last) {
        n = a.plan.tiles[x];
      } else {  // the spans' ends move with the rows
        PromptUnit u;
        set_unit(a, x, row_tiles, u);
        const int count = prompt_count(a, u.b), t0 = u.r0 >> g_shift;
        const int t1 = min((u.r0 + kRowsCta - 1) >> g_shift, count - 1);
        bool over;
        n = t0 > t1 ? 0 : tiles_of(span_of(a, u.b, t0, count, over).lo, span_of(a, u.b, t1, count, over).hi);
      }
      own[i] = n + kUnitEnd;
    }
    sum += own[i];
  }
  int inc = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(kFull, inc, d);
    if (lane >= d) inc += y;
  }
  if (lane == 31) sums[warp] = inc;
  if (tid < kBuckets) bucket[tid] = 0;
  __syncthreads();
  int at = inc - sum;
  for (int w = 0; w < warp; ++w) at += sums[w];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int x = tid * kEach + i;
    if (x < units) place[x] = at;
    at += own[i];
    if (x == units - 1) place[units] = at;
  }
  __syncthreads();
  const int total = place[units], per = max((total + kRuns - 1) / kRuns, kMinRun);
  if (tid < kRuns) a.plan.cut[tid] = make_int2(-1, 0);
  __syncthreads();
  // the pieces: one begins with each unit, and one with each run
  const auto piece = [&](int j, PromptPiece& p) {  // false: nothing of it is left
    int begin, x;
    if (j < units) {
      x = j;
      begin = place[x];
    } else {
      begin = (j - units) * per;
      if (begin >= total) return false;
      int y = units;  // the last unit that begins at or before it
      x = 0;
      while (y - x > 1) {
        const int z = (x + y) >> 1;
        (place[z] <= begin ? x : y) = z;
      }
      if (place[x] == begin) return false;  // (the unit's own piece)
    }
    const int run = begin / per, all = place[x + 1] - place[x] - kUnitEnd, k0 = begin - place[x];
    const int k1 = min((run + 1) * per - place[x], all);
    if (k0 >= all && k0 > 0) return false;
    p.unit = x;
    p.k0 = k0;
    p.k1 = k1;
    p.slot = k0 == 0 && k1 == all ? -1 : 2 * run + (k0 == 0);
    if (k0 == 0 && k1 < all) a.plan.cut[run] = make_int2(x, (place[x] + all - 1) / per);
    return true;
  };
  constexpr int kPieces = (kMaxUnits + kRuns + 1023) / 1024;
  PromptPiece p[kPieces];
  int b[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int j = tid + 1024 * i;
    b[i] = -1;
    if (j < units + kRuns && piece(j, p[i])) {
      b[i] = kBuckets - 1 - (int)((long long)(p[i].k1 - p[i].k0) * (kBuckets - 1) / per);
      atomicAdd(&bucket[b[i]], 1);
    }
  }
  __syncthreads();
  if (warp == 0) {  // each bucket's first place
    int before = 0;
    for (int i = lane; i < kBuckets; i += 32) {
      const int n = bucket[i];
      int s = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(kFull, s, d);
        if (lane >= d) s += y;
      }
      bucket[i] = before + s - n;
      before += __shfl_sync(kFull, s, 31);
    }
    if (lane == 0) sums[0] = before;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    if (b[i] >= 0) a.plan.piece[atomicAdd(&bucket[b[i]], 1)] = p[i];
  for (int j = sums[0] + tid; j < units + kRuns; j += 1024) a.plan.piece[j].unit = -1;
}

// The softmax of a piece for the warp's rows, and its result: to the output, or to a partial result.
template <int KIND, PromptMode MODE, bool STREAM>
__device__ __forceinline__ bool soften_piece(const CachePromptLaunch& a, PromptShared& sh, PromptRow& r, int i1, int n,
                                             int g_shift) {
  const int lane = threadIdx.x & 31, X = threadIdx.x >> 7;
  const uint32_t s = sh.tmem + 256 * X + ((threadIdx.x >> 5 & 3) << 21);  // (the warp's lanes: 32 (warp % 4) ..)
  bool two_step = false;
  for (int k = 0; k < n; ++k)
    if (!(MODE != kPromptPlain ? soften_scored<KIND, MODE>(a, sh, r, s, X, lane, i1 - 1 - k, k)
                 : soften<KIND>(sh, r, s, X, lane, i1 - 1 - k, k, two_step)))
      return false;
  if (n > 0 && !__all_sync(kFull, mbar_wait(&sh.pv_done[X], (n - 1) & 1, &sh.abort))) return false;
  tc_fence_after();
  int row = threadIdx.x;
  asm volatile("" : "+r"(row));  // (what follows is computed here, not kept since the beginning)
  const PromptUnit u = sh.unit;
  const int t = (u.r0 + row) >> g_shift, head = u.kv * a.G + ((u.r0 + row) & (a.G - 1));
  float l = r.l;
  if (r.lo >= r.hi) l = 0.f;  // (its weights were never masked: see soften)
  if (sh.bad && sees_bad(a, u, r)) {
    l = __int_as_float(0x7fc00000);
    set_status(a.status, PISA_ERR_DEVICE_BOUNDS);
  }
  float* part = STREAM && sh.slot >= 0 ? a.part + (size_t)sh.slot * kRowsCta * kPartRow + row : nullptr;
  const bool there = t < prompt_count(a, u.b);
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
    if (part) {
#pragma unroll
      for (int i = 0; i < 32; ++i) part[(32 * h + i) * kRowsCta] = o[i];
    } else if (there) {
      write_row(a, u, t, head, l, 32 * h, o);
    }
  }
  if (part) {
    part[64 * kRowsCta] = r.m;
    part[65 * kRowsCta] = l;
  }
  tc_fence_before();
  return true;
}

template <int KIND, PromptMode MODE, bool STREAM>
__global__ void __launch_bounds__(kPromptThreads, 1)
    cache_prompt_kernel(const __grid_constant__ CUtensorMap map, CachePromptLaunch a, int g_shift, int row_tiles,
                        int units) {
  extern __shared__ unsigned char prompt_smem[];
  __shared__ PromptShared sh;
  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  unsigned char* q = prompt_smem + ((1024 - (smem_u32(prompt_smem) & 1023)) & 1023);
  unsigned char* stages = q + 2 * kTileBytes;
  if (threadIdx.x == 0) {
    for (int i = 0; i < PCfg<KIND>::kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int X = 0; X < 2; ++X) {
      mbar_init(&sh.s_full[X], 1);
      mbar_init(&sh.s_free[X], 4);
      mbar_init(&sh.p_full[X], 4);
      mbar_init(&sh.pv_done[X], 1);
      mbar_init(&sh.drain[X], 1);
    }
    for (int i = 0; i < 2 * kLoadWarps; ++i) mbar_init(&sh.landed[i >> 1][i & 1], 1);
    mbar_fence_init();
    sh.abort = sh.odd = sh.bad = 0;
    sh.lo_min = sh.hi_min = INT_MAX;
    sh.lo_max = sh.hi_max = 0;
    for (int i = 0; i < kLoadWarps; ++i) sh.asked[i] = Asked{0, 0};
  }
  after_the_one_before();
  PromptPiece piece = {0, 0, INT_MAX, -1};
  if constexpr (STREAM) {
    piece = a.plan.piece[blockIdx.x];
    if (piece.unit < 0) return;
  } else {  // the longest row tiles first
    const int heads = units / row_tiles;
    piece.unit = (int)(blockIdx.x % heads) * row_tiles + row_tiles - 1 - (int)(blockIdx.x / heads);
  }
  if (warp == kSoftWarps + kLoadWarps) tmem_alloc<512>(&sh.tmem);  // (held by no kernel that waits for another one)
  PromptUnit u;
  set_unit(a, piece.unit, row_tiles, u);
  const int count = prompt_count(a, u.b);
  PromptRow r{};
  uint4 queries[8];
  if (warp < kSoftWarps) {
    fetch_queries(a, u, count, g_shift, queries);  // (on their way while the spans come)
    const int row = u.r0 + threadIdx.x, t = row >> g_shift;
    if (t < count) {
      bool over;
      const Span s = span_of(a, u.b, t, count, over);
      if (over) set_status(a.status, PISA_ERR_DEVICE_BOUNDS);
      r.lo = s.lo;
      r.hi = s.hi;
      if (MODE != kPromptPlain && a.score.slopes) {
        r.slope = slope2(a.score, u.kv * a.G + (row & (a.G - 1)));
        r.pos = s.pos;
        r.zero = s.pos - (r.slope < 0.f ? max(abs(s.pos - s.lo), abs(s.pos - s.hi + 1))
                                        : abs(s.pos - max(min(s.pos, s.hi - 1), s.lo)));
      }
    }
    r.m = kNone;
  }
  __syncthreads();
  if (warp < kSoftWarps) {
    const bool sees = r.lo < r.hi;
    const int lo_min = __reduce_min_sync(kFull, sees ? r.lo : INT_MAX);
    const int lo_max = __reduce_max_sync(kFull, sees ? r.lo : 0);
    const int hi_min = __reduce_min_sync(kFull, sees ? r.hi : INT_MAX);
    const int hi_max = __reduce_max_sync(kFull, sees ? r.hi : 0);
    if (lane == 0) {
      atomicMin(&sh.lo_min, lo_min);
      atomicMax(&sh.lo_max, lo_max);
      atomicMin(&sh.hi_min, hi_min);
      atomicMax(&sh.hi_max, hi_max);
    }
    stage_queries<KIND, MODE>(a, sh, q, queries);
    fence_async_proxy();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  u.i0 = sh.lo_min < sh.hi_max ? sh.lo_min / kKeys : 0;
  u.i1 = sh.lo_min < sh.hi_max ? (sh.hi_max + kKeys - 1) / kKeys : 0;
  // the piece of it
  u.i1 -= min(piece.k0, u.i1 - u.i0);
  u.i0 = max(u.i0, u.i1 - (piece.k1 - piece.k0));
  if (threadIdx.x == 0) {
    sh.unit = u;
    sh.slot = piece.slot;
  }
  __syncthreads();
  bool ok = true;
  // More registers for the softmax, whose scores spilled (1216 tokens at 16384 136 -> 132 us, 4 bits 151 -> 143): 8 x
  // 32 x 200 + 4 x 32 x 96 of the 384 x 168 that the CTA has.
  if (warp < kSoftWarps)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
  if (warp < kSoftWarps) {
    r.f = KIND == PISA_CACHE_E2M1 ? sh.factor[threadIdx.x] : MODE != kPromptPlain ? kScale : kScale * kLog2e;
    if (MODE != kPromptPlain) {
      r.cap = cap_row(r.f, a.score.inv_cap);
      r.f = r.cap.to_l;
    }
    ok = soften_piece<KIND, MODE, STREAM>(a, sh, r, u.i1, u.n(), g_shift);
  } else if (warp < kSoftWarps + kLoadWarps) {
    const int w = warp - kSoftWarps;
    if constexpr (KIND == PISA_CACHE_BF16)
      ok = load_bf16(a, &map, u, sh, stages, w, lane);
    else
      ok = load_e2m1(a, u, sh, stages, stages + 2 * PCfg<KIND>::kStages * kTileBytes + 2 * w * kRawBytes, w, lane);
  } else if (lane == 0) {
    const int Y = warp - kSoftWarps - kLoadWarps;
    ok = Y == 0 ? multiply_s<KIND>(u, sh, q, stages) : multiply_v<KIND>(u, sh, stages);
    if (!ok) {  // its products end before tensor memory is given back
      umma_commit(&sh.drain[Y]);
      mbar_wait(&sh.drain[Y], 0, nullptr);
    }
  }
  if (!ok) {  // a wait ran out: the others give up, too
    *const_cast<volatile int*>(&sh.abort) = 1;
    set_status(a.status, PISA_ERR_DEVICE_TIMEOUT);
  }
  __syncthreads();
  if (sh.abort && warp >= kSoftWarps && warp < kSoftWarps + kLoadWarps && lane == 0) {
    // given up: copies that are still on their way land before the shared memory is let go
    const Asked asked = sh.asked[warp - kSoftWarps];
    const int w = warp - kSoftWarps;
    if (KIND == PISA_CACHE_BF16) {
      for (int i = 0; i < PCfg<KIND>::kStages; ++i)
        if (asked.stages >> i & 1) mbar_wait(&sh.full[i], asked.stages >> (8 + i) & 1, nullptr);
    } else {
      for (unsigned i = asked.count > 2 ? asked.count - 2 : 0; i < asked.count; ++i)
        mbar_wait(&sh.landed[w][i & 1], (i >> 1) & 1, nullptr);
    }
  }
  __syncthreads();
  if (warp == kSoftWarps + kLoadWarps) tmem_dealloc<512>(sh.tmem);
}

// Joins the partial results of the units that lie in several runs: those of the unit that begins in run c and goes on.
// Sixteen CTAs a run, sixteen rows each; a thread has 16 dims of a row and every fourth partial result.
__global__ void __launch_bounds__(256) cache_prompt_join_kernel(CachePromptLaunch a, int g_shift, int row_tiles) {
  __shared__ float so[4][16][4][17];
  __shared__ float sm[4][16], sl[4][16];
  after_the_one_before();
  const int c = blockIdx.x >> 4;
  const int2 cut = a.plan.cut[c];
  if (cut.x < 0) return;
  PromptUnit u;
  set_unit(a, cut.x, row_tiles, u);
  const int row_in = threadIdx.x & 15, quad = (threadIdx.x >> 4) & 3, grp = threadIdx.x >> 6;
  const int row = (blockIdx.x & 15) * 16 + row_in;
  float m = -INFINITY, l = 0.f, o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  for (int i = c + grp; i <= cut.y; i += 4) {
    const float* p = a.part + ((size_t)i * 2 + (i == c)) * kRowsCta * kPartRow + row;
    const float mi = p[64 * kRowsCta], li = p[65 * kRowsCta];
    float y[16];
#pragma unroll
    for (int d = 0; d < 16; ++d) y[d] = p[(16 * quad + d) * kRowsCta];
    const float n = fmaxf(m, mi), f = ex2_approx(m - n), h = ex2_approx(mi - n);
    m = n;
    l = l * f + li * h;
#pragma unroll
    for (int d = 0; d < 16; ++d)  // (what a part without keys holds is nothing)
      o[d] = li == 0.f ? o[d] * f : o[d] * f + y[d] * h;
  }
  sm[grp][row_in] = m;
  sl[grp][row_in] = l;
#pragma unroll
  for (int d = 0; d < 16; ++d) so[grp][row_in][quad][d] = o[d];
  __syncthreads();
  if (grp) return;
  const int r = u.r0 + row, t = r >> g_shift;
  if (t >= prompt_count(a, u.b)) return;
#pragma unroll
  for (int x = 1; x < 4; ++x) m = fmaxf(m, sm[x][row_in]);
  l = 0.f;
#pragma unroll
  for (int d = 0; d < 16; ++d) o[d] = 0.f;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const float lx = sl[x][row_in], f = lx == 0.f ? 0.f : ex2_approx(sm[x][row_in] - m);
    l += lx == 0.f ? 0.f : lx * f;
#pragma unroll
    for (int d = 0; d < 16; ++d) o[d] += lx == 0.f ? 0.f : so[x][row_in][quad][d] * f;
  }
  const float f = l == 0.f ? 0.f : exp2i(a.cache.kind == PISA_CACHE_E2M1 ? a.cache.v_exp : 0) / l;
  const long long at = ((long long)u.b * a.T + t) * a.Hq + u.kv * a.G + (r & (a.G - 1));
  uint4* dst = reinterpret_cast<uint4*>(a.out + at * kD + 16 * quad);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = l == 0.f ? 0u : pack_bf16x2(o[8 * i + 2 * j] * f, o[8 * i + 2 * j + 1] * f);
    dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

size_t cache_prompt_part_bytes() { return kPromptPlanBytes + (size_t)kRuns * 2 * kRowsCta * kPartRow * 4; }

// Whether the stream form takes a call: `units` row tiles that see up to `tiles` key tiles each.  A CTA for each unit
// takes as long as its last wave; the stream's CTAs end together, but the plan, the pieces' begins and the join cost it
// about as much as 16 tiles, and the lengths (known to the device alone) a tenth.
inline bool takes_stream(long long units, long long tiles) {
  if (units > kMaxUnits) return false;
  const long long waves = (units + kRuns - 1) / kRuns;
  return 10 * kRuns * waves * tiles > 11 * units * tiles + 160 * kRuns;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_tiled() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// bf16 pages as [page][head, record, K or V][token of the record][64], a box of one record's keys or values.
bool map_pages(CUtensorMap* m, const CacheDev& c) {
  const auto encode = encode_tiled();
  if (!encode) return false;
  const cuuint64_t U = 1ull << c.rec_shift;
  const cuuint64_t dims[4] = {kD, U, (cuuint64_t)c.Hkv << (c.page_shift - c.rec_shift + 1), (cuuint64_t)c.n_pages};
  const cuuint64_t strides[3] = {2 * kD, 2 * kD * U, (cuuint64_t)c.page_stride};
  const cuuint32_t box[4] = {kD, (cuuint32_t)U, 1, 1}, es[4] = {1, 1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, c.pages, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int KIND, PromptMode MODE>
static cudaError_t launch_prompt(const CachePromptLaunch& L, cudaStream_t s) {
  int g_shift = 0;
  while ((1 << g_shift) < L.G) ++g_shift;
  const int row_tiles = (int)(((long long)L.T * L.G + kRowsCta - 1) / kRowsCta);
  const int units = row_tiles * L.cache.B * L.cache.Hkv;
  CUtensorMap map{};
  if (KIND == PISA_CACHE_BF16 && !map_pages(&map, L.cache)) return cudaErrorInvalidValue;
  long long keys = (long long)L.cache.max_pages << L.cache.page_shift;  // what a unit sees at most
  const long long reach = (long long)L.score.window + kRowsCta / L.G;
  if (!L.last && keys > reach) keys = reach;
  constexpr int kSmem = PCfg<KIND>::kSmem;
  if (!takes_stream(units, keys / kKeys))
    return launch_early<cache_prompt_kernel<KIND, MODE, false>>((unsigned)units, kPromptThreads, kSmem, s, map, L,
                                                                g_shift, row_tiles, units);
  cudaError_t e = cudaSuccess;
  if (L.first || L.last)
    e = launch_early<cache_prompt_tiles_kernel>((unsigned)(units + 7) / 8, 256, 0, s, L, g_shift, row_tiles, units);
  if (e == cudaSuccess) e = launch_early<cache_prompt_plan_kernel>(1, 1024, 0, s, L, g_shift, row_tiles, units);
  if (e != cudaSuccess) return e;
  e = launch_early<cache_prompt_kernel<KIND, MODE, true>>((unsigned)(units + kRuns), kPromptThreads, kSmem, s, map, L,
                                                          g_shift, row_tiles, units);
  if (e != cudaSuccess) return e;
  return launch_early<cache_prompt_join_kernel>(kRuns * 16, 256, 0, s, L, g_shift, row_tiles);
}

template <int KIND>
static cudaError_t launch_prompt_mode(const CachePromptLaunch& L, cudaStream_t s) {
  if (L.score.cap <= 0.f)
    return L.score.slopes ? launch_prompt<KIND, kPromptBias>(L, s) : launch_prompt<KIND, kPromptPlain>(L, s);
  if (L.score.slopes || L.score.cap > kCapExp) return launch_prompt<KIND, kPromptEither>(L, s);
  return launch_prompt<KIND, kPromptCapped>(L, s);
}

cudaError_t launch_cache_prompt(const CachePromptLaunch& L, cudaStream_t s) {
  return L.cache.kind == PISA_CACHE_BF16 ? launch_prompt_mode<PISA_CACHE_BF16>(L, s)
                                         : launch_prompt_mode<PISA_CACHE_E2M1>(L, s);
}

}  // namespace pisa
