// cache_attend.cuh -- attention of a sequence's newest tokens over its paged KV cache, all of
// it or the blocks that a selection listed; pages in bf16 or 4 bits.
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = exp(q . k_j / 8 - max_j)
// in one pass over the keys with a running maximum and sum per row (32 bits, base 2).
//
// The 16 rows of an mma.sync m16n8k16 tile are the query heads of one KV head's group (and of
// several queries, where the group is smaller); every warp of a CTA takes its own tiles of
// keys, and the CTA's warps are merged through shared memory at the end.
//
// What bounds it.  Per key and KV head 72 or 256 bytes are read.  bf16 pages: the memory;
// 8 ragged sequences up to 131072 tokens (384 MB) take 62.2 us = 6.17 TB/s, and a plain
// read-only sweep of as many bytes 59.5 us.  4-bit pages: the arithmetic; 16 x 131072 tokens
// (302 MB) take 71.1 us = 4.25 TB/s.  A tile of 64 keys costs 64 HMMA of 8 clocks and 128 HMUL2
// of 2 on its scheduler, which do not overlap on this machine, beside 157 conversions and 37
// logic operations on the other pipe (which do): about 250 clocks of an SM a tile, of the 285
// that it takes; the tile's bytes take 196.
//
// Two forms (launch_attend chooses):
//   direct, 4 to 12 warps a CTA: one CTA per unit (sequence, KV head and query, or row tile),
//     for listed blocks and for short caches;
//   split: the tiles of all units form one stream, which is cut into runs of equal cost, one
//     per SM, whatever the lengths; a unit that ends up in several runs is joined by a second kernel
//     from 32-bit partial results.
#pragma once

#include <climits>

#include "cache.cuh"
#include "tc.cuh"

namespace pisa {

constexpr int kPartFloats = 16 * 64 + 32;  // a partial result: O [16][64], row maxima, row sums
constexpr int kCaGrid = 152;               // CTAs of the split form: one on each SM
constexpr int kCaMinTiles = 12;            // places of the stream that a run has at least
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -0x1.fffffep127f;  // the reference of a row that has seen no logit above minus infinity
constexpr float kFar = 0x1p22f;            // references from which on weigh takes differences in two steps

inline size_t part_bytes() { return (size_t)kCaGrid * 2 * kPartFloats * sizeof(float); }

template <int KIND>
struct Cfg;
template <>
struct Cfg<PISA_CACHE_BF16> {
  static constexpr int KT = 32;     // keys of a tile
  static constexpr int kWarps = 8;  // of the split form, one CTA on an SM
  static constexpr int kHalf = 4, kThird = 4;  // of the direct form where two CTAs, or more, share an SM
  static constexpr int kStages = 3;
  static constexpr int kRow = kRowBf16;
  // Whether the split form's CTAs take a run's row tiles side by side, one each, so that they read
  // the same pages at the same time; else the row tiles are units of the stream like others.
  // Side by side / in the stream, us a call, two KV heads, G = 16 unless said:
  //   bf16    4 x 65536 T = 2 31.6 / 44.5, T = 8 94.8 / 138   16 x 16384 T = 8, 8 heads, G = 4 101 / 158
  //           (T = 16 ragged 139 / 134, one short sequence T = 9 33.0 / 31.5)
  //   4 bits  4 x 65536 T = 2 25.4 / 25.3, T = 8 75.1 / 71.4 (bound by the arithmetic; some CTAs are left over)
  static constexpr bool kSide = true;
  static constexpr int kChange = 36;  // places of the stream that a unit's end counts as (see unit_places)
  static constexpr float kShift = 0.f;  // weights are held times 2^kShift
  static constexpr float kSlack = 20.f;  // how far (base 2) a logit may pass the row's reference
};
template <>
struct Cfg<PISA_CACHE_E2M1> {
  static constexpr int KT = 64;
  static constexpr int kWarps = 12;  // (a multiple of four: an SM's four schedulers share the warps out evenly)
  static constexpr int kHalf = 6, kThird = 4;
  static constexpr int kStages = 3;
  static constexpr int kRow = kRowE2m1;
  static constexpr bool kSide = false;
  static constexpr int kChange = 24;
  static constexpr float kShift = 10.f;
  static constexpr float kSlack = 5.f;
};
template <int KIND>
constexpr int kStageBytes = Cfg<KIND>::KT * Cfg<KIND>::kRow;
// A warp's own shared memory: a block list or the weights of 16 keys; from kFarAt on each lane's
// factors and references of rows that are far (see weigh); at kBadAt the first token that lies in a
// page out of range.
constexpr int kFarAt = 1024, kBadAt = kFarAt + 32 * 16, kScratch = kBadAt + 16;
static_assert(kFarAt >= 16 * 16 * 4 && kFarAt >= kCacheMaxSel * 4, "");

extern __shared__ __align__(128) unsigned char ca_smem[];
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void cpa16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(ca_smem) + dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cpa_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cpa_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int KIND>
__device__ __forceinline__ void ca_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  if (KIND == PISA_CACHE_BF16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_addr(ca_smem) + addr)
               : "memory");
}
__device__ __forceinline__ void ldm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_addr(ca_smem) + addr)
               : "memory");
}
// (plain loads, which the compiler may schedule; a is an offset into the dynamic shared memory)
__device__ __forceinline__ uint32_t lds32(uint32_t a) { return *reinterpret_cast<const uint32_t*>(ca_smem + a); }
__device__ __forceinline__ void lds64(uint32_t a, uint32_t& x, uint32_t& y) {
  const uint2 v = *reinterpret_cast<const uint2*>(ca_smem + a);
  x = v.x;
  y = v.y;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) { return ca_smem[a]; }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 16-byte chunk ch (0..7) of row r of a staged matrix of 128-byte rows
__device__ __forceinline__ uint32_t swz128(int r, int ch) { return (uint32_t)(r * 128 + ((ch ^ (r & 7)) << 4)); }

// Where a 16-key group of a staged 4-bit tile begins (records of U tokens one after another).
template <int U>
struct E2m1Tile {
  static __device__ __forceinline__ int rec(int i) { return (16 * i / U) * U * kRowE2m1; }
  static __device__ __forceinline__ int row(int i) { return (16 * i) % U; }
  static __device__ __forceinline__ int k(int i) { return rec(i) + row(i) * 32; }
  static __device__ __forceinline__ int ks(int i) { return rec(i) + 32 * U + row(i) * 4; }
  static __device__ __forceinline__ int v(int i) { return rec(i) + 36 * U + row(i) * 32; }
  static __device__ __forceinline__ int vs(int i) { return rec(i) + 68 * U + row(i) * 4; }
};

// One row tile's state in a warp: rows g and g + 8 of the MMA tile.
template <int KIND>
struct RowState {
  uint32_t qa[4][4];  // A fragments of the queries
  float f0, f1;       // logit factors of rows g and g + 8, base 2
  float m0, m1;       // the rows' references: weights are 2^(logit - m)
  bool far;           // some row of the warp is far: factors and references are in shared memory
  float l0, l1;       // this lane's share of the sums of the weights
  float o[8][4];
  bool bad;  // a page out of range was met
};

// Where dims 4 c .. 4 c + 3 of row r lie in a warp's 16 x 64 part of the merge buffer (floats).
// The order spreads what merge_warps writes, and what merged reads, over all banks: written row
// by row, the 4-bit form's stores met 16 to a bank and cost 0.5 to 1 us a call.
__device__ __forceinline__ int merge_at(int r, int c) {
  return r * 64 + 4 * (c ^ ((c >> 3) << 1) ^ (r & 1) ^ ((r & 3) << 1));
}

// A unit: the row tile of (sequence b, KV head kv) that starts at row r0.
struct Unit {
  int b, kv, r0, t_first;  // t_first: the query of row 0
  int rows;                // rows of (b, kv): queries * G
  int n;                   // tokens the sequence holds
  const int32_t* sel;      // listed blocks, or nullptr
};

// This lane's part of the query rows r0 + g and r0 + g + 8 of a unit (row r: query r / G,
// head r % G): dims 16 j .. 16 j + 15 of each.
struct QueryWords {
  uint32_t w[2][8];
};

__device__ __forceinline__ void fetch_q(const CacheAttendLaunch& a, const Unit& u, int lane, QueryWords& q) {
  const int g = lane >> 2, j = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = u.r0 + g + 8 * h;
    uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
    if (r < u.rows) {
      const int t = u.t_first + r / a.G, head = u.kv * a.G + r % a.G;
      const uint4* p =
          reinterpret_cast<const uint4*>(a.q.data + u.b * a.q.sb + (long long)t * a.q.st + head * a.q.sh) + 2 * j;
      x0 = p[0];
      x1 = p[1];
    }
    q.w[h][0] = x0.x; q.w[h][1] = x0.y; q.w[h][2] = x0.z; q.w[h][3] = x0.w;
    q.w[h][4] = x1.x; q.w[h][5] = x1.y; q.w[h][6] = x1.z; q.w[h][7] = x1.w;
  }
}

template <int KIND>
__device__ __forceinline__ void reset(RowState<KIND>& s) {
  s.m0 = s.m1 = kNone;
  s.far = false;
  s.l0 = s.l1 = 0.f;
  s.bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) s.o[i][0] = s.o[i][1] = s.o[i][2] = s.o[i][3] = 0.f;
}

// The A fragments of the queries and the logit factors.
// In the 4-bit form the products are taken in fp16: the row is scaled by a power of two so
// that its largest element lies in [1, 2), where fp16 holds all 8 bits of a bf16 down to
// 2^-17 of it and is off by at most 2^-25 of it below (the fp32 sums of the products are
// off by as much).  Rows above 2^126 lie in [1, 4), and so does what is finite in a row with an
// infinity; rows below 2^-100 have logits of zero, whatever becomes of them.  A factor of the
// logits that is past the range of 32 bits is cut to it: logits of zero stay so, and others, if
// they fit 32 bits at all, still differ by far more than weights can show.
template <int KIND>
__device__ __forceinline__ void make_q(const CacheAttendLaunch& a, const QueryWords& q, int lane, RowState<KIND>& s) {
  const int j = lane & 3;
  float f[2] = {kScale * kLog2e, kScale * kLog2e};
  if (KIND == PISA_CACHE_E2M1) {
    uint32_t w[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t t = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) t = __vmaxu2(t, q.w[h][i] & 0x7fff7fffu);
      t = max(t & 0xffffu, t >> 16);
      t = max(t, __shfl_xor_sync(kFull, t, 1));
      t = max(t, __shfl_xor_sync(kFull, t, 2));
      const int e = max(min((int)(t >> 7) - 127, 126), -100);  // the largest lies in [2^e, 2^(e + 1))
      const float down = exp2i(-e);
      f[h] = fminf(f[h] * exp2i(e) * exp2i(a.cache.k_exp), 0x1.fffffep127f);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[h][i] = pack_f16x2(__uint_as_float(q.w[h][i] << 16) * down, __uint_as_float(q.w[h][i] & 0xffff0000u) * down);
    }
    // k-step ks of lane j: dims 16 j + 4 ks .. + 3 (two words)
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      s.qa[ks][0] = w[0][2 * ks];
      s.qa[ks][1] = w[1][2 * ks];
      s.qa[ks][2] = w[0][2 * ks + 1];
      s.qa[ks][3] = w[1][2 * ks + 1];
    }
  } else {
    // ldmatrix gives k-step ks dims 16 ks + 2 j, + 1 and 16 ks + 8 + 2 j, + 1: word j (or 4 + j) of
    // lane ks's 16 dims, fetched by shuffle
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = __shfl_sync(kFull, q.w[h][i], (lane & 28) | ks);
          const uint32_t y = __shfl_sync(kFull, q.w[h][4 + i], (lane & 28) | ks);
          if (i == j) {
            lo = x;
            hi = y;
          }
        }
        s.qa[ks][h] = lo;
        s.qa[ks][2 + h] = hi;
      }
  }
  s.f0 = f[0];
  s.f1 = f[1];
}

// The key (of 16 in a group) behind column element (half h of the group, e) of lane j.
template <int KIND>
__device__ __forceinline__ int key_of(int h, int j, int e) {
  return KIND == PISA_CACHE_BF16 ? 8 * h + 2 * j + e : 8 * h + j + 4 * e;
}

// V fragments of 16-key group i: b[n][0..1] for the eight column tiles n.
template <int KIND, int U>
__device__ __forceinline__ void load_v(uint32_t st, int i, int lane, uint32_t (&vb)[8][2]) {
  const int g = lane >> 2, j = lane & 3;
  if (KIND == PISA_CACHE_E2M1) {
    using L = E2m1Tile<U>;
    const uint32_t av = st + L::v(i) + j * 32 + 4 * g, as = st + L::vs(i) + j * 4 + (g >> 1);
#pragma unroll
    for (int y = 0; y < 2; ++y) {  // keys j and j + 4, then j + 8 and j + 12
      const uint32_t wa = lds32(av + 256 * y), wb = lds32(av + 256 * y + 128);
      const uint32_t s2 = e4m3x2(__byte_perm(lds8(as + 32 * y), lds8(as + 32 * y + 16), 0x0040));
      // bytes whose nibbles are one dim of both keys
      const uint32_t even = (wa & 0x0f0f0f0fu) | (__funnelshift_l(wb, wb, 4) & 0xf0f0f0f0u);
      const uint32_t odd = ((wa >> 4) & 0x0f0f0f0fu) | (wb & 0xf0f0f0f0u);
      uint32_t d[4];
      e2m1x8(even, d);
#pragma unroll
      for (int x = 0; x < 4; ++x) vb[2 * x][y] = hmul2u(d[x], s2);
      e2m1x8(odd, d);
#pragma unroll
      for (int x = 0; x < 4; ++x) vb[2 * x + 1][y] = hmul2u(d[x], s2);
    }
  } else {
    const uint32_t sV = st + 32 * 128;
#pragma unroll
    for (int dp = 0; dp < 4; ++dp) {
      uint32_t r[4];
      ldm_x4_t(sV + swz128(16 * i + (lane & 7) + 8 * ((lane >> 3) & 1), 2 * dp + (lane >> 4)), r);
      vb[2 * dp][0] = r[0];
      vb[2 * dp][1] = r[1];
      vb[2 * dp + 1][0] = r[2];
      vb[2 * dp + 1][1] = r[3];
    }
  }
}

// Makes the values of a staged tile's keys from `limit` on count as zeros, whatever the
// memory holds (4 bits: a zero scale; a code is always finite).
template <int KIND, int U>
__device__ __forceinline__ void clear_v(uint32_t st, int lane, int limit) {
  constexpr int KT = Cfg<KIND>::KT;
#pragma unroll
  for (int x = 0; x < KT / 32; ++x) {
    const int key = lane + 32 * x;
    if (key < limit) continue;
    if (KIND == PISA_CACHE_E2M1) {
      using L = E2m1Tile<U>;
      *reinterpret_cast<uint32_t*>(ca_smem + st + L::vs(key >> 4) + (key & 15) * 4) = 0u;
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4*>(ca_smem + st + KT * 128 + key * 128 + 16 * c) = make_uint4(0, 0, 0, 0);
    }
  }
}

// Two neighbouring dims (2 d, 2 d + 1) of a staged key's value, in 32 bits.
template <int KIND, int U>
__device__ __forceinline__ float2 value2(uint32_t st, int key, int d) {
  constexpr int KT = Cfg<KIND>::KT;
  if (KIND == PISA_CACHE_E2M1) {
    using L = E2m1Tile<U>;
    const uint32_t c = lds8(st + L::v(key >> 4) + (key & 15) * 32 + d);
    const uint32_t f = e4m3x2(lds8(st + L::vs(key >> 4) + (key & 15) * 4 + (d >> 3)));
    uint32_t v[4];
    e2m1x8(c, v);
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&v[0]));
    const float s = __low2float(*reinterpret_cast<const __half2*>(&f));
    return make_float2(x.x * s, x.y * s);
  }
  const uint32_t w = lds32(st + KT * 128 + swz128(key, d >> 2) + 4 * (d & 3));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// The weights of a tile as A fragments of 16 keys each, in NP parts that add up to them.
template <int KIND, int NP>
struct Weights {
  uint32_t a[NP][Cfg<KIND>::KT / 16][4];
};

// The products of two tiles, their instructions side by side: the logits of the tile staged
// at st_k (QK), and O += P V for the tile staged at st_v with the weights w (PV).
template <int KIND, int U, int NP, bool QK, bool PV>
__device__ __forceinline__ void products(uint32_t st_k, uint32_t st_v, int lane, RowState<KIND>& s,
                                         float (&sc)[Cfg<KIND>::KT / 8][4], const Weights<KIND, NP>& w) {
  constexpr int KT = Cfg<KIND>::KT;
  const int g = lane >> 2, j = lane & 3;
#pragma unroll
  for (int i = 0; i < KT / 16; ++i) {
    if (QK) {
      float(&d0)[4] = sc[2 * i];
      float(&d1)[4] = sc[2 * i + 1];
      d0[0] = d0[1] = d0[2] = d0[3] = d1[0] = d1[1] = d1[2] = d1[3] = 0.f;
      if (KIND == PISA_CACHE_E2M1) {
        using L = E2m1Tile<U>;
        const int key = (g >> 1) + 4 * (g & 1);
        const uint32_t ak = st_k + L::k(i) + key * 32 + 8 * j, as = st_k + L::ks(i) + key * 4 + j;
        const uint32_t s2 = e4m3x2(__byte_perm(lds8(as), lds8(as + 32), 0x0040));
        const __half2 p = *reinterpret_cast<const __half2*>(&s2);
        const __half2 q0 = __low2half2(p), q1 = __high2half2(p);
        const uint32_t f0 = *reinterpret_cast<const uint32_t*>(&q0), f1 = *reinterpret_cast<const uint32_t*>(&q1);
        uint32_t x0, x1, y0, y1, b[4], c[4];
        lds64(ak, x0, x1);
        lds64(ak + 256, y0, y1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          e2m1x8(h ? x1 : x0, b);
          e2m1x8(h ? y1 : y0, c);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t(&q)[4] = s.qa[2 * h + k];
            ca_mma<KIND>(d0, q[0], q[1], q[2], q[3], hmul2u(b[2 * k], f0), hmul2u(b[2 * k + 1], f0));
            ca_mma<KIND>(d1, q[0], q[1], q[2], q[3], hmul2u(c[2 * k], f1), hmul2u(c[2 * k + 1], f1));
          }
        }
      } else {
#pragma unroll
        for (int kp = 0; kp < 2; ++kp) {
          uint32_t b[4], c[4];
          ldm_x4(st_k + swz128(16 * i + (lane & 7), 4 * kp + (lane >> 3)), b);
          ldm_x4(st_k + swz128(16 * i + 8 + (lane & 7), 4 * kp + (lane >> 3)), c);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t(&q)[4] = s.qa[2 * kp + k];
            ca_mma<KIND>(d0, q[0], q[1], q[2], q[3], b[2 * k], b[2 * k + 1]);
            ca_mma<KIND>(d1, q[0], q[1], q[2], q[3], c[2 * k], c[2 * k + 1]);
          }
        }
      }
    }
    if (PV) {
      uint32_t vb[8][2];
      load_v<KIND, U>(st_v, i, lane, vb);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const uint32_t(&a)[4] = w.a[p][i];
#pragma unroll
        for (int n = 0; n < 8; ++n) ca_mma<KIND>(s.o[n], a[0], a[1], a[2], a[3], vb[n][0], vb[n][1]);
      }
    }
  }
}

// What the rows of a row tile see of the tile of keys that starts at token `first`.
struct Sight {
  int n0, n1;      // tokens that rows g and g + 8 see
  int n_lo, n_hi;  // tokens that all rows, that any row sees
};

// The running softmax: logits to weights.  O must hold all earlier tiles.
template <int KIND, int U, int NP>
__device__ __forceinline__ void weigh(uint32_t st, int first, const Sight& see, int lane, RowState<KIND>& s,
                                      float (&sc)[Cfg<KIND>::KT / 8][4], Weights<KIND, NP>& w, float* scratch) {
  using C = Cfg<KIND>;
  constexpr int KT = C::KT;
  const int g = lane >> 2, j = lane & 3;
  const bool masked = first + KT > see.n_lo;
  if (masked) {
#pragma unroll
    for (int nt = 0; nt < KT / 8; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = first + 16 * (nt >> 1) + key_of<KIND>(nt & 1, j, e);
        if (key >= see.n0) sc[nt][e] = -INFINITY;
        if (key >= see.n1) sc[nt][2 + e] = -INFINITY;
      }
  }
  // A row's reference m is, where it was last set, the maximum of its logits so far less kShift; it is
  // set anew only when one passes that maximum by more than kSlack, so that few tiles rescale O.  In
  // fp16 a weight is so held times 2^10: those down to 2^-24 of the reference keep all 11 bits (sums
  // of many small weights stay unbiased), and 2^kSlack times it still fits.
  float b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
  for (int nt = 0; nt < KT / 8; ++nt) {
    b0 = max3(b0, sc[nt][0], sc[nt][1]);
    b1 = max3(b1, sc[nt][2], sc[nt][3]);
  }
  constexpr float kTop = C::kShift + C::kSlack;
  if (__any_sync(kFull, s.far || b0 * s.f0 > s.m0 + kTop || b1 * s.f1 > s.m1 + kTop)) {
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
      b0 = fmaxf(b0, __shfl_xor_sync(kFull, b0, x));
      b1 = fmaxf(b1, __shfl_xor_sync(kFull, b1, x));
    }
    float4& side = reinterpret_cast<float4*>(scratch + kFarAt / 4)[lane];
    if (s.far) {
      const float4 z = side;
      s.f0 = z.x;
      s.f1 = z.y;
      s.m0 = z.z;
      s.m1 = z.w;
    }
    // (past 2^26 a step of 32 bits is eight and more, too coarse for the shift; nothing that it is for
    // is left there)
    const float t0 = __fmul_rn(b0, s.f0), t1 = __fmul_rn(b1, s.f1);
    const float n0 = fmaxf(s.m0, fabsf(t0) < 16.f * kFar ? t0 - C::kShift : t0);
    const float n1 = fmaxf(s.m1, fabsf(t1) < 16.f * kFar ? t1 - C::kShift : t1);
    const float a0 = ex2_approx(s.m0 - n0), a1 = ex2_approx(s.m1 - n1);
    s.m0 = n0;
    s.m1 = n1;
    s.l0 *= a0;
    s.l1 *= a1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s.o[i][0] *= a0;
      s.o[i][1] *= a0;
      s.o[i][2] *= a1;
      s.o[i][3] *= a1;
    }
    // Below, logit - m is the exact product less the reference, a rounded product: for the largest
    // logit that is up to 2^-24 of the reference instead of zero.  It is no error, as all weights of
    // the row have the factor, until the factor overflows.  So from kFar on the products are rounded
    // first: differences of rounded products, taken here, are zero for the largest.  What is
    // below then leaves them as they are, and the warp comes here for every tile.
    if (__any_sync(kFull, s.far || (fabsf(n0) >= kFar && n0 != kNone) || (fabsf(n1) >= kFar && n1 != kNone))) {
#pragma unroll
      for (int nt = 0; nt < KT / 8; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sc[nt][e] = __fsub_rn(__fmul_rn(sc[nt][e], s.f0), n0);
          sc[nt][2 + e] = __fsub_rn(__fmul_rn(sc[nt][2 + e], s.f1), n1);
        }
      side = make_float4(s.f0, s.f1, n0, n1);
      s.f0 = s.f1 = 1.f;
      s.m0 = s.m1 = 0.f;
      s.far = true;
    }
  }
  const unsigned long long f0 = f2_pack(s.f0, s.f0), f1 = f2_pack(s.f1, s.f1);
  const unsigned long long cc0 = f2_pack(-s.m0, -s.m0), cc1 = f2_pack(-s.m1, -s.m1);
  unsigned long long l0 = f2_pack(s.l0, 0.f), l1 = f2_pack(s.l1, 0.f);
#pragma unroll
  for (int nt = 0; nt < KT / 8; ++nt) {
    f2_unpack(f2_fma(f2_pack(sc[nt][0], sc[nt][1]), f0, cc0), sc[nt][0], sc[nt][1]);
    f2_unpack(f2_fma(f2_pack(sc[nt][2], sc[nt][3]), f1, cc1), sc[nt][2], sc[nt][3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) sc[nt][e] = ex2_approx(sc[nt][e]);
    l0 = f2_add(l0, f2_pack(sc[nt][0], sc[nt][1]));
    l1 = f2_add(l1, f2_pack(sc[nt][2], sc[nt][3]));
  }
  float x, y;
  f2_unpack(l0, x, y);
  s.l0 = x + y;
  f2_unpack(l1, x, y);
  s.l1 = x + y;
  if (masked) {
    // Values that no row sees must not count, not even as 0 * inf.  Nor must those that some
    // rows see (of the row tile's later queries) reach the others: these few keys are added
    // one by one to the rows that see them, and cleared like the rest.
    const int k_lo = min(max(see.n_lo - first, 0), KT), k_hi = min(max(see.n_hi - first, 0), KT);
    if (k_lo < k_hi) {  // (at most 15 keys: those between the first and the last query)
#pragma unroll
      for (int nt = 0; nt < KT / 8; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = 16 * (nt >> 1) + key_of<KIND>(nt & 1, j, e) - k_lo;
          if (key >= 0 && key < 16) {
            scratch[key * 16 + g] = sc[nt][e];
            scratch[key * 16 + g + 8] = sc[nt][2 + e];
          }
        }
      __syncwarp();
      for (int key = k_lo; key < k_hi; ++key) {
        const float p0 = scratch[(key - k_lo) * 16 + g], p1 = scratch[(key - k_lo) * 16 + g + 8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float v[2];
          if (KIND == PISA_CACHE_BF16) {
            const float2 z = value2<KIND, U>(st, key, 4 * i + j);
            v[0] = z.x;
            v[1] = z.y;
          } else {  // dims 16 j + i and 16 j + 8 + i
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 z = value2<KIND, U>(st, key, 8 * j + 4 * e + (i >> 1));
              v[e] = i & 1 ? z.y : z.x;
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (first + key < see.n0) s.o[i][e] = fmaf(p0, v[e], s.o[i][e]);
            if (first + key < see.n1) s.o[i][2 + e] = fmaf(p1, v[e], s.o[i][2 + e]);
          }
        }
      }
      __syncwarp();
    }
    clear_v<KIND, U>(st, lane, k_lo);
    __syncwarp();
  }
  // The weights go into the product with V as one fp16 part (4-bit pages) or two bf16 parts, and
  // one part more for 32-bit results.  A bf16 result is off by up to 2^-8 of itself from its own
  // rounding; weights off by up to 2^-11 each, and not all to one side, add little (16 x 131072
  // tokens of 4 bits: error against 64 bits 1.67e-3 instead of 1.66e-3), while a second part would
  // take 90.6 us instead of 71.1.
#pragma unroll
  for (int i = 0; i < KT / 16; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float u = sc[2 * i + (k >> 1)][2 * (k & 1)], v = sc[2 * i + (k >> 1)][2 * (k & 1) + 1];
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const uint32_t h = KIND == PISA_CACHE_E2M1 ? pack_f16x2(u, v) : pack_bf16x2(u, v);
        w.a[p][i][k] = h;
        if (p + 1 < NP) {
          if (KIND == PISA_CACHE_E2M1) {
            const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&h));
            u -= r.x;
            v -= r.y;
          } else {
            u -= __uint_as_float(h << 16);
            v -= __uint_as_float(h & 0xffff0000u);
          }
        }
      }
    }
}

// Tiles [i0, i1) of a unit (u.sel: all of the listed blocks that begin in sight; blk: this
// lane's entries of the list, lane and lane + 32), shared out among the CTA's W warps; on
// return every warp holds its own partial sums.  A warp copies its tiles ahead into a ring of
// three stages: while one is on its way, the logits of the next tile and the products with V
// of the one before are computed side by side.  (Keys and values in rings of their own, with
// two tiles on their way, were 2 to 4 % slower: the memory system is full with one.)
template <int KIND, int U, int NP, int W, bool LIST>
__device__ __forceinline__ void run_tiles(const CacheAttendLaunch& a, const Unit& u, const QueryWords& q,
                                          const int (&blk)[2], int i0, int i1, uint32_t ring, float* scratch, int warp,
                                          int lane, RowState<KIND>& s) {
  using C = Cfg<KIND>;
  constexpr int KT = C::KT;
  const bool listed = LIST && u.sel != nullptr;
  constexpr int E = KT > U ? KT / U : 1;  // records of a tile
  constexpr int kAhead = 32 / E;          // tiles a look ahead covers
  constexpr uint32_t kStage = kStageBytes<KIND>;
  static_assert(C::kStages == 3, "");
  const int g = lane >> 2;
  // what each row sees: tokens before n_vis(t) = n - T + t + 1
  const int ra = u.r0 + g, rb = ra + 8;
  const int base = u.n - a.T + 1 + u.t_first;
  const int last = min(u.rows, u.r0 + 16) - 1;
  const Sight see = {ra < u.rows ? base + ra / a.G : 0, rb < u.rows ? base + rb / a.G : 0, base + u.r0 / a.G,
                     base + last / a.G};
  int* list = reinterpret_cast<int*>(scratch);  // (listed: a row tile is one query's, so weigh leaves it alone)
  if (listed) {  // the listed blocks that count, in the order of the list
    unsigned some[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      some[h] = __ballot_sync(kFull, blk[h] >= 0 && blk[h] < (1 << 21) && blk[h] * kC < see.n_hi);
    const unsigned below = (1u << lane) - 1u;
    if (some[0] >> lane & 1) list[__popc(some[0] & below)] = blk[0];
    if (some[1] >> lane & 1) list[__popc(some[0]) + __popc(some[1] & below)] = blk[1];
    __syncwarp();
    i1 = (__popc(some[0]) + __popc(some[1])) * (kC / KT);
  } else {
    i1 = min(i1, (max(see.n_hi, 0) + KT - 1) / KT);
  }
  const int mine = i1 - i0 > warp ? (i1 - i0 - warp + W - 1) / W : 0;  // the warp's tiles
  if (mine == 0) return;
  const int32_t* table = a.cache.table + (long long)u.b * a.cache.max_pages;

  auto first_of = [&](int x) {  // the first token of the warp's tile number x
    const int i = i0 + warp + W * x;
    return listed ? list[i * KT / kC] * kC + (i * KT) % kC : i * KT;
  };
  // Lane l looks ahead: where record l % E of the warp's tile number x + l / E lies.  Records
  // that nothing sees are read from the first page instead.
  long long off = 0;
  auto look = [&](int x) {
    int page = 0;
    off = 0;
    const int y = x + lane / E;
    int* first_bad = reinterpret_cast<int*>(scratch + kBadAt / 4);
    if (y < mine) {
      const int p = first_of(y) + (lane % E) * U;
      if (p < see.n_hi) {
        page = table[p >> a.cache.page_shift];
        if (page >= 0 && page < a.cache.n_pages) {
          off = cache_record(a.cache, C::kRow, page, u.kv, p);
          // (bf16: the tile may start inside a record)
          if (KIND == PISA_CACHE_BF16 && U > KT) off += (p & (U - 1)) * 128;
        } else {
          page = -1;
        }
      }
    }
    if (__any_sync(kFull, page < 0)) {
      const int p = page < 0 ? first_of(y) + (lane % E) * U : INT_MAX, q = __reduce_min_sync(kFull, p);
      if (lane == 0) *first_bad = s.bad ? min(*first_bad, q) : q;
      s.bad = true;
      __syncwarp();
    }
  };
  auto issue = [&](int x, uint32_t dst) {  // the copies of the warp's tile number x
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const unsigned char* src = a.cache.pages + __shfl_sync(kFull, off, (x % kAhead) * E + e);
      if (KIND == PISA_CACHE_E2M1) {
        constexpr int kChunks = (U < KT ? U : KT) * kRowE2m1 / 16;
        src += lane * 16;
        const uint32_t d = dst + e * U * kRowE2m1 + lane * 16;
#pragma unroll
        for (int c = 0; c < (kChunks + 31) / 32; ++c)
          if ((c + 1) * 32 <= kChunks || c * 32 + lane < kChunks) cpa16(d + c * 512, src + c * 512);
      } else {
        constexpr int kRows = U < KT ? U : KT;  // rows of K (and of V) in this record
#pragma unroll
        for (int c = 0; c < kRows / 4; ++c) {
          const int r = 4 * c + (lane >> 3), ch = lane & 7;
          const uint32_t d = dst + swz128(e * U + r, ch);
          cpa16(d, src + r * 128 + ch * 16);
          cpa16(d + KT * 128, src + U * 128 + r * 128 + ch * 16);
        }
      }
    }
  };
  float sc[KT / 8][4];
  Weights<KIND, NP> w;
  look(0);
  issue(0, ring);
  cpa_commit();
  if (mine > 1) issue(1, ring + kStage);
  cpa_commit();
  make_q(a, q, lane, s);
  cpa_wait<1>();
  __syncwarp();
  const int f0 = first_of(0);
  products<KIND, U, NP, true, false>(ring, 0, lane, s, sc, w);
  weigh<KIND, U, NP>(ring, f0, see, lane, s, sc, w, scratch);
  uint32_t cur = ring, next = ring + kStage, spare = ring + 2 * kStage;
  for (int x = 0; x + 1 < mine; ++x) {
    if (x + 2 < mine) {
      if ((x + 2) % kAhead == 0) look(x + 2);
      issue(x + 2, spare);
    }
    cpa_commit();
    cpa_wait<1>();  // tile x + 1 has come
    __syncwarp();
    products<KIND, U, NP, true, true>(next, cur, lane, s, sc, w);
    weigh<KIND, U, NP>(next, first_of(x + 1), see, lane, s, sc, w, scratch);
    __syncwarp();  // the reads of tile x are done before its stage is refilled
    const uint32_t t = cur;
    cur = next;
    next = spare;
    spare = t;
  }
  products<KIND, U, NP, false, true>(0, cur, lane, s, sc, w);
  cpa_wait<0>();
  if (s.far) {
    const float4 z = reinterpret_cast<const float4*>(scratch + kFarAt / 4)[lane];
    s.m0 = z.z;
    s.m1 = z.w;
  }
  if (s.bad) {  // the rows that see a page out of range become NaN
    const int first_bad = *reinterpret_cast<const int*>(scratch + kBadAt / 4);
    if (first_bad < see.n0) s.l0 = __int_as_float(0x7fc00000);
    if (first_bad < see.n1) s.l1 = __int_as_float(0x7fc00000);
  }
}

// Puts the warps' partial sums where merged() finds them: O into the ring, which is idle then.
template <int KIND, int W>
__device__ __forceinline__ void merge_warps(RowState<KIND>& s, float* mo, float (*ml)[2][16], int warp, int lane) {
  static_assert(Cfg<KIND>::kStages * kStageBytes<KIND> >= 4096, "");
  const int g = lane >> 2, j = lane & 3;
#pragma unroll
  for (int x = 1; x < 4; x <<= 1) {
    s.l0 += __shfl_xor_sync(kFull, s.l0, x);
    s.l1 += __shfl_xor_sync(kFull, s.l1, x);
  }
  if (j == 0) {
    ml[warp][0][g] = s.m0;
    ml[warp][0][g + 8] = s.m1;
    ml[warp][1][g] = s.l0;
    ml[warp][1][g + 8] = s.l1;
  }
  __syncthreads();  // every warp's tiles are done
  float* o = mo + warp * 1024;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = g + 8 * h;
    if (KIND == PISA_CACHE_BF16) {  // column tile i: dims 8 i + 2 j and the next
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<float2*>(o + merge_at(r, 2 * i + (j >> 1)) + 2 * (j & 1)) =
            make_float2(s.o[i][2 * h], s.o[i][2 * h + 1]);
    } else {  // one word of eight codes a key gives column n dims 8 n ..: tile i is dims 16 j + i and 16 j + 8 + i
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int i = 4 * (c & 1), e = 2 * h + (c >> 1);
        *reinterpret_cast<float4*>(o + merge_at(r, 4 * j + c)) =
            make_float4(s.o[i][e], s.o[i + 1][e], s.o[i + 2][e], s.o[i + 3][e]);
      }
    }
  }
  __syncthreads();
}

// Dims 4 quad .. + 3 of a row's sum over the warps, the row's reference and sum of weights.
template <int W>
__device__ __forceinline__ float4 merged(const float* mo, const float (*ml)[2][16], int row, int quad, float& m,
                                         float& l) {
  m = kNone;
#pragma unroll
  for (int w = 0; w < W; ++w) m = fmaxf(m, ml[w][0][row]);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  l = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const float mw = ml[w][0][row], lw = ml[w][1][row];
    const float f = ex2_approx(mw - m);
    l = fmaf(f, lw, l);  // (a warp without keys adds 0, or the NaN of a bad page)
    const float4 x = *reinterpret_cast<const float4*>(mo + w * 1024 + merge_at(row, quad));
    acc.x = fmaf(f, x.x, acc.x);
    acc.y = fmaf(f, x.y, acc.y);
    acc.z = fmaf(f, x.z, acc.z);
    acc.w = fmaf(f, x.w, acc.w);
  }
  return acc;
}

// Writes dims 4 quad .. + 3 of a unit's row, normalised; rows without keys get zeros.
__device__ __forceinline__ void write_out(const CacheAttendLaunch& a, const Unit& u, int row, int quad, float4 acc,
                                          float l) {
  const int r = u.r0 + row;
  if (r >= u.rows) return;
  const int t = u.t_first + r / a.G, head = u.kv * a.G + r % a.G;
  const float f = l == 0.f ? 0.f : exp2i(a.cache.kind == PISA_CACHE_E2M1 ? a.cache.v_exp : 0) / l;
  if (l == 0.f) acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const long long at = (((long long)u.b * a.T + t) * a.Hq + head) * kD + 4 * quad;
  acc.x *= f;
  acc.y *= f;
  acc.z *= f;
  acc.w *= f;
  if (a.out_f32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = acc;
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) =
        make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
}

// The tokens of sequence b (lengths past the table's capacity are an error, and cut).
__device__ __forceinline__ int seq_len(const CacheAttendLaunch& a, int b, bool& over) {
  const long long cap = (long long)a.cache.max_pages << a.cache.page_shift;
  const int n = a.lengths[b];
  over = n > cap;
  return n < 0 ? 0 : over ? (int)cap : n;
}

// Places that a unit of nt tiles has in the stream: its tiles, and some for what a run spends at
// its end (the warps' merge, the next unit's chain of loads; about 4 us), so that the runs that
// change units take as long as the others.  Places at the end 0 / 12 / 24 / 36 / 48, us a call:
//   4 bits  16 x 131072 73.5 / 72.1 / 71.5 / 71.6 / 71.9   64 x 9000 ragged, 8 heads 88.8 / 63.6 / 56.7 / 57.5 / 59.8
//   bf16    8 x 131072 ragged 64.8 / 63.8 / 63.3 / 63.0 / 63.3   64 x 9000 ragged, 8 heads 119.7 / 103 / 96.3 / 96.5 / 97.4
template <int KIND>
__device__ __forceinline__ int unit_places(int nt) {
  return nt ? nt + Cfg<KIND>::kChange : 0;
}

// Places of all units before sequence b (b = B: of all): every warp computes it by itself.
template <int KIND>
__device__ __forceinline__ long long places_before(const CacheAttendLaunch& a, int b, int units, int lane) {
  constexpr int KT = Cfg<KIND>::KT;
  long long sum = 0;
  bool over;
  for (int i = lane; i < b; i += 32) sum += unit_places<KIND>((seq_len(a, i, over) + KT - 1) / KT);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(kFull, sum, x);
  return sum * units;
}

// The sequence that place `at` of the stream belongs to, and the places before that sequence: 32
// sequences at a time.
template <int KIND>
__device__ __forceinline__ int seq_of(const CacheAttendLaunch& a, long long at, int units, int lane, long long& base) {
  constexpr int KT = Cfg<KIND>::KT;
  base = 0;
  for (int b0 = 0; b0 < a.cache.B; b0 += 32) {
    bool over;
    const int n = b0 + lane < a.cache.B ? seq_len(a, b0 + lane, over) : 0;
    const long long t = (long long)unit_places<KIND>((n + KT - 1) / KT) * units;
    long long inc = t;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const long long y = __shfl_up_sync(kFull, inc, x);
      if (lane >= x) inc += y;
    }
    const unsigned hit = __ballot_sync(kFull, base + inc > at);
    if (hit) {
      const int l = __ffs(hit) - 1;
      base += __shfl_sync(kFull, inc - t, l);
      return b0 + l;
    }
    base += __shfl_sync(kFull, inc, 31);
  }
  return a.cache.B;  // (past the last place)
}

// Places per CTA of the split form.
__device__ __forceinline__ long long run_length(long long total, int grid) {
  const long long per = total < (1 << 30) ? ((int)total + grid - 1) / grid : (total + grid - 1) / grid;
  return per < kCaMinTiles ? kCaMinTiles : per;
}

template <int KIND, int W>
constexpr int kRing = W* Cfg<KIND>::kStages* kStageBytes<KIND>;
template <int KIND, int W>
constexpr int attend_smem() {
  return kRing<KIND, W> + W * (kScratch + 2 * 16 * 4);
}

template <int KIND, int U, int NP, int W>
__global__ void __launch_bounds__(W * 32, Cfg<KIND>::kWarps / W) cache_attend_direct_kernel(CacheAttendLaunch a) {
  using C = Cfg<KIND>;
  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (uniform to the compiler)
  const uint32_t ring = warp * C::kStages * kStageBytes<KIND>;                        // (offset into the shared memory)
  float* mo = reinterpret_cast<float*>(ca_smem);
  float* scratch = reinterpret_cast<float*>(ca_smem + kRing<KIND, W> + warp * kScratch);
  float(*ml)[2][16] = reinterpret_cast<float(*)[2][16]>(ca_smem + kRing<KIND, W> + W * kScratch);
  after_the_one_before();
  // one CTA per (b, t, kv) with a list, per (b, row tile, kv) without
  const unsigned id = blockIdx.x;
  Unit u;
  u.kv = id % a.cache.Hkv;
  const unsigned bt = id / a.cache.Hkv;
  int blk[2] = {-1, -1};
  if (a.idx) {
    u.t_first = bt % a.T;
    u.b = bt / a.T;
    u.r0 = 0;
    u.rows = a.G;
    u.sel = a.idx + (((long long)u.b * a.cache.Hkv + u.kv) * a.T + u.t_first) * a.Ksel;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (lane + 32 * h < a.Ksel) blk[h] = u.sel[lane + 32 * h];
  } else {
    const unsigned RT = (a.T * a.G + 15) / 16;
    u.t_first = 0;
    u.r0 = (bt % RT) * 16;
    u.b = bt / RT;
    u.rows = a.T * a.G;
    u.sel = nullptr;
  }
  bool over;
  u.n = seq_len(a, u.b, over);
  QueryWords q;
  fetch_q(a, u, lane, q);
  RowState<KIND> s;
  reset(s);
  run_tiles<KIND, U, NP, W, true>(a, u, q, blk, 0, 1 << 30, ring, scratch, warp, lane, s);
  if ((threadIdx.x == 0 && over) || (lane == 0 && s.bad)) set_status(a.status, PISA_ERR_DEVICE_BOUNDS);
  merge_warps<KIND, W>(s, mo, ml, warp, lane);
  for (int i = threadIdx.x; i < 256; i += W * 32) {
    float m, l;
    const float4 acc = merged<W>(mo, ml, i >> 4, i & 15, m, l);
    write_out(a, u, i >> 4, i & 15, acc, l);
  }
}

template <int KIND, int U, int NP>
__global__ void __launch_bounds__(Cfg<KIND>::kWarps * 32, 1) cache_attend_split_kernel(CacheAttendLaunch a) {
  using C = Cfg<KIND>;
  constexpr int KT = C::KT, W = C::kWarps;
  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t ring = warp * C::kStages * kStageBytes<KIND>;
  float* mo = reinterpret_cast<float*>(ca_smem);
  float* scratch = reinterpret_cast<float*>(ca_smem + kRing<KIND, W> + warp * kScratch);
  float(*ml)[2][16] = reinterpret_cast<float(*)[2][16]>(ca_smem + kRing<KIND, W> + W * kScratch);
  after_the_one_before();
  RowState<KIND> s;
  Unit u;
  bool over;
  const int blk[2] = {-1, -1};
  // this CTA's run of the stream (and its row tile, where the row tiles go side by side)
  const int RT = (a.T * a.G + 15) / 16;
  const int units = a.cache.Hkv * (C::kSide ? 1 : RT);  // of a sequence
  const long long total = places_before<KIND>(a, a.cache.B, units, lane);
  const long long per = run_length(total, C::kSide ? gridDim.x / RT : gridDim.x);
  long long cur = per * (C::kSide ? blockIdx.x / RT : blockIdx.x);
  const long long end = cur + per < total ? cur + per : total;
  // sequences without tokens: zeros
  for (int b = blockIdx.x; b < a.cache.B; b += gridDim.x)
    if (seq_len(a, b, over) == 0) {
      const long long at = (long long)b * a.T * a.Hq * kD;
      for (int i = threadIdx.x; i < a.T * a.Hq * kD / 8; i += W * 32) {
        if (a.out_f32) {
          reinterpret_cast<float4*>(static_cast<float*>(a.out) + at)[2 * i] = make_float4(0.f, 0.f, 0.f, 0.f);
          reinterpret_cast<float4*>(static_cast<float*>(a.out) + at)[2 * i + 1] = make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
          reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at)[i] = make_uint4(0, 0, 0, 0);
        }
      }
    }
  if (cur >= end) return;  // (CTAs left over where RT does not divide the grid, too)
  long long base;  // places before sequence u.b
  u.b = seq_of<KIND>(a, cur, units, lane, base);
  u.t_first = 0;
  u.rows = a.T * a.G;
  u.sel = nullptr;
  while (cur < end) {
    u.n = seq_len(a, u.b, over);
    const int nt = (u.n + KT - 1) / KT;  // tiles of a unit of this sequence
    const int places = unit_places<KIND>(nt);
    if (nt == 0 || cur >= base + (long long)places * units) {  // on to the next sequence
      base += (long long)places * units;
      ++u.b;
      continue;
    }
    // (places of one sequence: below 2^22 * 32 heads * 16 row tiles + 2^15, within 32 bits)
    const unsigned at = (unsigned)(cur - base), un = at / (unsigned)places;
    const int i0 = (int)(at - un * places);
    if (i0 >= nt) {  // behind a unit's tiles
      cur += places - i0;
      continue;
    }
    const int i1 = (int)(end - cur < nt - i0 ? i0 + (end - cur) : nt);
    u.kv = C::kSide ? un : un / RT;
    u.r0 = ((C::kSide ? blockIdx.x : un) % RT) * 16;
    QueryWords q;
    fetch_q(a, u, lane, q);
    reset(s);
    run_tiles<KIND, U, NP, W, false>(a, u, q, blk, i0, i1, ring, scratch, warp, lane, s);
    if ((threadIdx.x == 0 && over) || (lane == 0 && s.bad)) set_status(a.status, PISA_ERR_DEVICE_BOUNDS);
    merge_warps<KIND, W>(s, mo, ml, warp, lane);
    if (threadIdx.x < 256) {
      const int row = threadIdx.x >> 4, quad = threadIdx.x & 15;
      float m, l;
      const float4 acc = merged<W>(mo, ml, row, quad, m, l);
      if (i0 == 0 && i1 == nt) {
        write_out(a, u, row, quad, acc, l);
      } else {  // slot 1: a unit that begins in the run, slot 0: one that began before
        float* p = a.part + ((long long)blockIdx.x * 2 + (i0 == 0)) * kPartFloats;
        *reinterpret_cast<float4*>(p + row * 64 + 4 * quad) = acc;
        if (quad == 0) {
          p[1024 + row] = m;
          p[1040 + row] = l;
        }
      }
    }
    cur += i1 < nt ? i1 - i0 : places - i0;
    __syncthreads();  // the merge buffers are free again
  }
}

// Joins the partial results of the units that lie in several runs.
//   FEW: 16 CTAs a unit, one row each: 16 quads x 16 groups of partials (few units are cut into
//     many runs each: a call for one sequence, two units, of 131072 tokens 15.0 -> 12.4 us).
//   else: at most one such unit begins in a run, the one that holds the run's last place.  Four
//     CTAs a run and row tile, four rows each: 4 rows x 16 quads x 4 groups of partials.
// The kernel starts while the one before it runs, and reads the lengths, which that one only
// reads too; the partial results after the wait, which every CTA passes (a grid that ended
// without it would let the next kernel of the stream overtake the one before).
template <int KIND, bool FEW>
__global__ void __launch_bounds__(256) cache_join_kernel(CacheAttendLaunch a, int grid) {
  constexpr int KT = Cfg<KIND>::KT;
  constexpr int kRows = FEW ? 1 : 4, kGroups = 16 / kRows;
  __shared__ float4 so[kGroups][kRows][16];
  __shared__ float sm[kGroups][kRows], sl[kGroups][kRows];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int quad = threadIdx.x & 15, rq = (threadIdx.x >> 4) % kRows, grp = (threadIdx.x >> 4) / kRows;
  constexpr bool kSide = Cfg<KIND>::kSide;
  const int RT = (a.T * a.G + 15) / 16, side = kSide ? RT : 1;
  const int runs = kSide ? grid / RT : grid, units = kSide ? a.cache.Hkv : a.cache.Hkv * RT;
  const int row = (int)(blockIdx.x % (16 / kRows)) * kRows + rq;
  const long long total = places_before<KIND>(a, a.cache.B, units, lane);
  const long long per = run_length(total, runs);
  Unit u;
  int c0, c1 = 0;  // the runs that hold its tiles
  int beside;      // which of the row tiles side by side
  bool cut;
  auto set_unit = [&](unsigned un) {  // the unit's number in its sequence
    u.kv = kSide ? un : un / RT;
    u.r0 = (kSide ? beside : un % RT) * 16;
    u.rows = a.T * a.G;
    u.t_first = 0;
    u.sel = nullptr;
  };
  if (FEW) {
    const unsigned id = blockIdx.x / 16, unit = kSide ? id / RT : id;
    beside = kSide ? id - unit * RT : 0;
    u.b = unit / units;
    const unsigned un = unit % units;
    set_unit(un);
    bool over;
    u.n = seq_len(a, u.b, over);
    const int nt = (u.n + KT - 1) / KT;
    const long long w0 = places_before<KIND>(a, u.b, units, lane) + (long long)un * unit_places<KIND>(nt);
    c0 = (int)(w0 / per);
    c1 = (int)((w0 + nt - 1) / per);
    cut = nt != 0 && c0 != c1;
  } else {
    const int cta = blockIdx.x / 4;
    c0 = kSide ? cta / RT : cta;
    beside = kSide ? cta - c0 * RT : 0;
    const long long end = per * (c0 + 1);  // the run's end, if the stream goes on after it
    cut = end < total;
    if (cut) {
      long long base;
      u.b = seq_of<KIND>(a, end - 1, units, lane, base);
      bool over;
      u.n = seq_len(a, u.b, over);
      const int nt = (u.n + KT - 1) / KT, places = unit_places<KIND>(nt);
      const unsigned un = (unsigned)(end - 1 - base) / (unsigned)places;
      set_unit(un);
      const long long w0 = base + (long long)un * places, w1 = w0 + nt;
      cut = w1 > end && w0 >= end - per;
      c1 = (int)((w1 - 1) / per);
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!cut) return;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = c0 + grp; c <= c1; c += kGroups) {
    const int slot = c == c0 ? 1 : 0;
    const float* p = a.part + (((long long)c * side + beside) * 2 + slot) * kPartFloats;
    const float mc = p[1024 + row], lc = p[1040 + row];
    const float4 x = *reinterpret_cast<const float4*>(p + row * 64 + 4 * quad);
    const float n = fmaxf(m, mc);
    const float f = m == -INFINITY ? 0.f : ex2_approx(m - n), h = mc == -INFINITY ? 0.f : ex2_approx(mc - n);
    l = (m == -INFINITY ? l : l * f) + (mc == -INFINITY ? lc : lc * h);
    acc.x = acc.x * f + x.x * h;
    acc.y = acc.y * f + x.y * h;
    acc.z = acc.z * f + x.z * h;
    acc.w = acc.w * f + x.w * h;
    m = n;
  }
  so[grp][rq][quad] = acc;
  if (quad == 0) {
    sm[grp][rq] = m;
    sl[grp][rq] = l;
  }
  __syncthreads();
  if (grp) return;
  m = sm[0][rq];
#pragma unroll
  for (int x = 1; x < kGroups; ++x) m = fmaxf(m, sm[x][rq]);
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  l = 0.f;
#pragma unroll
  for (int x = 0; x < kGroups; ++x) {
    const float mx = sm[x][rq], lx = sl[x][rq];
    const float f = mx == -INFINITY ? 0.f : ex2_approx(mx - m);
    const float4 v = so[x][rq][quad];
    l += mx == -INFINITY ? lx : lx * f;
    acc.x += v.x * f;
    acc.y += v.y * f;
    acc.z += v.z * f;
    acc.w += v.w * f;
  }
  write_out(a, u, row, quad, acc, l);
}

template <int KIND, int U, int NP, int W>
static cudaError_t launch_direct(const CacheAttendLaunch& L, unsigned units, cudaStream_t s) {
  return launch_early<cache_attend_direct_kernel<KIND, U, NP, W>>(units, W * 32, attend_smem<KIND, W>(), s, L);
}

// Whether the direct form takes whole caches of up to `cap` tokens.  It saves the second kernel and
// each run's changes of unit.  Direct / split, us a call, 4 bits (bf16), two KV heads:
//   units x tokens  32 x 1500 7.4 / 8.3 (7.9 / 10.0)       64 x 4096 13.6 / 14.1 (16.7 / 18.7)
//                   256 x 4096 23.9 / 34.0 (42.8 / 50.0)   128 x 8192 24.4 / 29.3 (42.5 / 47.7)
// It loses where units are few for their length (8 x 4096 13.1 / 8.2, 64 x 8192 23.4 / 19.0), and
// where few of many units are long (256 x 16384 full 76.3 / 79.7, ragged 73.7 / 53.5).
inline bool takes_direct(long long cap, long long units) {
  const long long most = 64 * units < 8192 ? 64 * units : 8192;
  return cap <= (most > 2048 ? most : 2048);
}

template <int KIND, int U, int NP>
static cudaError_t launch_attend(const CacheAttendLaunch& L, cudaStream_t s) {
  using C = Cfg<KIND>;
  const int RT = (L.T * L.G + 15) / 16;
  const long long cap = (long long)L.cache.max_pages << L.cache.page_shift;
  const long long units = (long long)L.cache.B * L.cache.Hkv * (L.idx ? L.T : RT);
  if (L.idx || takes_direct(cap, units)) {
    // The more units there are, the fewer warps share one out, so that all CTAs run at once
    // (128 x 2 units of 32 blocks: six warps 15.1 us, four 18.7, twelve 19.1).
    if (units <= kCaGrid) return launch_direct<KIND, U, NP, C::kWarps>(L, (unsigned)units, s);
    if (units <= 2 * kCaGrid) return launch_direct<KIND, U, NP, C::kHalf>(L, (unsigned)units, s);
    return launch_direct<KIND, U, NP, C::kThird>(L, (unsigned)units, s);
  }
  cudaError_t e = launch_early<cache_attend_split_kernel<KIND, U, NP>>(kCaGrid, C::kWarps * 32,
                                                                       attend_smem<KIND, C::kWarps>(), s, L);
  if (e != cudaSuccess) return e;
  if (units <= kCaGrid / 4)
    return launch_early<cache_join_kernel<KIND, true>>((unsigned)units * 16, 256, 0, s, L, kCaGrid);
  return launch_early<cache_join_kernel<KIND, false>>(kCaGrid * 4, 256, 0, s, L, kCaGrid);
}

template <int KIND, int U>
static cudaError_t launch_attend_u(const CacheAttendLaunch& L, cudaStream_t s) {
  constexpr int NP = KIND == PISA_CACHE_BF16 ? 2 : 1;  // parts of the weights (see weigh)
  return L.out_f32 ? launch_attend<KIND, U, NP + 1>(L, s) : launch_attend<KIND, U, NP>(L, s);
}

template <int KIND>
static cudaError_t launch_attend_k(const CacheAttendLaunch& L, cudaStream_t s) {
  switch (L.cache.rec_shift) {
    case 4: return launch_attend_u<KIND, 16>(L, s);
    case 5: return launch_attend_u<KIND, 32>(L, s);
    default: return launch_attend_u<KIND, 64>(L, s);
  }
}

}  // namespace pisa
