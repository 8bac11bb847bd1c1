// cache_attend.cu -- attention of a sequence's newest tokens over its paged KV cache, all of
// it or the blocks that a selection listed; pages in bf16 or 4 bits.
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = exp(q . k_j / 8 - max_j)
// in one pass over the keys with a running maximum and sum per row (32 bits, base 2).
//
// The 16 rows of an mma.sync m16n8k16 tile are the query heads of one KV head's group (and of
// several queries, where the group is smaller); every warp of a CTA takes its own tiles of
// keys, and the CTA's warps are merged through shared memory at the end.  Per key the kernel
// reads 72 or 256 bytes and does 4 * 64 * 16 multiply-adds, so the bytes bound it; mma.sync
// at its rate of about 1024 multiply-adds per clock and SM takes 2/3 of the time the 4-bit
// bytes take.
//
// Without a list the tiles of all (sequence, KV head, row tile) units form one stream, which
// is cut into equal runs, one per CTA, whatever the lengths; a unit that ends up in several
// CTAs is joined by a second kernel from 32-bit partial results.
#include <mutex>

#include "cache.cuh"
#include "tc.cuh"

namespace pisa {

constexpr int kCaWarps = 8;
constexpr int kCaStages = 2;
constexpr int kPartFloats = 16 * 64 + 32;  // a partial result: O [16][64], row maxima, row sums
constexpr int kCaGridMax = 304;            // CTAs of the split form: two on each of 152 SMs
constexpr int kCaMinTiles = 8;             // tiles a CTA of the split form takes at least
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPShift = 14.f;  // fp16 weights are held times 2^14 (see below)

size_t cache_part_bytes() { return (size_t)kCaGridMax * 2 * kPartFloats * sizeof(float); }

template <int KIND>
struct Cfg;
template <>
struct Cfg<PISA_CACHE_BF16> {
  static constexpr int KT = 32;  // keys of a tile
  static constexpr int kRow = kRowBf16;
  static constexpr int kCtasPerSm = 1;
};
template <>
struct Cfg<PISA_CACHE_E2M1> {
  static constexpr int KT = 64;
  static constexpr int kRow = kRowE2m1;
  static constexpr int kCtasPerSm = 2;
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void cpa16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void lds64(uint32_t a, uint32_t& x, uint32_t& y) {
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
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
  float m0, m1, l0, l1;
  float o[8][4];
  bool bad;  // a page out of range was met
};

// The dims of output column (tile i, element e) of lane j: the 4-bit form gives a lane one
// word of eight codes per key, dims 8 n .. 8 n + 7 of MMA column n, so tile i is dim 8 n + i.
template <int KIND>
__device__ __forceinline__ int out_dim(int i, int j, int e) {
  return KIND == PISA_CACHE_BF16 ? 8 * i + 2 * j + e : 8 * (2 * j + e) + i;
}

// Loads the query rows r0 + g and r0 + g + 8 of `rows` (row r: query r / G, head r % G).
// In the 4-bit form the products are taken in fp16: the row is scaled by a power of two so
// that its largest element lies in [1, 2), where fp16 holds all 8 bits of a bf16 down to
// 2^-17 of it and is off by at most 2^-25 of it below (the fp32 sums of the products are
// off by as much).
template <int KIND>
__device__ __forceinline__ void load_q(const CacheAttendLaunch& a, int b, int kv, int t_first, int r0, int rows,
                                       int lane, RowState<KIND>& s) {
  const int g = lane >> 2, j = lane & 3;
  uint32_t w[2][8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = r0 + g + 8 * h;
    uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
    if (r < rows) {
      const int t = t_first + r / a.G, head = kv * a.G + r % a.G;
      const uint4* p =
          reinterpret_cast<const uint4*>(a.q.data + b * a.q.sb + (long long)t * a.q.st + head * a.q.sh) + 2 * j;
      x0 = __ldg(p);
      x1 = __ldg(p + 1);
    }
    w[h][0] = x0.x; w[h][1] = x0.y; w[h][2] = x0.z; w[h][3] = x0.w;
    w[h][4] = x1.x; w[h][5] = x1.y; w[h][6] = x1.z; w[h][7] = x1.w;
  }
  float f[2] = {kScale * kLog2e, kScale * kLog2e};
  if (KIND == PISA_CACHE_E2M1) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t t = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) t = __vmaxu2(t, w[h][i] & 0x7fff7fffu);
      t = max(t & 0xffffu, t >> 16);
      t = max(t, __shfl_xor_sync(kFull, t, 1));
      t = max(t, __shfl_xor_sync(kFull, t, 2));
      int e = (int)(t >> 7) - 127;              // the largest lies in [2^e, 2^(e + 1))
      e = t == 0 || t >= 0x7f80u ? 0 : max(min(e, 100), -100);
      const float down = exp2i(-e);
      f[h] *= exp2i(e) * exp2i(a.cache.k_exp);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[h][i] = pack_f16x2(__uint_as_float(w[h][i] << 16) * down, __uint_as_float(w[h][i] & 0xffff0000u) * down);
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
          const uint32_t u = __shfl_sync(kFull, w[h][i], (lane & 28) | ks);
          const uint32_t v = __shfl_sync(kFull, w[h][4 + i], (lane & 28) | ks);
          if (i == j) {
            lo = u;
            hi = v;
          }
        }
        s.qa[ks][h] = lo;
        s.qa[ks][2 + h] = hi;
      }
  }
  s.f0 = f[0];
  s.f1 = f[1];
  s.m0 = s.m1 = -INFINITY;
  s.l0 = s.l1 = 0.f;
  s.bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) s.o[i][0] = s.o[i][1] = s.o[i][2] = s.o[i][3] = 0.f;
}

// The key (of 16 in a group) behind column element (half h of the group, e) of lane j.
template <int KIND>
__device__ __forceinline__ int key_of(int h, int j, int e) {
  return KIND == PISA_CACHE_BF16 ? 8 * h + 2 * j + e : 8 * h + j + 4 * e;
}

// V fragments of 16-key group i: b[n][0..1] for the eight column tiles n.  Keys at or past
// `limit` (relative to the tile) count as zeros, whatever the memory holds.
template <int KIND, int U, bool MASK>
__device__ __forceinline__ void load_v(uint32_t st, int i, int lane, int limit, uint32_t (&vb)[8][2]) {
  const int g = lane >> 2, j = lane & 3;
  if (KIND == PISA_CACHE_E2M1) {
    using L = E2m1Tile<U>;
    const uint32_t av = st + L::v(i) + 4 * g, as = st + L::vs(i) + (g >> 1);
    uint32_t w[4], sc[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {  // keys j, j + 4, j + 8, j + 12
      w[x] = lds32(av + (j + 4 * x) * 32);
      sc[x] = lds8(as + (j + 4 * x) * 4);
      if (MASK && 16 * i + j + 4 * x >= limit) sc[x] = 0;
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const uint32_t wa = w[2 * y], wb = w[2 * y + 1];
      const uint32_t s2 = e4m3x2(sc[2 * y] | (sc[2 * y + 1] << 8));
      // bytes whose nibbles are one dim of both keys
      const uint32_t even = (wa & 0x0f0f0f0fu) | ((wb << 4) & 0xf0f0f0f0u);
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
    uint32_t m0 = 0xffffffffu, m1 = 0xffffffffu;
    if (MASK) {
      const int n0 = limit - 16 * i - 2 * j, n1 = n0 - 8;
      m0 = n0 >= 2 ? 0xffffffffu : n0 == 1 ? 0xffffu : 0u;
      m1 = n1 >= 2 ? 0xffffffffu : n1 == 1 ? 0xffffu : 0u;
    }
#pragma unroll
    for (int dp = 0; dp < 4; ++dp) {
      uint32_t r[4];
      ldm_x4_t(sV + swz128(16 * i + (lane & 7) + 8 * ((lane >> 3) & 1), 2 * dp + (lane >> 4)), r);
      vb[2 * dp][0] = r[0] & m0;
      vb[2 * dp][1] = r[1] & m1;
      vb[2 * dp + 1][0] = r[2] & m0;
      vb[2 * dp + 1][1] = r[3] & m1;
    }
  }
}

// One staged tile of KT keys.  MASK: row g sees the tile's first v0 keys, row g + 8 the first
// v1 (possibly none); t_lo .. t_hi are the queries of the row tile and lim(t) the keys of
// the tile that query t sees.
template <int KIND, int U, bool MASK, typename Lim>
__device__ __forceinline__ void do_tile(uint32_t st, int lane, RowState<KIND>& s, int v0, int v1, int t_lo, int t_hi,
                                        int tr0, int tr1, Lim lim) {
  constexpr int KT = Cfg<KIND>::KT;
  const int g = lane >> 2, j = lane & 3;
  float sc[KT / 8][4];
#pragma unroll
  for (int nt = 0; nt < KT / 8; ++nt) {
    sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
    if (KIND == PISA_CACHE_E2M1) {
      using L = E2m1Tile<U>;
      const int i = nt >> 1;
      const int key = 8 * (nt & 1) + (g >> 1) + 4 * (g & 1);
      uint32_t w0, w1, d0[4], d1[4];
      lds64(st + L::k(i) + key * 32 + 8 * j, w0, w1);
      const uint32_t s1 = lds8(st + L::ks(i) + key * 4 + j);
      const uint32_t s2 = e4m3x2(s1 | (s1 << 8));
      e2m1x8(w0, d0);
      e2m1x8(w1, d1);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        ca_mma<KIND>(sc[nt], s.qa[ks][0], s.qa[ks][1], s.qa[ks][2], s.qa[ks][3], hmul2u(d0[2 * ks], s2),
                     hmul2u(d0[2 * ks + 1], s2));
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        ca_mma<KIND>(sc[nt], s.qa[2 + ks][0], s.qa[2 + ks][1], s.qa[2 + ks][2], s.qa[2 + ks][3],
                     hmul2u(d1[2 * ks], s2), hmul2u(d1[2 * ks + 1], s2));
      }
    } else {
#pragma unroll
      for (int kp = 0; kp < 2; ++kp) {
        uint32_t r[4];
        ldm_x4(st + swz128(8 * nt + (lane & 7), 4 * kp + (lane >> 3)), r);
        ca_mma<KIND>(sc[nt], s.qa[2 * kp][0], s.qa[2 * kp][1], s.qa[2 * kp][2], s.qa[2 * kp][3], r[0], r[1]);
        ca_mma<KIND>(sc[nt], s.qa[2 * kp + 1][0], s.qa[2 * kp + 1][1], s.qa[2 * kp + 1][2], s.qa[2 * kp + 1][3], r[2],
                     r[3]);
      }
    }
  }
  // the running maximum (of the logits times their positive factor) and sum
  float b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
  for (int nt = 0; nt < KT / 8; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (MASK) {
        const int key = 16 * (nt >> 1) + key_of<KIND>(nt & 1, j, e);
        if (key >= v0) sc[nt][e] = -INFINITY;
        if (key >= v1) sc[nt][2 + e] = -INFINITY;
      }
      b0 = fmaxf(b0, sc[nt][e]);
      b1 = fmaxf(b1, sc[nt][2 + e]);
    }
#pragma unroll
  for (int x = 1; x < 4; x <<= 1) {
    b0 = fmaxf(b0, __shfl_xor_sync(kFull, b0, x));
    b1 = fmaxf(b1, __shfl_xor_sync(kFull, b1, x));
  }
  b0 *= s.f0;
  b1 *= s.f1;
  if (__any_sync(kFull, b0 > s.m0 || b1 > s.m1)) {
    const float n0 = fmaxf(s.m0, b0), n1 = fmaxf(s.m1, b1);
    const float a0 = n0 == -INFINITY ? 1.f : ex2_approx(s.m0 - n0), a1 = n1 == -INFINITY ? 1.f : ex2_approx(s.m1 - n1);
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
  }
  // p = 2^(logit - max).  In fp16 it is held times 2^14, so that weights down to 2^-28 of
  // the largest keep all 11 bits (sums of many small weights stay unbiased).
  const float shift = KIND == PISA_CACHE_E2M1 ? kPShift : 0.f;
  const float c0 = s.m0 == -INFINITY ? 0.f : shift - s.m0, c1 = s.m1 == -INFINITY ? 0.f : shift - s.m1;
#pragma unroll
  for (int nt = 0; nt < KT / 8; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      sc[nt][e] = ex2_approx(fmaf(sc[nt][e], s.f0, c0));
      sc[nt][2 + e] = ex2_approx(fmaf(sc[nt][2 + e], s.f1, c1));
      s.l0 += sc[nt][e];
      s.l1 += sc[nt][2 + e];
    }
  // O += P V: the logit fragments of 16 keys are the A fragment
#pragma unroll
  for (int i = 0; i < KT / 16; ++i) {
    const float(&x)[4] = sc[2 * i];
    const float(&y)[4] = sc[2 * i + 1];
    uint32_t hi[4], lo[4];
    if (KIND == PISA_CACHE_E2M1) {
      hi[0] = pack_f16x2(x[0], x[1]);
      hi[1] = pack_f16x2(x[2], x[3]);
      hi[2] = pack_f16x2(y[0], y[1]);
      hi[3] = pack_f16x2(y[2], y[3]);
    } else {  // two bf16 parts hold 16 bits of a weight
      const float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        hi[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
        lo[k] = pack_bf16x2(v[2 * k] - __uint_as_float(hi[k] << 16), v[2 * k + 1] - __uint_as_float(hi[k] & 0xffff0000u));
      }
    }
    uint32_t vb[8][2];
    if (!MASK || t_lo == t_hi) {
      load_v<KIND, U, MASK>(st, i, lane, MASK ? lim(t_lo) : 0, vb);
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        ca_mma<KIND>(s.o[n], hi[0], hi[1], hi[2], hi[3], vb[n][0], vb[n][1]);
        if (KIND == PISA_CACHE_BF16) ca_mma<KIND>(s.o[n], lo[0], lo[1], lo[2], lo[3], vb[n][0], vb[n][1]);
      }
    } else {
      // the rows belong to several queries, which end at different keys: one pass for each,
      // so that an infinite or NaN value of a later key does not reach an earlier query by
      // way of 0 * inf
      for (int t = t_lo; t <= t_hi; ++t) {
        load_v<KIND, U, MASK>(st, i, lane, lim(t), vb);
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          ca_mma<KIND>(d, hi[0], hi[1], hi[2], hi[3], vb[n][0], vb[n][1]);
          if (KIND == PISA_CACHE_BF16) ca_mma<KIND>(d, lo[0], lo[1], lo[2], lo[3], vb[n][0], vb[n][1]);
          if (tr0 == t) {
            s.o[n][0] += d[0];
            s.o[n][1] += d[1];
          }
          if (tr1 == t) {
            s.o[n][2] += d[2];
            s.o[n][3] += d[3];
          }
        }
      }
    }
  }
}

// A unit: the row tile of (sequence b, KV head kv) that starts at row r0.
struct Unit {
  int b, kv, r0, t_first;  // t_first: the query of row 0
  int rows;                // rows of (b, kv): queries * G
  int n;                   // tokens the sequence holds
  const int32_t* sel;      // listed blocks, or nullptr
};

// Tiles [i0, i1) of a unit, shared out among the CTA's warps; on return every warp holds its
// own partial sums.
template <int KIND, int U, bool SEL>
__device__ __forceinline__ void run_tiles(const CacheAttendLaunch& a, const Unit& u, int i0, int i1, uint32_t ring,
                                          int warp, int lane, RowState<KIND>& s) {
  using C = Cfg<KIND>;
  constexpr int KT = C::KT;
  constexpr int E = KT > U ? KT / U : 1;  // records of a tile
  constexpr uint32_t kStage = KT * C::kRow;
  const int g = lane >> 2;
  // what each row sees: tokens before n_vis(t) = n - T + t + 1
  const int ra = u.r0 + g, rb = ra + 8;
  const int tr0 = u.t_first + ra / a.G, tr1 = u.t_first + rb / a.G;
  const int n0 = ra < u.rows ? u.n - a.T + tr0 + 1 : 0, n1 = rb < u.rows ? u.n - a.T + tr1 + 1 : 0;
  const int last = min(u.rows, u.r0 + 16) - 1;
  const int t_lo = u.t_first + u.r0 / a.G, t_hi = u.t_first + last / a.G;
  const int n_lo = u.n - a.T + t_lo + 1, n_hi = u.n - a.T + t_hi + 1;
  const int32_t* table = a.cache.table + (long long)u.b * a.cache.max_pages;

  // Lane l looks ahead: record l % E of the warp's tile number base + l / E.
  long long off = -1;
  int tok = 0x7fffffff;  // the first token of that tile
  auto look = [&](int base) {
    const int i = i0 + warp + kCaWarps * (base + lane / E);
    off = -1;
    tok = 0x7fffffff;
    if (i < i1) {
      int first;
      if (SEL) {
        const int blk = u.sel[i * KT / kC];
        first = blk >= 0 && blk < (1 << 21) ? blk * kC + (i * KT) % kC : 0x7fffffff;
      } else {
        first = i * KT;
      }
      tok = first;
      const long long p = (long long)first + (lane % E) * U;
      if (first < n_hi && p < n_hi) {
        const int page = __ldg(table + (p >> a.cache.page_shift));
        if (page >= 0 && page < a.cache.n_pages) {
          off = cache_record(a.cache, C::kRow, page, u.kv, p);
          // (bf16: the tile may start inside a record)
          if (KIND == PISA_CACHE_BF16 && U > KT) off += (p & (U - 1)) * 128;
        } else {
          off = -2;
        }
      }
    }
    if (__any_sync(kFull, off == -2)) {
      s.bad = true;
      if (off == -2) off = -1;
    }
  };
  auto issue = [&](int seq, int stage) {  // the copies of the warp's tile number seq
    const int l0 = (seq % (32 / E)) * E;
    const uint32_t dst = ring + stage * kStage;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const long long o = __shfl_sync(kFull, off, l0 + e);
      if (o < 0) continue;
      const unsigned char* src = a.cache.pages + o;
      if (KIND == PISA_CACHE_E2M1) {
        constexpr int kChunks = (U < KT ? U : KT) * kRowE2m1 / 16;
#pragma unroll
        for (int c = 0; c < (kChunks + 31) / 32; ++c)
          if (c * 32 + lane < kChunks) cpa16(dst + e * U * kRowE2m1 + (c * 32 + lane) * 16, src + (c * 32 + lane) * 16);
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
    cpa_commit();
  };
  const int mine = i1 - i0 > warp ? (i1 - i0 - warp + kCaWarps - 1) / kCaWarps : 0;  // the warp's tiles
  if (mine == 0) return;
  look(0);
  // the tiles being computed lie one look-ahead behind those being issued, so their first
  // tokens are kept in a queue of the stages
  int first[kCaStages];
  __syncwarp();
#pragma unroll
  for (int x = 0; x < kCaStages - 1; ++x) {
    if (x < mine) {
      if (x && x % (32 / E) == 0) look(x);
      first[x] = __shfl_sync(kFull, tok, (x % (32 / E)) * E);
      issue(x, x);
    } else {
      first[x] = 0x7fffffff;
      cpa_commit();
    }
  }
  int stage = 0;
  for (int x = 0; x < mine; ++x) {
    const int nx = x + kCaStages - 1;
    int stage_n = stage + kCaStages - 1;
    if (stage_n >= kCaStages) stage_n -= kCaStages;
    if (nx < mine) {
      if (nx % (32 / E) == 0) look(nx);
      first[kCaStages - 1] = __shfl_sync(kFull, tok, (nx % (32 / E)) * E);
      issue(nx, stage_n);
    } else {
      cpa_commit();
    }
    cpa_wait<kCaStages - 1>();
    __syncwarp();
    const int f = first[0];
    if (f < n_hi) {
      const uint32_t st = ring + stage * kStage;
      if (f + KT <= n_lo) {
        do_tile<KIND, U, false>(st, lane, s, 0, 0, 0, 0, 0, 0, [](int) { return 0; });
      } else {
        do_tile<KIND, U, true>(st, lane, s, n0 - f, n1 - f, t_lo, t_hi, tr0, tr1,
                               [&](int t) { return u.n - a.T + t + 1 - f; });
      }
    }
    __syncwarp();  // the stage's reads are done before it is refilled
#pragma unroll
    for (int y = 0; y + 1 < kCaStages; ++y) first[y] = first[y + 1];
    stage = stage + 1 == kCaStages ? 0 : stage + 1;
  }
  cpa_wait<0>();
}

// Merges the warps' partial sums; thread (row, quad) of the CTA gets four dims of the sum over
// the warps, its row's maximum and sum.
template <int KIND>
__device__ __forceinline__ float4 merge_warps(RowState<KIND>& s, float* mo, float (*ml)[2][16], int warp, int lane,
                                              float& m, float& l) {
  const int g = lane >> 2, j = lane & 3;
#pragma unroll
  for (int x = 1; x < 4; x <<= 1) {
    s.l0 += __shfl_xor_sync(kFull, s.l0, x);
    s.l1 += __shfl_xor_sync(kFull, s.l1, x);
  }
  if (s.bad) s.l0 = s.l1 = __int_as_float(0x7fc00000);  // a page out of range: the unit's rows become NaN
  if (j == 0) {
    ml[warp][0][g] = s.m0;
    ml[warp][0][g + 8] = s.m1;
    ml[warp][1][g] = s.l0;
    ml[warp][1][g + 8] = s.l1;
  }
  float* o = mo + warp * 1024;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      o[g * 64 + out_dim<KIND>(i, j, e)] = s.o[i][e];
      o[(g + 8) * 64 + out_dim<KIND>(i, j, e)] = s.o[i][2 + e];
    }
  __syncthreads();
  const int row = threadIdx.x >> 4, quad = threadIdx.x & 15;
  m = -INFINITY;
#pragma unroll
  for (int w = 0; w < kCaWarps; ++w) m = fmaxf(m, ml[w][0][row]);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kCaWarps; ++w) {
    const float mw = ml[w][0][row], lw = ml[w][1][row];
    const float f = mw == -INFINITY ? 0.f : ex2_approx(mw - m);
    l += mw == -INFINITY ? lw : f * lw;  // (a warp without keys adds 0, or the NaN of a bad page)
    const float4 x = *reinterpret_cast<const float4*>(mo + w * 1024 + row * 64 + 4 * quad);
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

// Tiles of all units before sequence b (b = B: of all): every warp computes it by itself.
template <int KT>
__device__ __forceinline__ long long tiles_before(const CacheAttendLaunch& a, int b, int units, int lane) {
  long long sum = 0;
  bool over;
  for (int i = lane; i < b; i += 32) sum += (seq_len(a, i, over) + KT - 1) / KT;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(kFull, sum, x);
  return sum * units;
}

// Tiles per CTA of the split form.
__device__ __forceinline__ long long run_length(long long total, int grid) {
  const long long per = (total + grid - 1) / grid;
  return per < kCaMinTiles ? kCaMinTiles : per;
}

template <int KIND>
constexpr int attend_smem() {
  return kCaWarps * kCaStages * Cfg<KIND>::KT * Cfg<KIND>::kRow + kCaWarps * 1024 * 4 + kCaWarps * 2 * 16 * 4;
}

template <int KIND, int U, bool SEL>
__global__ void __launch_bounds__(kCaWarps * 32, Cfg<KIND>::kCtasPerSm) cache_attend_kernel(CacheAttendLaunch a) {
  using C = Cfg<KIND>;
  constexpr int KT = C::KT;
  extern __shared__ __align__(128) unsigned char ca_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_addr(ca_smem) + warp * kCaStages * KT * C::kRow;
  float* mo = reinterpret_cast<float*>(ca_smem + kCaWarps * kCaStages * KT * C::kRow);
  float(*ml)[2][16] = reinterpret_cast<float(*)[2][16]>(mo + kCaWarps * 1024);
  const int row = threadIdx.x >> 4, quad = threadIdx.x & 15;
  RowState<KIND> s;
  Unit u;
  bool over;
  if (SEL) {  // one CTA per (b, t, kv)
    const unsigned id = blockIdx.x;
    u.kv = id % a.cache.Hkv;
    const unsigned bt = id / a.cache.Hkv;
    u.t_first = bt % a.T;
    u.b = bt / a.T;
    u.r0 = 0;
    u.rows = a.G;
    u.n = seq_len(a, u.b, over);
    u.sel = a.idx + (((long long)u.b * a.cache.Hkv + u.kv) * a.T + u.t_first) * a.Ksel;
    load_q<KIND>(a, u.b, u.kv, u.t_first, 0, u.rows, lane, s);
    run_tiles<KIND, U, SEL>(a, u, 0, a.Ksel * (kC / KT), ring, warp, lane, s);
    if (threadIdx.x == 0 && over) set_status(a.status, PISA_ERR_DEVICE_BOUNDS);
    if (lane == 0 && s.bad) set_status(a.status, PISA_ERR_DEVICE_BOUNDS);
    float m, l;
    const float4 acc = merge_warps<KIND>(s, mo, ml, warp, lane, m, l);
    write_out(a, u, row, quad, acc, l);
    return;
  }
  // the split form: this CTA's run of the stream of tiles
  const int RT = (a.T * a.G + 15) / 16;
  const int units = a.cache.Hkv * RT;  // of a sequence
  const long long total = tiles_before<KT>(a, a.cache.B, units, lane);
  const long long per = run_length(total, gridDim.x);
  long long cur = per * blockIdx.x;
  const long long end = cur + per < total ? cur + per : total;
  if (cur >= end) return;
  // the sequence that tile `cur` belongs to: 32 sequences at a time
  long long base = 0;  // tiles before sequence u.b
  int nt = 0;          // tiles of a unit of it
  u.b = 0;
  for (int b0 = 0; b0 < a.cache.B; b0 += 32) {
    const int n = b0 + lane < a.cache.B ? seq_len(a, b0 + lane, over) : 0;
    const long long t = (long long)((n + KT - 1) / KT) * units;
    long long inc = t;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const long long y = __shfl_up_sync(kFull, inc, x);
      if (lane >= x) inc += y;
    }
    const unsigned hit = __ballot_sync(kFull, base + inc > cur);
    if (hit) {
      const int l = __ffs(hit) - 1;
      u.b = b0 + l;
      base += __shfl_sync(kFull, inc - t, l);
      break;
    }
    base += __shfl_sync(kFull, inc, 31);
  }
  u.t_first = 0;
  u.rows = a.T * a.G;
  u.sel = nullptr;
  int slot = 0;
  while (cur < end) {
    u.n = seq_len(a, u.b, over);
    nt = (u.n + KT - 1) / KT;
    if (nt == 0 || cur >= base + (long long)nt * units) {  // on to the next sequence
      base += (long long)nt * units;
      ++u.b;
      continue;
    }
    if (threadIdx.x == 0 && over) set_status(a.status, PISA_ERR_DEVICE_BOUNDS);
    const int un = (int)((cur - base) / nt);
    const int i0 = (int)((cur - base) - (long long)un * nt);
    const int i1 = (int)(end - cur < nt - i0 ? i0 + (end - cur) : nt);
    u.kv = un / RT;
    u.r0 = (un % RT) * 16;
    load_q<KIND>(a, u.b, u.kv, 0, u.r0, u.rows, lane, s);
    run_tiles<KIND, U, SEL>(a, u, i0, i1, ring, warp, lane, s);
    if (lane == 0 && s.bad) set_status(a.status, PISA_ERR_DEVICE_BOUNDS);
    float m, l;
    const float4 acc = merge_warps<KIND>(s, mo, ml, warp, lane, m, l);
    if (i0 == 0 && i1 == nt) {
      write_out(a, u, row, quad, acc, l);
    } else {  // slot 0: the run's first unit, slot 1: its last
      float* p = a.part + ((long long)blockIdx.x * 2 + slot) * kPartFloats;
      *reinterpret_cast<float4*>(p + row * 64 + 4 * quad) = acc;
      if (quad == 0) {
        p[1024 + row] = m;
        p[1040 + row] = l;
      }
    }
    slot = 1;
    cur += i1 - i0;
    __syncthreads();  // the merge buffers are free again
  }
}

// Joins the partial results of the units that lie in several runs, and writes zeros for
// sequences without tokens.  One CTA per (unit, four rows): 4 rows x 16 quads x 4 groups of
// partials.
template <int KT>
__global__ void __launch_bounds__(256) cache_join_kernel(CacheAttendLaunch a, int grid) {
  __shared__ float4 so[4][4][16];
  __shared__ float sm[4][4], sl[4][4];
  const int lane = threadIdx.x & 31;
  const int quad = threadIdx.x & 15, rq = (threadIdx.x >> 4) & 3, grp = threadIdx.x >> 6;
  const int RT = (a.T * a.G + 15) / 16, units = a.cache.Hkv * RT;
  const unsigned id = blockIdx.x >> 2;
  const int row = (blockIdx.x & 3) * 4 + rq;
  Unit u;
  u.b = id / units;
  const int un = id % units;
  u.kv = un / RT;
  u.r0 = (un % RT) * 16;
  u.rows = a.T * a.G;
  u.t_first = 0;
  bool over;
  u.n = seq_len(a, u.b, over);
  const int nt = (u.n + KT - 1) / KT;
  if (nt == 0) {
    if (grp == 0) write_out(a, u, row, quad, make_float4(0.f, 0.f, 0.f, 0.f), 0.f);
    return;
  }
  const long long before = tiles_before<KT>(a, u.b, units, lane);
  const long long total = tiles_before<KT>(a, a.cache.B, units, lane);
  const long long per = run_length(total, grid);
  const long long w0 = before + (long long)un * nt, w1 = w0 + nt;
  const int c0 = (int)(w0 / per), c1 = (int)((w1 - 1) / per);
  if (c0 == c1) return;  // a run held all of it and wrote it
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = c0 + grp; c <= c1; c += 4) {
    const int slot = c == c0 && w0 > per * c ? 1 : 0;
    const float* p = a.part + ((long long)c * 2 + slot) * kPartFloats;
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
  m = fmaxf(fmaxf(sm[0][rq], sm[1][rq]), fmaxf(sm[2][rq], sm[3][rq]));
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  l = 0.f;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
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

template <int KIND, int U, bool SEL>
static cudaError_t launch_attend_t(const CacheAttendLaunch& L, cudaStream_t s) {
  using C = Cfg<KIND>;
  constexpr int smem = attend_smem<KIND>();
  // (the attribute belongs to the device, so it is set for each call's: a host-side cost of about 1 us)
  cudaError_t e = cudaFuncSetAttribute(cache_attend_kernel<KIND, U, SEL>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  if (SEL) {
    cache_attend_kernel<KIND, U, SEL>
        <<<(unsigned)(L.cache.B * L.T * L.cache.Hkv), kCaWarps * 32, smem, s>>>(L);
    note_launch();
    return cudaGetLastError();
  }
  const int RT = (L.T * L.G + 15) / 16;
  const int grid = 152 * C::kCtasPerSm;
  cache_attend_kernel<KIND, U, SEL><<<grid, kCaWarps * 32, smem, s>>>(L);
  note_launch();
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cache_join_kernel<C::KT><<<(unsigned)(L.cache.B * L.cache.Hkv * RT * 4), 256, 0, s>>>(L, grid);
  note_launch();
  return cudaGetLastError();
}

template <int KIND, int U>
static cudaError_t launch_attend_u(const CacheAttendLaunch& L, cudaStream_t s) {
  return L.idx ? launch_attend_t<KIND, U, true>(L, s) : launch_attend_t<KIND, U, false>(L, s);
}

cudaError_t launch_cache_attend(const CacheAttendLaunch& L, cudaStream_t s) {
  if (L.cache.kind == PISA_CACHE_BF16) switch (L.cache.rec_shift) {
      case 4: return launch_attend_u<PISA_CACHE_BF16, 16>(L, s);
      case 5: return launch_attend_u<PISA_CACHE_BF16, 32>(L, s);
      default: return launch_attend_u<PISA_CACHE_BF16, 64>(L, s);
    }
  switch (L.cache.rec_shift) {
    case 4: return launch_attend_u<PISA_CACHE_E2M1, 16>(L, s);
    case 5: return launch_attend_u<PISA_CACHE_E2M1, 32>(L, s);
    default: return launch_attend_u<PISA_CACHE_E2M1, 64>(L, s);
  }
}

}  // namespace pisa
