// cache_append.cu -- new queries and keys are rotated by their positions, keys and values go
// into the pages of a paged cache; and the way back, cached tokens as dense bf16 rows.
//
// Rotation of a pair (a, b) at a position with cosine c and sine s:
//   a' = a c - b s,  b' = b c + a s
// Eight lanes hold one row of 64 (16 bytes each), a warp four rows.  In the split-halves
// order the other member of a pair is rot/2 dims away, which is a whole number of lanes, so
// it comes by shuffle; in the interleaved order it is the neighbouring element.  Query rows
// that turn as a whole in halves have four lanes, each with both members of eight pairs: no
// shuffle, and each element is unpacked once (53.2 -> 50.7 us for 32768 tokens).
//
// Both kernels only move rows, so the bytes of the rows in and out bound them.  Measured: 32768
// tokens of 32 + 2 + 2 heads into bf16 pages (319 MB) 49.8 us = 6.40 TB/s; 131072 tokens of 2
// heads read back from 4 bits (86 MB) 16.1 us = 5.35 TB/s; 65 single tokens 1.9 us.  With positions on
// three axes 32768 tokens take 58.7 us: images' angles come from three rows, a pair's word at a time.
#include "cache.cuh"

#include <type_traits>

namespace pisa {

constexpr int kAppWarps = 4;
constexpr int kAppPrefetch = 912;  // tokens ahead (six an SM) whose rows are asked into L2: 61.4 -> 57 us for 32768
constexpr int kAppBatch = 2;  // groups of four rows whose loads a warp issues together, ahead of their use

// x c + p s rounded to 32 bits from nearly twice as many: both products and their sum as
// unevaluated pairs (the error of a product by fma, that of a sum by Knuth's two-sum), off by at
// most 2^-46 (|x c| + |p s|) before the last rounding.  Every step is rounded by itself, by
// intrinsics: a product fused into one of the sums would count its error twice.
__device__ __forceinline__ float sum2(float x, float c, float p, float s) {
  const float h1 = __fmul_rn(x, c), h2 = __fmul_rn(p, s);
  const float l1 = __fmaf_rn(x, c, -h1), l2 = __fmaf_rn(p, s, -h2);
  const float h = __fadd_rn(h1, h2), z = __fsub_rn(h, h1);
  const float e = __fadd_rn(__fsub_rn(h1, __fsub_rn(h, z)), __fsub_rn(h2, z));
  const float l = __fadd_rn(e, __fadd_rn(l1, l2));
  return fabsf(h) < INFINITY ? __fadd_rn(h, l) : h;  // (an infinity has no error term)
}

// Eight rotated elements x c + p s (p the pair's other member, s signed), as the bf16 values
// that the exact sum rounds to (by way of 32 bits).  In 32 bits the sum r is off by at most
// (|p s| + |r|) 2^-24 (results below 2^-100 aside); where every value within twice that
// rounds to the same bf16 that is the answer, else (one element in some thousands) the sums
// are taken with their errors.  (Whether the compiler fuses a product into e or r +- e does not
// matter: twice the error leaves room for that.)  So a key has the same bits however it was
// appended, which matters where it is quantised next.  The branch takes the products from here
// because both are the same intrinsic; with * here the kernel took 53.4 us instead of 49.8 for
// 32768 tokens.  (64-bit arithmetic in the branch cost half of the kernel's time: the compiler
// hoists the conversions, and the 64-bit pipe is slow.)
// there: whether the row exists and turns (the zeros of one that does not would take the
// branch: r - e and r + e of a negative zero differ).
__device__ __forceinline__ void rotate8(uint32_t (&w)[4], const uint32_t (&o)[4], const float (&c)[8],
                                        const float (&s)[8], bool there) {
  uint32_t lo[4], differ = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float x0 = __uint_as_float(w[k] << 16), x1 = __uint_as_float(w[k] & 0xffff0000u);
    const float p0 = __uint_as_float(o[k] << 16), p1 = __uint_as_float(o[k] & 0xffff0000u);
    const float m0 = __fmul_rn(p0, s[2 * k]), m1 = __fmul_rn(p1, s[2 * k + 1]);
    const float r0 = fmaf(x0, c[2 * k], m0), r1 = fmaf(x1, c[2 * k + 1], m1);
    const float e0 = (fabsf(m0) + fabsf(r0)) * 0x1p-23f, e1 = (fabsf(m1) + fabsf(r1)) * 0x1p-23f;
    lo[k] = pack_bf16x2(r0 - e0, r1 - e1);
    differ |= lo[k] ^ pack_bf16x2(r0 + e0, r1 + e1);
  }
  if (differ && there) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      lo[k] = pack_bf16x2(sum2(__uint_as_float(w[k] << 16), c[2 * k], __uint_as_float(o[k] << 16), s[2 * k]),
                          sum2(__uint_as_float(w[k] & 0xffff0000u), c[2 * k + 1],
                               __uint_as_float(o[k] & 0xffff0000u), s[2 * k + 1]));
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = lo[k];
}

// Both members of eight pairs (a, b), from the same lane: a' = a c - b s, b' = b c + a s, the same
// bits as rotate8 gives.
__device__ __forceinline__ void rotate_pairs(uint32_t (&a)[4], uint32_t (&b)[4], const float (&c)[8],
                                             const float (&s)[8], bool there) {
  uint32_t na[4], nb[4], differ = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float r[2][2], e[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float x = __uint_as_float(h ? a[k] & 0xffff0000u : a[k] << 16);
      const float y = __uint_as_float(h ? b[k] & 0xffff0000u : b[k] << 16);
      const float m = __fmul_rn(y, -s[2 * k + h]), n = __fmul_rn(x, s[2 * k + h]);
      r[0][h] = fmaf(x, c[2 * k + h], m);
      r[1][h] = fmaf(y, c[2 * k + h], n);
      e[0][h] = (fabsf(m) + fabsf(r[0][h])) * 0x1p-23f;
      e[1][h] = (fabsf(n) + fabsf(r[1][h])) * 0x1p-23f;
    }
    na[k] = pack_bf16x2(r[0][0] - e[0][0], r[0][1] - e[0][1]);
    nb[k] = pack_bf16x2(r[1][0] - e[1][0], r[1][1] - e[1][1]);
    differ |= na[k] ^ pack_bf16x2(r[0][0] + e[0][0], r[0][1] + e[0][1]);
    differ |= nb[k] ^ pack_bf16x2(r[1][0] + e[1][0], r[1][1] + e[1][1]);
  }
  if (differ && there) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x0 = __uint_as_float(a[k] << 16), x1 = __uint_as_float(a[k] & 0xffff0000u);
      const float y0 = __uint_as_float(b[k] << 16), y1 = __uint_as_float(b[k] & 0xffff0000u);
      na[k] = pack_bf16x2(sum2(x0, c[2 * k], y0, -s[2 * k]), sum2(x1, c[2 * k + 1], y1, -s[2 * k + 1]));
      nb[k] = pack_bf16x2(sum2(y0, c[2 * k], x0, s[2 * k]), sum2(y1, c[2 * k + 1], x1, s[2 * k + 1]));
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    a[k] = na[k];
    b[k] = nb[k];
  }
}

// The 4-bit form of a row: this lane's 8 of 64 values (bf16 pairs w) and, with the
// neighbouring lane's, the scale of their 16.  Steps, each exact or rounded once:
//   top = largest |x| (compared as integers, so that an infinity or a NaN is the largest)
//   scale = e4m3(top 2^-exp / 6), to nearest even, at most 448; code = e2m1(x 2^-exp / scale)
// x is a bf16 (8 bits) and a border between two codes times the scale has at most 7, so a
// quotient that is not on a border is at least 2^-10 from it (borders lie in [1/4, 5], and
// so does any quotient near one).  x times the reciprocal (off by 2^-23 of itself), rounded
// once or, with the sum below fused, not at all, is off by 2^-20 there at most; rounding it
// to a multiple of 2^-11 (by adding 1.5 * 2^12) puts the quotients that are on a border exactly
// there and moves no other one across, so the conversion's ties-to-even rule decides them.
// Likewise the scale: six times a border between two e4m3 numbers has at most 7 bits, so a
// top / 6 that is not a border is at least 2^-8 of itself from it, and 16 bits hold every border.
__device__ __forceinline__ void quantise8(const uint32_t (&w)[4], int exp, uint32_t& codes, uint32_t& scale) {
  uint32_t t = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                        __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
  t = max(t & 0xffffu, t >> 16);
  t = max(t, __shfl_xor_sync(kFull, t, 1));
  const float down = exp2i(-exp);
  // top / 6, off by less than 2^-22 of it, snapped to 16 bits
  const uint32_t q = (__float_as_uint(__uint_as_float(t << 16) * down * (1.f / 6.f)) + 0x80u) & 0xffffff00u;
  scale = __nv_cvt_float_to_fp8(__uint_as_float(q), __NV_SATFINITE, __NV_E4M3);
  const float sv = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)scale, __NV_E4M3)));
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(sv));
  inv = sv > 0.f ? inv * down : 0.f;
  constexpr float kSnap = 6144.f;  // 1.5 * 2^12: sums near it are multiples of 2^-11
  float z[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    z[2 * i] = (__uint_as_float(w[i] << 16) * inv + kSnap) - kSnap;
    z[2 * i + 1] = (__uint_as_float(w[i] & 0xffff0000u) * inv + kSnap) - kSnap;
  }
  asm("{ .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d}; }"
      : "=r"(codes)
      : "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7]));
  if (t >= 0x7f80u) {  // an infinity or a NaN among the 16: the block stands for NaNs
    scale = 0x7f;
    codes = 0;
  }
}

// The rotation of this lane's 8 dims at one position.
struct Turn {
  float c[8], s[8];  // cosines and signed sines
  int from;          // lane that holds the pairs' other members (split halves)
  bool on;           // whether the dims turn at all
};

// Whether a query row's pairs lie in one lane: the two halves of a row that turns as a whole.
template <bool INTER, bool FULL>
constexpr bool kPairs = FULL && !INTER;

constexpr int kMaxAxes = 4;

// Where the angles of a token's axes lie: its positions times rot / 16, in steps of 16 floats (positions are below
// 2^27 where there are axes).
struct AxisRows {
  uint32_t at[kMaxAxes];
  bool one;  // all axes agree, as in text
};

// The angles of pairs i .. i + N - 1, each from its own axis's row: every lane of the warp loads those of the pair of
// its number, and the lanes take them from one another (each its own pairs' by word loads took 59.6 instead of
// 58.7 us for 32768 tokens).
template <int N>
__device__ __forceinline__ void load_axes(const CacheAppendLaunch& a, const AxisRows& rows, int lane, int i,
                                          float (&u)[N], float (&v)[N]) {
  float c = 0.f, s = 0.f;
  if (lane < a.rot >> 1) {
    const unsigned axis = (unsigned)(a.axis_of >> (2 * lane)) & 3u;
    const uint32_t lo = axis & 1 ? rows.at[1] : rows.at[0], hi = axis & 1 ? rows.at[3] : rows.at[2];
    const float* row = a.rotary + (size_t)(axis & 2 ? hi : lo) * 16 + lane;
    c = row[0];
    s = row[a.rot >> 1];
  }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    u[e] = __shfl_sync(kFull, c, i + e);
    v[e] = __shfl_sync(kFull, s, i + e);
  }
}

template <bool INTER, bool AXES>
__device__ __forceinline__ void load_turn(const CacheAppendLaunch& a, long long p, const AxisRows& rows, int lane,
                                          Turn& t) {
  const int c = lane & 7;
  const int half = a.rot >> 4;  // lanes of one half of the rotated dims (split-halves order)
  t.on = c < 2 * half;
  t.from = lane;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    t.c[e] = 1.f;
    t.s[e] = 0.f;
  }
  const bool low = c < half;
  constexpr int kAngles = INTER ? 4 : 8;  // of a lane
  float uu[kAngles], vv[kAngles];
  const bool apart = AXES && !rows.one;  // (the same for the whole warp)
  if (apart) load_axes(a, rows, lane, INTER ? 4 * c : 8 * (low ? c : c - half), uu, vv);
  if (!t.on) return;
  const float* row = a.rotary + p * a.rot;
  if constexpr (INTER) {
    if (!apart) {
      const float4 u = *reinterpret_cast<const float4*>(row + 4 * c);
      const float4 v = *reinterpret_cast<const float4*>(row + (a.rot >> 1) + 4 * c);
      uu[0] = u.x, uu[1] = u.y, uu[2] = u.z, uu[3] = u.w;
      vv[0] = v.x, vv[1] = v.y, vv[2] = v.z, vv[3] = v.w;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      t.c[e] = uu[e >> 1];
      t.s[e] = (e & 1) ? vv[e >> 1] : -vv[e >> 1];
    }
  } else {
    t.from = low ? lane + half : lane - half;
    if (!apart) {
      const float4* u = reinterpret_cast<const float4*>(row + 8 * (low ? c : c - half));
      const float4* v = reinterpret_cast<const float4*>(row + (a.rot >> 1) + 8 * (low ? c : c - half));
      const float4 u0 = u[0], u1 = u[1], v0 = v[0], v1 = v[1];
      uu[0] = u0.x, uu[1] = u0.y, uu[2] = u0.z, uu[3] = u0.w, uu[4] = u1.x, uu[5] = u1.y, uu[6] = u1.z, uu[7] = u1.w;
      vv[0] = v0.x, vv[1] = v0.y, vv[2] = v0.z, vv[3] = v0.w, vv[4] = v1.x, vv[5] = v1.y, vv[6] = v1.z, vv[7] = v1.w;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      t.c[e] = uu[e];
      t.s[e] = low ? -vv[e] : vv[e];
    }
  }
}

// rotate: whether the row exists and turns.  (Lanes that do not turn compute as well and keep
// their words: cheaper than a branch.)  ALL: every lane's dims turn, and what becomes of a row
// that does not exist does not matter.
template <bool INTER, bool ALL>
__device__ __forceinline__ void turn_row(const Turn& t, bool rotate, uint32_t (&w)[4]) {
  uint32_t o[4], y[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    o[k] = INTER ? __byte_perm(w[k], 0, 0x1032) : __shfl_sync(kFull, w[k], t.from);
    y[k] = w[k];
  }
  rotate8(y, o, t.c, t.s, (ALL || t.on) && rotate);
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = ALL || (t.on && rotate) ? y[k] : w[k];
}

// A warp takes every parts-th group of four rows of one token: the groups of its query rows,
// then those of its key and value rows (keys first).  FULL: all 64 dims turn (the query rows then
// need no choice between old and new words: 55.8 -> 53.2 us for 32768 tokens).
// AXES: a token turns by positions of its own, one for each axis, instead of its place in the cache.
template <int KIND, bool INTER, bool FULL, bool AXES>
__global__ void __launch_bounds__(kAppWarps * 32, 6) cache_append_kernel(CacheAppendLaunch a, int parts) {
  after_the_one_before();
  const int lane = threadIdx.x & 31, sub = lane >> 3, c = lane & 7;
  const int job = blockIdx.x * kAppWarps + __shfl_sync(kFull, threadIdx.x >> 5, 0);  // (token, part)
  const int t = job / parts, part = job - t * parts, b = blockIdx.z;
  if (t >= a.T) return;
  const int Hkv = a.cache.Hkv, Hq = a.q.data ? a.Hq : 0;
  // (a prompt's rows behind its count are not even read; a single token's are, rather than wait)
  if (a.T > 1 && a.counts && t >= a.counts[b]) return;
  // PAIRS: a lane has dims 8 (lane & 3) .. + 7 of a query row, whose angles load_turn gives it, and
  // their partners 32 dims on; a group is eight rows.  Else as in key and value rows.
  constexpr bool PAIRS = kPairs<INTER, FULL>;
  constexpr int kRows = PAIRS ? 8 : 4;
  const int qsub = PAIRS ? lane >> 2 : sub, qcol = PAIRS ? 8 * (lane & 3) : 8 * c;
  const int gq = (Hq + kRows - 1) / kRows, groups = gq + ((2 * Hkv + 3) >> 2);
  // the rows this lane has a part in: query row kRows i + qsub of group i, row 4 (i - gq) + sub of
  // keys and values
  const __nv_bfloat16* qs = a.q.data + b * a.q.sb + t * a.q.st + (kRows * part + qsub) * a.q.sh + qcol;
  const long long step = kRows * parts * a.q.sh;
  constexpr int kTurns = PAIRS ? 1 : kAppBatch;  // groups of a batch
  const int turns = kTurns * parts;
  auto fetch_q = [&](int i, uint4 (&z)[kAppBatch]) {
#pragma unroll
    for (int n = 0; n < kAppBatch; ++n) {
      z[n] = make_uint4(0, 0, 0, 0);
      const int g = PAIRS ? i : i + n * parts;
      if (kRows * g + qsub < Hq) z[n] = *reinterpret_cast<const uint4*>(PAIRS ? qs + 32 * n : qs + n * step);
    }
    qs += kTurns * step;
  };
  uint4 x[kAppBatch];
  fetch_q(part, x);  // (these loads do not wait for the position)
  int ikv = part - gq;
  if (ikv < 0) ikv += (-ikv + parts - 1) / parts * parts;
  auto fetch_kv = [&](int i) {
    const int r = 4 * i + sub;
    const RowsDev& src = r < Hkv ? a.k : a.v;
    const int kv = r < Hkv ? r : r - Hkv;
    uint4 z = make_uint4(0, 0, 0, 0);
    if (r < 2 * Hkv) z = *reinterpret_cast<const uint4*>(src.data + b * src.sb + t * src.st + kv * src.sh + 8 * c);
    return z;
  };
  uint4 xkv = fetch_kv(ikv);
  AxisRows rows;
  long long turn_at = 0;  // the position that a token whose axes agree turns by
  bool placed = true;  // whether all positions are in the table
  if constexpr (AXES) {
    int at[kMaxAxes];
#pragma unroll
    for (int x = 0; x < kMaxAxes; ++x)
      at[x] = x < a.n_axes ? a.positions[((long long)x * a.cache.B + b) * a.T + t] : at[0];
    rows.one = true;
    turn_at = at[0];
#pragma unroll
    for (int x = 0; x < kMaxAxes; ++x) {
      placed = placed && at[x] >= 0 && at[x] < a.n_rot;
      rows.one = rows.one && at[x] == at[0];
      rows.at[x] = (uint32_t)at[x] * (uint32_t)(a.rot >> 4);
    }
  }
  const int count = a.counts ? a.counts[b] : a.T;
  const long long p = (long long)a.start[b] + t;
  if (t >= count) return;
  if (parts == 1 && t + kAppPrefetch < min(count, a.T)) {  // a prompt: a later token's rows and angles into L2
    const int later = t + kAppPrefetch;
    for (int r = lane; r < Hq + 2 * Hkv; r += 32) {
      const RowsDev& from = r < Hq ? a.q : r < Hq + Hkv ? a.k : a.v;
      const int h = r < Hq ? r : r < Hq + Hkv ? r - Hq : r - Hq - Hkv;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(from.data + b * from.sb + later * from.st + h * from.sh));
    }
    const long long at = (long long)a.start[b] + later;
    if (!AXES && lane < 2 && a.rot && at >= 0 && at < a.n_rot)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.rotary + at * a.rot + (a.rot > 32 ? 32 * lane : 0)));
  }
  const long long cap = (long long)a.cache.max_pages << a.cache.page_shift;
  bool ok = p >= 0 && p < cap && (AXES ? placed : a.rot == 0 || p < a.n_rot);
  int page = -1;
  Turn turn;
  if (ok) {
    page = a.cache.table[(long long)b * a.cache.max_pages + (p >> a.cache.page_shift)];
    load_turn<INTER, AXES>(a, AXES ? turn_at : p, rows, lane, turn);
    ok = page >= 0 && page < a.cache.n_pages;
  }
  if (!ok) {  // the token is left out
    if (lane == 0) set_status(a.status, PISA_ERR_DEVICE_BOUNDS);
    return;
  }
  __nv_bfloat16* qd = a.q_out.data + b * a.q_out.sb + t * a.q_out.st + (kRows * part + qsub) * a.q_out.sh + qcol;
  const long long step_out = kRows * parts * a.q_out.sh;
  auto put_q = [&](int i, const uint4 (&z)[kAppBatch]) {
    if constexpr (PAIRS) {
      const bool there = 8 * i + qsub < Hq;
      uint32_t u[4] = {z[0].x, z[0].y, z[0].z, z[0].w}, w[4] = {z[1].x, z[1].y, z[1].z, z[1].w};
      rotate_pairs(u, w, turn.c, turn.s, there);
      if (there) {
        *reinterpret_cast<uint4*>(qd) = make_uint4(u[0], u[1], u[2], u[3]);
        *reinterpret_cast<uint4*>(qd + 32) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      qd += step_out;
    } else {
#pragma unroll
      for (int n = 0; n < kAppBatch; ++n) {
        uint32_t w[4] = {z[n].x, z[n].y, z[n].z, z[n].w};
        turn_row<INTER, FULL>(turn, 4 * (i + n * parts) + sub < Hq, w);
        if (4 * (i + n * parts) + sub < Hq) *reinterpret_cast<uint4*>(qd) = make_uint4(w[0], w[1], w[2], w[3]);
        qd += step_out;
      }
    }
  };
  auto put_kv = [&] {
    const int U = 1 << a.cache.rec_shift, u = (int)(p & (U - 1));
    for (int i = ikv; i < groups - gq; i += parts) {
      const int r = 4 * i + sub;
      const bool is_v = r >= Hkv, there = r < 2 * Hkv;
      const int kv = is_v ? r - Hkv : r;
      uint32_t w[4] = {xkv.x, xkv.y, xkv.z, xkv.w};
      xkv = fetch_kv(i + parts);
      turn_row<INTER, false>(turn, !is_v && there, w);
      const uint4 y = make_uint4(w[0], w[1], w[2], w[3]);
      if (!is_v && a.k_out.data)
        *reinterpret_cast<uint4*>(a.k_out.data + b * a.k_out.sb + t * a.k_out.st + kv * a.k_out.sh + 8 * c) = y;
      if (KIND == PISA_CACHE_BF16) {
        if (there) {
          unsigned char* rec = a.cache.pages + cache_record(a.cache, kRowBf16, page, kv, p) + (is_v ? U * 128 : 0);
          *reinterpret_cast<uint4*>(rec + u * 128 + 16 * c) = y;
        }
      } else {
        uint32_t codes, scale;
        quantise8(w, is_v ? a.cache.v_exp : a.cache.k_exp, codes, scale);
        if (there) {
          unsigned char* rec = a.cache.pages + cache_record(a.cache, kRowE2m1, page, kv, p) + (is_v ? U * 36 : 0);
          *reinterpret_cast<uint32_t*>(rec + u * 32 + 4 * c) = codes;
          if (!(c & 1)) rec[U * 32 + u * 4 + (c >> 1)] = (unsigned char)scale;
        }
      }
    }
  };
  // Keys and values first, while the query rows are on their way (in the interleaved order last,
  // which is faster there: 51.7 and 55.1 us for 32768 tokens; in halves 50.7 and 49.7).
  if constexpr (PAIRS) {
    put_kv();
#pragma unroll
    for (int e = 0; e < 8; ++e) turn.s[e] = c < 4 ? -turn.s[e] : turn.s[e];  // (a lane has both halves of a query row)
  }
  // (two batches a turn, so that neither is copied)
  for (int i = part; i < gq; i += 2 * turns) {
    uint4 y[kAppBatch];
    fetch_q(i + turns, y);
    put_q(i, x);
    if (i + turns >= gq) break;
    fetch_q(i + 2 * turns, x);
    put_q(i + turns, y);
  }
  if constexpr (!PAIRS) put_kv();
}

// A warp reads kReadBatch groups of four tokens of one head, eight lanes a token.
constexpr int kReadBatch = 2;

template <int KIND>
__global__ void __launch_bounds__(256) cache_read_kernel(CacheReadLaunch a) {
  after_the_one_before();
  const int lane = threadIdx.x & 31, c = lane & 7, b = blockIdx.z, kv = blockIdx.y;
  const int t0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * (4 * kReadBatch) + (lane >> 3);
  const int n = a.counts ? min(a.T, a.counts[b]) : a.T;
  const long long first = a.start[b], cap = (long long)a.cache.max_pages << a.cache.page_shift;
  const int32_t* table = a.cache.table + (long long)b * a.cache.max_pages;
  const int U = 1 << a.cache.rec_shift;
  constexpr int kRow = KIND == PISA_CACHE_BF16 ? kRowBf16 : kRowE2m1;
  const unsigned char* rec[kReadBatch];
  bool ok[kReadBatch];
#pragma unroll
  for (int i = 0; i < kReadBatch; ++i) {
    const int t = t0 + 4 * i;
    const long long p = first + t;
    int page = 0;
    ok[i] = t < n;
    if (ok[i]) {
      page = p >= 0 && p < cap ? table[p >> a.cache.page_shift] : -1;
      if (page < 0 || page >= a.cache.n_pages) {
        if (c == 0) set_status(a.status, PISA_ERR_DEVICE_BOUNDS);
        ok[i] = false;
        page = 0;
      }
    }
    // (in bounds whether ok or not: the row of p's remainder in page 0)
    const int u = (int)(p & (U - 1));
    rec[i] = a.cache.pages + cache_record(a.cache, kRow, page, kv, p) + u * (KIND == PISA_CACHE_BF16 ? 128 : 32);
  }
  if (KIND == PISA_CACHE_BF16) {
    uint4 y[kReadBatch][2];
#pragma unroll
    for (int i = 0; i < kReadBatch; ++i) {
      if (!ok[i]) continue;
      y[i][0] = *reinterpret_cast<const uint4*>(rec[i] + 16 * c);
      y[i][1] = *reinterpret_cast<const uint4*>(rec[i] + U * 128 + 16 * c);
    }
#pragma unroll
    for (int i = 0; i < kReadBatch; ++i) {
      if (!ok[i]) continue;
      const long long t = t0 + 4 * i;
      if (a.k_out.data)
        *reinterpret_cast<uint4*>(a.k_out.data + b * a.k_out.sb + t * a.k_out.st + kv * a.k_out.sh + 8 * c) = y[i][0];
      if (a.v_out.data)
        *reinterpret_cast<uint4*>(a.v_out.data + b * a.v_out.sb + t * a.v_out.st + kv * a.v_out.sh + 8 * c) = y[i][1];
    }
  } else {
    uint32_t w[kReadBatch][2], z[kReadBatch][2];
#pragma unroll
    for (int i = 0; i < kReadBatch; ++i) {
      if (!ok[i]) continue;
      const int u = (int)((first + t0 + 4 * i) & (U - 1));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        w[i][h] = *reinterpret_cast<const uint32_t*>(rec[i] + h * 36 * U + 4 * c);
        z[i][h] = rec[i][h * 36 * U + 32 * U - 28 * u + (c >> 1)];
      }
    }
#pragma unroll
    for (int i = 0; i < kReadBatch; ++i) {
      if (!ok[i]) continue;
      const long long t = t0 + 4 * i;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const RowsDev& dst = h ? a.v_out : a.k_out;
        const uint32_t s = e4m3x2(z[i][h]);
        const float f = __low2float(*reinterpret_cast<const __half2*>(&s)) * exp2i(h ? a.cache.v_exp : a.cache.k_exp);
        uint32_t d[4], o[4];
        e2m1x8(w[i][h], d);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&d[k]));
          o[k] = pack_bf16x2(v.x * f, v.y * f);
        }
        if (dst.data)
          *reinterpret_cast<uint4*>(dst.data + b * dst.sb + t * dst.st + kv * dst.sh + 8 * c) =
              make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

cudaError_t launch_cache_append(const CacheAppendLaunch& L, cudaStream_t s) {
  const int rows = L.rot == kD && !L.interleaved ? 8 : 4;  // of a group of query rows (see kPairs)
  const int groups = ((L.q.data ? L.Hq : 0) + rows - 1) / rows + (2 * L.cache.Hkv + 3) / 4;
  // One warp a token where there are many; where there are few, as many as there are groups
  // of rows, so that a step's latency is one row's.
  const long long tokens = (long long)L.cache.B * L.T;
  int parts = 1;
  while (parts < groups && tokens * parts < 152 * 16) ++parts;
  const dim3 grid((unsigned)(((long long)L.T * parts + kAppWarps - 1) / kAppWarps), 1, (unsigned)L.cache.B);
  constexpr int kThreads = kAppWarps * 32;
  const auto launch = [&](auto kind, auto inter, auto axes) {
    constexpr int kKind = decltype(kind)::value;
    constexpr bool kInter = decltype(inter)::value, kAxes = decltype(axes)::value;
    return L.rot == kD ? launch_early<cache_append_kernel<kKind, kInter, true, kAxes>>(grid, kThreads, 0, s, L, parts)
                       : launch_early<cache_append_kernel<kKind, kInter, false, kAxes>>(grid, kThreads, 0, s, L, parts);
  };
  const auto go = [&](auto kind, auto inter) {
    return L.positions ? launch(kind, inter, std::true_type{}) : launch(kind, inter, std::false_type{});
  };
  using Bf16 = std::integral_constant<int, PISA_CACHE_BF16>;
  using E2m1 = std::integral_constant<int, PISA_CACHE_E2M1>;
  if (L.cache.kind == PISA_CACHE_BF16)
    return L.interleaved ? go(Bf16{}, std::true_type{}) : go(Bf16{}, std::false_type{});
  return L.interleaved ? go(E2m1{}, std::true_type{}) : go(E2m1{}, std::false_type{});
}

cudaError_t launch_cache_read(const CacheReadLaunch& L, cudaStream_t s) {
  const dim3 grid((unsigned)((L.T + 32 * kReadBatch - 1) / (32 * kReadBatch)), (unsigned)L.cache.Hkv,
                  (unsigned)L.cache.B);
  if (L.cache.kind == PISA_CACHE_BF16) return launch_early<cache_read_kernel<PISA_CACHE_BF16>>(grid, 256, 0, s, L);
  return launch_early<cache_read_kernel<PISA_CACHE_E2M1>>(grid, 256, 0, s, L);
}

}  // namespace pisa
