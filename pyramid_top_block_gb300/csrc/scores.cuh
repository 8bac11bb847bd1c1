// scores.cuh -- scores that are not plain products: capped by a tanh, with a bias by distance.
//
//   x = q . k / 8;  cap > 0: x = cap tanh(x / cap);  x -= slope |p - j|  (p the query's position, j the key's)
// In base 2, as the softmax takes them.
#pragma once

#include "tc.cuh"

namespace pisa {

constexpr int kNoWindow = 1 << 28;  // past every position (tokens are below 2^27)

// What is done to the scores of a call (cap 0: not capped; slopes nullptr: no bias; window kNoWindow: none).
struct ScoreDev {
  float cap, inv_cap;
  const float* slopes;  // [Hq]
  int window;           // a query sees tokens p - window + 1 and later
};

// A head's slope in base 2.  Past 2^96 it is cut, so that times a distance, below 2^28, it fits 32 bits.
__device__ __forceinline__ float slope2(const ScoreDev& s, int head) {
  return fminf(fmaxf(s.slopes[head], -0x1p96f), 0x1p96f) * 1.4426950408889634f;
}

// tanh(y) / y as polynomials in u = y y: the interpolations at the Chebyshev nodes, of degree 6 on |y| <= 1, off by at
// most 6.0e-8 of the value (a rounding to 32 bits), and of degree 3 on |y| <= 1/2 (5.6e-07).  One minus twice the
// reciprocal of 1 + e^(2 y) would take two slow instructions a score, and loses small scores' last bits.
struct Tanh {
  static constexpr int n = 7;
  float c[n] = {0x1.fffffep-1f, -0x1.555402p-2f, 0x1.10e5c6p-3f, -0x1.b5e03ap-5f,
                0x1.4c4342p-6f, -0x1.95f386p-8f, 0x1.101cb0p-10f};
};
struct TanhHalf {
  static constexpr int n = 4;
  float c[n] = {0x1.ffffeep-1f, -0x1.5542dap-2f, 0x1.0e2146p-3f, -0x1.6baa52p-5f};
};
__device__ __forceinline__ unsigned long long f2_mul(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// tanh(y) / y of two values.
template <typename P>
__device__ __forceinline__ unsigned long long tanh_ratio(unsigned long long y) {
  constexpr P k;
  const unsigned long long u = f2_mul(y, y);
  unsigned long long q = f2_pack(k.c[P::n - 1], k.c[P::n - 1]);
#pragma unroll
  for (int i = P::n - 2; i >= 0; --i) q = f2_fma(q, u, f2_pack(k.c[i], k.c[i]));
  return q;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Factors of a row: y = score * to_y (to the cap's units), logit = score * to_l tanh(y) / y.
// Large ones are cut, so that a product of zero stays zero: a 4-bit page's other products, 2^-34 or more, are far past
// the cap then.
struct CapRow {
  float to_y, to_l;
};
__device__ __forceinline__ CapRow cap_row(float factor, float inv_cap) {
  return CapRow{fminf(factor * inv_cap, 0x1p100f), fminf(factor * 1.4426950408889634f, 0x1.fffffep127f)};
}

// Factors of the short polynomial: logit = x (c[0] + x x (c[1] + ..)), x the product.  They fit 32 bits for
// kCapLeast <= to_y <= kCapMost (caps are at most 2^20).  4-bit pages' products are below 2^19: with a smaller to_y the
// last factor may fall below 2^-149, but what is lost of a logit is below 2^-18 of the larger of it and 1.
struct CapPoly {
  float c[TanhHalf::n];
};
constexpr float kCapLeast = 0x1p-18f, kCapMost = 0x1p10f;
__device__ __forceinline__ CapPoly cap_poly(const CapRow& r) {
  constexpr TanhHalf k;
  CapPoly p;
  float f = r.to_l;
#pragma unroll
  for (int i = 0; i < TanhHalf::n; ++i, f = f * r.to_y * r.to_y) p.c[i] = k.c[i] * f;
  return p;
}

// Two scores with |y| <= 1, capped.
__device__ __forceinline__ void cap_small(float& a, float& b, const CapRow& r) {
  const unsigned long long x = f2_pack(a, b);
  f2_unpack(f2_mul(f2_mul(x, f2_pack(r.to_l, r.to_l)), tanh_ratio<Tanh>(f2_mul(x, f2_pack(r.to_y, r.to_y)))), a, b);
}

// Two scores of any size, capped: cap tanh y = cap - 2 cap / (1 + e^(2 y)), off by up to 2^-20.5 of the cap (so 1.3e-4
// in base 2 for a cap of 128, the largest that this is used for).  An infinity gives plus or minus the cap, a NaN a
// NaN.  two = 2 log2 e to_y, top = cap log2 e.
__device__ __forceinline__ void cap_exp(float& a, float& b, float two, float top) {
  float x, y;
  f2_unpack(f2_mul(f2_pack(a, b), f2_pack(two, two)), x, y);
  f2_unpack(f2_add(f2_pack(ex2_approx(x), ex2_approx(y)), f2_pack(1.f, 1.f)), x, y);
  f2_unpack(f2_fma(f2_pack(rcp_approx(x), rcp_approx(y)), f2_pack(-2.f * top, -2.f * top), f2_pack(top, top)), a, b);
}
constexpr float kCapExp = 128.f;

// One score of any size, capped; top = cap log2 e.  An infinity gives plus or minus top, a NaN a NaN.
__device__ __forceinline__ float cap_any(float x, const CapRow& r, float top) {
  const float y = fabsf(x * r.to_y);
  if (!(y <= 1.f)) {
    const float e = ex2_approx(-2.f * 1.4426950408889634f * y);  // tanh y = (1 - e) / (1 + e)
    return copysignf(top, x) * __fdividef(1.f - e, 1.f + e);
  }
  const float u = y * y;
  constexpr Tanh k;
  float q = k.c[6];
#pragma unroll
  for (int i = 5; i >= 0; --i) q = fmaf(q, u, k.c[i]);
  return x * r.to_l * q;
}

}  // namespace pisa
