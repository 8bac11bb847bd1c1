"""What the cache kernels' sources must keep to, checked on their text and on their host-compiled arithmetic."""
import ctypes
import os
import re
import subprocess
from fractions import Fraction

import numpy as np
import pytest

import pyramid_top_block_gb300 as pisa

CSRC = os.path.join(os.path.dirname(pisa.__file__), "csrc")


def code_of(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


EARLY = sorted(f for f in os.listdir(CSRC) if "griddepcontrol" in code_of(f) or "launch_early" in code_of(f))


def test_the_early_kernels_are_found():
    assert {"cache.cuh", "cache_append.cu", "cache_attend.cuh"} <= set(EARLY)


@pytest.mark.parametrize("name", EARLY)
def test_kernels_that_start_early_load_coherently(name):
    """A kernel that starts while the one before it still writes may not use the read-only path: such a load
    promises that nothing writes the memory while the kernel lives, and may move ahead of the wait."""
    found = re.findall(r"__ldg\b|\bld\.global(?:\.\w+)*\.nc\b|__restrict__|__ldlu\b", code_of(name))
    assert not found, found


# ------------------------------------------------------------------- the rotation's sum with its error terms


HOST = r"""
#include <cmath>
#include <cstdint>
#define __device__
#define __forceinline__ inline
// A float whose products are fused into every sum that takes them, which a compiler may do.
struct Num {
  float v, a = 0, b = 0;
  bool product = false;
  Num(float x = 0) : v(x) {}
};
static Num operator-(Num x) { return Num(-x.v); }
static Num operator*(Num x, Num y) {
  Num r(x.v * y.v);
  r.a = x.v, r.b = y.v, r.product = true;
  return r;
}
static Num operator+(Num x, Num y) {
  if (x.product) return Num(std::fma(x.a, x.b, y.v));
  if (y.product) return Num(std::fma(y.a, y.b, x.v));
  return Num(x.v + y.v);
}
static Num operator-(Num x, Num y) {
  if (x.product) return Num(std::fma(x.a, x.b, -y.v));
  if (y.product) return Num(std::fma(-y.a, y.b, x.v));
  return Num(x.v - y.v);
}
static bool operator<(Num x, Num y) { return x.v < y.v; }
// one rounding each, and never fused
static Num __fmul_rn(Num a, Num b) { return Num((a * b).v); }
static Num __fadd_rn(Num a, Num b) { return Num(a.v + b.v); }
static Num __fsub_rn(Num a, Num b) { return Num(a.v - b.v); }
static Num __fmaf_rn(Num a, Num b, Num c) { return Num(std::fma(a.v, b.v, c.v)); }
static Num fmaf(Num a, Num b, Num c) { return Num(std::fma(a.v, b.v, c.v)); }
static Num fabsf(Num a) { return Num(std::fabs(a.v)); }
#define float Num
%s
#undef float
extern "C" void sums(const float* x, const float* c, const float* p, const float* s, float* out, int64_t n) {
  for (int64_t i = 0; i < n; ++i) out[i] = sum2(x[i], c[i], p[i], s[i]).v;
}
"""


def bf16(x):
    """fp32 values of x cut to bf16 (they only have to be such values)."""
    return (np.asarray(x, np.float32).view(np.uint32) & np.uint32(0xffff0000)).view(np.float32)


def test_rotation_sum_where_products_may_be_fused(tmp_path):
    """sum2 gives the exact x c + p s rounded to 32 bits also where products are fused into sums, as the CUDA
    compiler may do.  Off by more than half a step only by what its error term loses: 2^-24 of the parts of that
    term, which are at most 2^-24 (|h| + |x c| + |p s|), twice; so at most 2^-46 (|x c| + |p s|)."""
    source = re.search(r"__device__ __forceinline__ float sum2\(.*?\n}\n", code_of("cache_append.cu"), re.S)
    assert source
    src, lib = tmp_path / "sum2.cpp", tmp_path / "sum2.so"
    src.write_text(HOST % source.group(0))
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-shared", "-fPIC", str(src), "-o", str(lib)],
                   check=True)
    fn = ctypes.CDLL(str(lib)).sums
    rng = np.random.default_rng(1)
    n = 20000
    x, p = bf16(rng.standard_normal(n)), bf16(rng.standard_normal(n))
    angle = rng.uniform(0, 100, n)
    c, s = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    # a quarter cancels almost, a quarter lies next to a border between two bf16 values
    k = n // 4
    c[:k] = (-p[:k].astype(np.float64) * s[:k] / x[:k]).astype(np.float32)
    border = bf16(rng.standard_normal(k)).astype(np.float64)
    border += np.ldexp(1.0, np.frexp(border)[1] - 9)  # half of a bf16's step on
    c[k:2 * k] = ((border - p[k:2 * k].astype(np.float64) * s[k:2 * k]) / x[k:2 * k]).astype(np.float32)
    out = np.empty(n, np.float32)
    ptr = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    fn(ptr(x), ptr(c), ptr(p), ptr(s), ptr(out), ctypes.c_int64(n))
    bad = 0
    for i in range(n):
        a, b = Fraction(float(x[i])) * Fraction(float(c[i])), Fraction(float(p[i])) * Fraction(float(s[i]))
        step = Fraction(float(np.spacing(np.abs(out[i]))))
        bad += abs(Fraction(float(out[i])) - (a + b)) > step / 2 + Fraction(1, 1 << 46) * (abs(a) + abs(b))
    assert bad == 0, f"{bad} of {n}"
