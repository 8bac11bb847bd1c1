"""The stream that attention's split form cuts into runs: the split kernel's and the joining kernel's index arithmetic,
compiled for the host from the header that both take it from, and replayed against one another."""
import ctypes
import os
import random
import re
import subprocess

import numpy as np
import pytest

from test_cache_sources import CSRC, code_of

HOST = r"""
#include <cstdint>
#include <map>
#include <vector>
#define __host__
#define __device__
#define __forceinline__ inline
#include "cache_stream.cuh"
using namespace pisa;

struct Part { int b; unsigned un; int i0, i1; };
struct SeqTiles { int first, tiles, places; };
template <int KT, bool WINDOWED>
static SeqTiles seq_tiles(int n, int T, int window, int change) {
  const int tiles = unit_tiles<KT, WINDOWED>(n, T, window);
  const int places = change == 36 ? unit_places<36>(tiles) : unit_places<24>(tiles);
  return {first_tile<KT, WINDOWED>(n, T, window), tiles, places};
}

// Replays a call on `runs` runs, `units` units a sequence.  Returns 0, or which rule does not hold.
template <int KT, bool WINDOWED>
static int replay(const int* n, int B, int T, int window, int change, int units, int runs, int64_t* cuts) {
  std::vector<long long> base(B + 1, 0);
  for (int b = 0; b < B; ++b)
    base[b + 1] = base[b] + (long long)seq_tiles<KT, WINDOWED>(n[b], T, window, change).places * units;
  const long long total = base[B], per = run_length(total, runs);
  if (per * runs < total) return 1;
  // the split kernel: a unit's result, or up to two partial ones a run (slot 1: the unit begins in the run)
  std::map<std::pair<int, int>, Part> part;
  std::map<std::pair<int, unsigned>, int> whole, tiles;
  for (int run = 0; run < runs; ++run) {
    long long cur = per * run;
    const long long end = cur + per < total ? cur + per : total;
    int b = 0;
    while (cur < end) {
      while (cur >= base[b + 1]) ++b;
      const SeqTiles s = seq_tiles<KT, WINDOWED>(n[b], T, window, change);
      const unsigned un = unit_at(cur - base[b], s.places);
      const int i0 = (int)(cur - base[b] - (long long)un * s.places);
      if (un >= (unsigned)units) return 2;
      if (i0 >= s.tiles) {
        cur += s.places - i0;
        continue;
      }
      const int i1 = (int)(end - cur < s.tiles - i0 ? i0 + (end - cur) : s.tiles);
      tiles[{b, un}] += i1 - i0;
      if (i0 == 0 && i1 == s.tiles) {
        ++whole[{b, un}];
      } else {
        if (part.count({run, i0 == 0})) return 3;
        part[{run, i0 == 0}] = Part{b, un, i0, i1};
      }
      cur += i1 < s.tiles ? i1 - i0 : s.places - i0;
    }
  }
  // what a unit has to have: tiles up to the sequence's end, from the first one that a query sees
  for (int b = 0; b < B; ++b) {
    const SeqTiles s = seq_tiles<KT, WINDOWED>(n[b], T, window, change);
    long long lo = WINDOWED ? (long long)n[b] - T + 1 - window : 0;
    if (lo < 0) lo = 0;
    if (n[b] && (s.first * (long long)KT > lo || (s.first + 1) * (long long)KT <= lo)) return 4;
    const long long stop = s.first + s.tiles;
    if (n[b] && (stop * KT < n[b] || (stop - 1) * KT >= n[b])) return 5;
    for (int un = 0; un < units; ++un)
      if (tiles[{b, un}] != s.tiles) return 6;
  }
  // the joining kernel, both forms of it: the same units, each from all of its parts in order
  std::map<std::pair<int, unsigned>, int> joined[2];
  auto join = [&](int form, int b, unsigned un, long long w0, int nt, int c0) {
    int c1 = 0;
    if (!goes_on(w0, nt, per, c0, c1)) return 0;
    if (c1 <= c0 || c1 >= runs) return 10;
    int at = 0;
    for (int c = c0; c <= c1; ++c) {
      const auto p = part.find({c, c == c0});
      if (p == part.end() || p->second.b != b || p->second.un != un || p->second.i0 != at) return 11;
      at = p->second.i1;
    }
    if (at != nt) return 12;
    ++joined[form][{b, un}];
    return 0;
  };
  for (int run = 0; run < runs; ++run) {  // by the run's last place
    const long long end = per * (run + 1);
    if (end >= total) continue;
    int b = 0;
    while (end - 1 >= base[b + 1]) ++b;
    const SeqTiles s = seq_tiles<KT, WINDOWED>(n[b], T, window, change);
    const unsigned un = unit_at(end - 1 - base[b], s.places);
    if (const int bad = join(0, b, un, base[b] + (long long)un * s.places, s.tiles, run)) return bad;
  }
  for (int b = 0; b < B; ++b)  // unit by unit
    for (int un = 0; un < units; ++un) {
      const SeqTiles s = seq_tiles<KT, WINDOWED>(n[b], T, window, change);
      const long long w0 = base[b] + (long long)un * s.places;
      if (const int bad = join(1, b, un, w0, s.tiles, (int)(w0 / per))) return bad;
    }
  *cuts += joined[1].size();
  for (int b = 0; b < B; ++b)
    for (unsigned un = 0; un < (unsigned)units; ++un)
      for (auto& j : joined)
        if (whole[{b, un}] + j[{b, un}] != (n[b] > 0)) return 20;
  return 0;
}
extern "C" int call(const int* n, int B, int T, int window, int kt, int change, int units, int runs, int windowed,
                    int64_t* cuts) {
  const auto f = kt == 32 ? (windowed ? replay<32, true> : replay<32, false>)
                          : (windowed ? replay<64, true> : replay<64, false>);
  return f(n, B, T, window, change, units, runs, cuts);
}
"""


@pytest.fixture(scope="module")
def call(tmp_path_factory):
    d = tmp_path_factory.mktemp("stream")
    (d / "s.cpp").write_text(HOST)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I" + CSRC, str(d / "s.cpp"), "-o",
                    str(d / "s.so")], check=True)
    fn = ctypes.CDLL(str(d / "s.so")).call

    def run(lengths, T, window, kt, change, units, runs):
        n, cuts = np.asarray(lengths, np.int32), ctypes.c_int64()
        bad = fn(n.ctypes.data_as(ctypes.c_void_p), n.size, T, 1 << 28 if window is None else window, kt, change,
                 units, runs, int(window is not None), ctypes.byref(cuts))
        return bad, cuts.value

    return run


# tiles of 32 keys (bf16 pages; row tiles side by side share the grid out) and of 64 (4 bits), places at a unit's end
KINDS = [(32, 36), (64, 24)]


@pytest.mark.parametrize("kt,change", KINDS)
@pytest.mark.parametrize("lengths,T,window,units,runs", [
    ([16384] * 32, 1, 4096, 2, 152),
    ([131072] * 64, 1, 16384, 8, 152),
    ([262144] * 3, 16, 4096, 1, 9),
    ([20000, 100, 0, 4096, 4097, 70000] * 8, 1, 4096, 2, 152),
    ([9000 + 517 * b for b in range(40)], 4, 5000, 6, 152),
    ([131072] * 16, 1, None, 2, 152),
])
def test_cut_units_are_joined(call, kt, change, lengths, T, window, units, runs):
    bad, cuts = call(lengths, T, window, kt, change, units, runs)
    assert bad == 0 and cuts > 0


@pytest.mark.parametrize("kt,change", KINDS)
def test_any_lengths(call, kt, change):
    rng = random.Random(kt)
    cuts = 0
    for _ in range(400):
        B, top = rng.randint(1, 70), int(2 ** rng.uniform(1, 19))
        lengths = [rng.choice([top, rng.randint(0, top), rng.randint(0, 40)]) for _ in range(B)]
        args = (lengths, rng.randint(1, 16), rng.choice([None, 1, int(2 ** rng.uniform(0, 19))]), rng.randint(1, 12),
                rng.choice([152, 76, 9, 1]))
        bad, n = call(args[0], args[1], args[2], kt, change, args[3], args[4])
        assert bad == 0, (bad, args)
        cuts += n
    assert cuts > 400


def test_the_kernels_take_the_arithmetic_from_the_header():
    """Neither kernel counts tiles, places or runs of a sequence by itself."""
    text = code_of("cache_attend.cuh")
    for name in ("cache_attend_split_kernel", "cache_join_kernel"):
        body = re.search(name + r"\(CacheAttendLaunch a.*?\n}\n", text, re.S).group(0)
        for part in ("tiles_of_seq<KIND, MODE>", "places_of<KIND>", "run_length(", "unit_at("):
            assert part in body
        body = body.replace("c0 = (int)(w0 / per)", "").replace("first_tile<C::KT, ", "")
        assert not re.search(r"\bKT\b|kChange|/ per|/ \(unsigned\)", body)
    assert text.count("goes_on(") == 2


def test_the_kinds_are_the_kernels():
    text = code_of("cache_attend.cuh")
    got = [(int(a), int(b)) for a, b in re.findall(r"int KT = (\d+);.*?int kChange = (\d+);", text, re.S)]
    assert got == KINDS and os.path.exists(os.path.join(CSRC, "cache_stream.cuh"))
