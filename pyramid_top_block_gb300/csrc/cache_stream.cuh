// cache_stream.cuh -- the arithmetic of the stream that attention's split form cuts into runs (cache_attend.cuh):
// which tiles the units of a sequence have, which places of the stream they take, which unit holds a place, and which
// runs a unit lies in.  The split kernel and the joining one have to agree on all of it, so both take it from here.
// Whole numbers alone: it compiles for the host as well, where its test replays both kernels.
#pragma once

namespace pisa {

constexpr int kCaMinTiles = 12;  // places of the stream that a run has at least

// A unit (KV head and row tile) of a sequence of n tokens, whose newest T are queries: the first tile that any of them
// sees ..
template <int KT, bool WINDOWED>
__host__ __device__ __forceinline__ int first_tile(int n, int T, int window) {
  const int before = WINDOWED ? n - T + 1 - window : 0;  // tokens before the first query's window
  return before > 0 ? before / KT : 0;
}
// .. how many there are, ..
template <int KT, bool WINDOWED>
__host__ __device__ __forceinline__ int unit_tiles(int n, int T, int window) {
  return (n + KT - 1) / KT - first_tile<KT, WINDOWED>(n, T, window);
}
// .. and their places in the stream: the tiles, and CHANGE more for the unit's end.
// (All three as one struct from one function: 8 x 131072 tokens of bf16, T = 3, 141.2 instead of 137.5 us, T = 8 352
// instead of 342.)
template <int CHANGE>
__host__ __device__ __forceinline__ int unit_places(int tiles) {
  return tiles ? tiles + CHANGE : 0;
}

// Places of a run.
__host__ __device__ __forceinline__ long long run_length(long long total, int runs) {
  const long long per = total < (1 << 30) ? ((int)total + runs - 1) / runs : (total + runs - 1) / runs;
  return per < kCaMinTiles ? kCaMinTiles : per;
}

// The unit of a sequence that holds place `at` behind the sequence's first, each unit having `places`.
// (places of one sequence: below 2^22 * 32 heads * 16 row tiles + 2^15, within 32 bits)
__host__ __device__ __forceinline__ unsigned unit_at(long long at, int places) {
  return (unsigned)at / (unsigned)places;
}

// Whether a unit, its tiles at the places w0 .. w0 + tiles - 1, begins in run `run` and goes on in others; `last` is
// the last of them.
__host__ __device__ __forceinline__ bool goes_on(long long w0, int tiles, long long per, int run, int& last) {
  const long long begin = per * run, end = begin + per, w1 = w0 + tiles;
  if (tiles == 0 || w0 < begin || w0 >= end || w1 <= end) return false;
  last = (int)((w1 - 1) / per);
  return true;
}

}  // namespace pisa
