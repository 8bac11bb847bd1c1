// cache_prompt.cuh -- attention of a prompt's tokens over the paged cache: the launch's description.
#pragma once

#include "cache.cuh"

namespace pisa {

constexpr int kPromptRuns = 152;               // CTAs of the stream form: one on each SM
constexpr int kPromptUnits = 8 * kPromptRuns;  // row tiles that it takes at most

// A piece of the stream: tiles k0 .. k1 - 1 of a unit (-1: none), and which partial result it leaves (-1: it is the
// whole unit).
struct PromptPiece {
  int unit, k0, k1, slot;
};
// In the workspace.
struct PromptPlan {
  PromptPiece* piece;  // [kPromptUnits + kPromptRuns]
  // [kPromptRuns] the unit that begins in a run and goes on (-1: none), and the last run that it lies in
  int2* cut;
  int32_t* tiles;      // [kPromptUnits]
};
constexpr size_t kPromptPlanBytes = (kPromptUnits + kPromptRuns) * sizeof(PromptPiece) + kPromptRuns * sizeof(int2) +
                                    kPromptUnits * sizeof(int32_t);

struct CachePromptLaunch {
  CacheDev cache;
  RowsDev q;
  int T, Hq, G;
  const int32_t* start;
  const int32_t* counts;  // may be nullptr: T of every sequence
  const int32_t* first;   // [B, T] first token that a query sees, or nullptr: 0
  const int32_t* last;    // [B, T] token behind the last that it sees, or nullptr: its own position + 1
  ScoreDev score;
  __nv_bfloat16* out;  // [B, T, Hq, 64]
  int* status;
  // of the stream form (cache_prompt.cu):
  PromptPlan plan;
  float* part;  // partial results
};

// The tokens that query t of sequence b sees: lo .. hi - 1 (none where hi <= lo).  Positions are cut to what
// the table holds; `over` says that they were.
struct Span {
  int pos, lo, hi;
};
__device__ __forceinline__ Span span_of(const CachePromptLaunch& a, int b, int t, int count, bool& over) {
  const long long cap = (long long)a.cache.max_pages << a.cache.page_shift;
  const long long start = a.start[b], p = start + t, end = start + count;
  over = start < 0 || end > cap;
  Span s;
  // (one past either end of the table as the end itself: that adds as much to the distance of all that it sees, and
  // stays far from 32 bits' ends)
  s.pos = (int)(p < 0 ? 0 : p > cap ? cap : p);
  long long hi = a.last ? a.last[(long long)b * a.T + t] : p + 1, lo = a.first ? a.first[(long long)b * a.T + t] : 0;
  hi = hi < end ? hi : end;
  hi = hi < cap ? hi : cap;
  if (a.score.window < kNoWindow && p - a.score.window + 1 > lo) lo = p - a.score.window + 1;
  s.lo = (int)(lo < 0 ? 0 : lo > cap ? cap : lo);
  s.hi = (int)(hi < 0 ? 0 : hi);
  return s;
}

__device__ __forceinline__ int prompt_count(const CachePromptLaunch& a, int b) {
  return a.counts ? min(max(a.counts[b], 0), a.T) : a.T;
}

size_t cache_prompt_part_bytes();
cudaError_t launch_cache_prompt(const CachePromptLaunch& L, cudaStream_t s);

}  // namespace pisa
