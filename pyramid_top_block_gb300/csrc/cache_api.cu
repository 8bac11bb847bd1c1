// cache_api.cu -- the C ABI of the paged KV cache (include/pisa.h): argument checks and
// launches.  No allocation, no exceptions, one stream.
#include "cache.cuh"
#include "pool.cuh"
#include "cache_prompt.cuh"

using namespace pisa;

namespace {

constexpr size_t kCacheStatusBytes = 256;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int page_shift_of(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

// Checks a cache descriptor and fills in the kernels' form of it.
int check_cache(const pisa_paged_cache* c, CacheDev& d) {
  if (!c || !c->pages || !c->table) return PISA_ERR_INVALID_ARG;
  if (c->B < 1 || c->Hkv < 1 || c->n_pages < 1 || c->max_pages < 1 || c->page_size < 1) return PISA_ERR_INVALID_ARG;
  if (!aligned(c->pages, 16) || !aligned(c->table, 4)) return PISA_ERR_INVALID_ARG;
  const int shift = page_shift_of(c->page_size);
  if (shift < 0 || c->d != kD || c->Hkv > 32 || (long long)c->B * c->Hkv > 65535) return PISA_ERR_UNSUPPORTED;
  if (c->kind != PISA_CACHE_BF16 && c->kind != PISA_CACHE_E2M1) return PISA_ERR_UNSUPPORTED;
  if (((long long)c->max_pages << shift) > (1LL << 27)) return PISA_ERR_UNSUPPORTED;
  if (c->kind == PISA_CACHE_BF16 ? (c->k_exp || c->v_exp)
                                 : (c->k_exp < -24 || c->k_exp > 24 || c->v_exp < -24 || c->v_exp > 24))
    return PISA_ERR_UNSUPPORTED;
  if (c->page_stride % 16 || c->page_stride < (int64_t)pisa_cache_page_bytes(c->page_size, c->Hkv, c->kind))
    return PISA_ERR_INVALID_ARG;
  if (c->page_stride > (INT64_MAX >> 1) / c->n_pages) return PISA_ERR_INVALID_ARG;
  d.pages = static_cast<unsigned char*>(c->pages);
  d.table = c->table;
  d.page_stride = c->page_stride;
  d.B = c->B;
  d.Hkv = c->Hkv;
  d.n_pages = c->n_pages;
  d.max_pages = c->max_pages;
  d.page_shift = shift;
  d.rec_shift = shift < kLog2C ? shift : kLog2C;
  d.kind = c->kind;
  d.k_exp = c->k_exp;
  d.v_exp = c->v_exp;
  return PISA_OK;
}

// Rows of an operand (nullptr: absent, allowed only when `optional`).
int check_rows(const pisa_rows* r, bool optional, RowsDev& d) {
  d = RowsDev{nullptr, 0, 0, 0};
  if (!r || !r->data) return optional ? PISA_OK : PISA_ERR_INVALID_ARG;
  if (!aligned(r->data, 16) || ((r->stride_b | r->stride_t | r->stride_h) & 7)) return PISA_ERR_INVALID_ARG;
  d = RowsDev{static_cast<__nv_bfloat16*>(r->data), r->stride_b, r->stride_t, r->stride_h};
  return PISA_OK;
}

bool group_ok(int Hq, int Hkv) {
  if (Hq < 1 || Hq % Hkv) return false;
  const int G = Hq / Hkv;
  return G <= 16 && (G & (G - 1)) == 0;
}

// What is done to the scores.  (The cap's limits keep its reciprocal, and the cap in base 2, within 32 bits.)
int check_score(float cap, const float* slopes, int window, ScoreDev& d) {
  if (!aligned(slopes, 4) || window < 0 || !(cap >= 0.f)) return PISA_ERR_INVALID_ARG;
  if (cap != 0.f && (cap < 0x1p-20f || cap > 0x1p20f)) return PISA_ERR_UNSUPPORTED;
  d = ScoreDev{cap, cap > 0.f ? 1.f / cap : 0.f, slopes, window == 0 || window > kNoWindow ? kNoWindow : window};
  return PISA_OK;
}

// Checks a pool descriptor.
int check_pool(const pisa_page_pool* c, PoolDev& d) {
  if (!c || !c->pages || !c->table || !c->refs) return PISA_ERR_INVALID_ARG;
  if (c->B < 1 || c->n_pages < 1 || c->max_pages < 1 || c->page_size < 1 || c->page_bytes < 1)
    return PISA_ERR_INVALID_ARG;
  if (!aligned(c->pages, 16) || !aligned(c->table, 4) || !aligned(c->refs, 4)) return PISA_ERR_INVALID_ARG;
  if (c->page_bytes % 16 || c->page_stride % 16 || c->page_stride < c->page_bytes) return PISA_ERR_INVALID_ARG;
  if (c->page_stride > (INT64_MAX >> 1) / c->n_pages) return PISA_ERR_INVALID_ARG;
  const int shift = page_shift_of(c->page_size);
  if (shift < 0 || ((long long)c->max_pages << shift) > (1LL << 27)) return PISA_ERR_UNSUPPORTED;
  // (a page's pieces are numbered in 32 bits; so are the pages of a cluster's eighths, with room for a turn more)
  if (c->B > 65535 || c->n_pages > (1 << 30) || c->page_bytes > (1LL << 40)) return PISA_ERR_UNSUPPORTED;
  d.pages = static_cast<unsigned char*>(c->pages);
  d.table = c->table;
  d.refs = c->refs;
  d.page_stride = c->page_stride;
  d.page_bytes = c->page_bytes;
  d.B = c->B;
  d.n_pages = c->n_pages;
  d.max_pages = c->max_pages;
  d.page_shift = shift;
  return PISA_OK;
}

// Whether two lists of whole numbers share entries (none: nullptr).
bool overlap(const int32_t* a, long long n, const int32_t* b, long long m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + 4 * (uintptr_t)m && y < x + 4 * (uintptr_t)n;
}

// Whether a list of n entries that a call writes lies in what it keeps in line.
bool in_pool(const PoolDev& p, const int32_t* x, long long n) {
  return overlap(x, n, p.table, (long long)p.B * p.max_pages) || overlap(x, n, p.refs, p.n_pages);
}

// The lists of whole numbers behind the status word.
PoolScratch pool_scratch(const PoolDev& p, void* ws) {
  int32_t* x = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + kCacheStatusBytes);
  PoolScratch s;
  s.counts = x;
  s.list_a = x + 64;
  s.list_b = s.list_a + p.n_pages;
  s.list_c = s.list_b + p.n_pages;
  s.per_seq = s.list_c + p.n_pages;
  return s;
}

int cuda_code(cudaError_t e) { return e == cudaSuccess ? PISA_OK : PISA_ERR_CUDA; }

}  // namespace

extern "C" {

size_t pisa_cache_page_bytes(int page_size, int Hkv, int kind) {
  if (page_shift_of(page_size) < 0 || Hkv < 1 || Hkv > 32) return 0;
  if (kind != PISA_CACHE_BF16 && kind != PISA_CACHE_E2M1) return 0;
  return (size_t)page_size * Hkv * (kind == PISA_CACHE_BF16 ? kRowBf16 : kRowE2m1);
}

size_t pisa_cache_workspace_bytes(void) {
  const size_t a = cache_part_bytes(), b = cache_prompt_part_bytes();
  return kCacheStatusBytes + (a > b ? a : b);
}

size_t pisa_cache_attention_workspace_bytes(void) { return kCacheStatusBytes + cache_part_bytes(); }

static int cache_append(const pisa_paged_cache* cache, int T, const pisa_rows* q, int Hq, const pisa_rows* k,
                      const pisa_rows* v, const int32_t* start, const int32_t* counts, const float* rotary,
                      int64_t n_rot, int rot, int interleaved, const pisa_rows* q_out, const pisa_rows* k_out,
                      const int32_t* positions, int n_axes, uint64_t axis_of, void* ws, void* stream) {
  CacheAppendLaunch L{};
  int st = check_cache(cache, L.cache);
  if (st) return st;
  const bool with_q = q && q->data;
  if (T < 1 || !start || (with_q && Hq < 1)) return PISA_ERR_INVALID_ARG;
  if ((st = check_rows(q, true, L.q)) || (st = check_rows(k, false, L.k)) || (st = check_rows(v, false, L.v)) ||
      (st = check_rows(q_out, !with_q, L.q_out)) || (st = check_rows(k_out, true, L.k_out)))
    return st;
  if (rot < 0 || rot > kD || rot % 16) return PISA_ERR_UNSUPPORTED;
  if (rot && (!rotary || !aligned(rotary, 16) || n_rot < 1)) return PISA_ERR_INVALID_ARG;
  if (with_q && !group_ok(Hq, cache->Hkv)) return PISA_ERR_UNSUPPORTED;
  if (!aligned(start, 4) || !aligned(counts, 4) || !aligned(ws, 4)) return PISA_ERR_INVALID_ARG;
  // 32-bit job numbers: at most one for four rows of a token
  if ((long long)T * (((with_q ? Hq : 0) + 2 * cache->Hkv + 7) / 4) >= (1LL << 31) - 1024) return PISA_ERR_UNSUPPORTED;
  L.T = T;
  L.Hq = Hq;
  L.start = start;
  L.counts = counts;
  L.rotary = rotary;
  L.n_rot = n_rot;
  L.rot = rot;
  L.interleaved = interleaved != 0;
  L.positions = positions;
  L.n_axes = n_axes;
  L.axis_of = axis_of;
  L.status = static_cast<int*>(ws);
  return cuda_code(launch_cache_append(L, static_cast<cudaStream_t>(stream)));
}

int pisa_cache_append(const pisa_paged_cache* cache, int T, const pisa_rows* q, int Hq, const pisa_rows* k,
                      const pisa_rows* v, const int32_t* start, const int32_t* counts, const float* rotary,
                      int64_t n_rot, int rot, int interleaved, const pisa_rows* q_out, const pisa_rows* k_out,
                      void* ws, void* stream) {
  return cache_append(cache, T, q, Hq, k, v, start, counts, rotary, n_rot, rot, interleaved, q_out, k_out, nullptr, 0,
                      0, ws, stream);
}

int pisa_cache_append_axes(const pisa_paged_cache* cache, int T, const pisa_rows* q, int Hq, const pisa_rows* k,
                           const pisa_rows* v, const int32_t* start, const int32_t* counts, const float* rotary,
                           int64_t n_rot, int rot, int interleaved, const int32_t* positions, int n_axes,
                           uint64_t axis_of, const pisa_rows* q_out, const pisa_rows* k_out, void* ws, void* stream) {
  if (!positions || !aligned(positions, 4) || n_axes < 1 || rot < 1) return PISA_ERR_INVALID_ARG;
  if (n_axes > 4 || n_rot > (1LL << 27) || rot > kD || rot % 16) return PISA_ERR_UNSUPPORTED;
  for (int i = 0; i < rot / 2; ++i)
    if ((int)(axis_of >> (2 * i) & 3) >= n_axes) return PISA_ERR_INVALID_ARG;
  return cache_append(cache, T, q, Hq, k, v, start, counts, rotary, n_rot, rot, interleaved, q_out, k_out, positions,
                      n_axes, axis_of, ws, stream);
}

int pisa_cache_read(const pisa_paged_cache* cache, int T, const int32_t* start, const int32_t* counts,
                    const pisa_rows* k_out, const pisa_rows* v_out, void* ws, void* stream) {
  CacheReadLaunch L{};
  int st = check_cache(cache, L.cache);
  if (st) return st;
  if (T < 1 || !start) return PISA_ERR_INVALID_ARG;
  if ((st = check_rows(k_out, true, L.k_out)) || (st = check_rows(v_out, true, L.v_out))) return st;
  if (!L.k_out.data && !L.v_out.data) return PISA_ERR_INVALID_ARG;
  if (!aligned(start, 4) || !aligned(counts, 4) || !aligned(ws, 4)) return PISA_ERR_INVALID_ARG;
  if (T >= (1 << 30)) return PISA_ERR_UNSUPPORTED;  // 32-bit token numbers
  L.T = T;
  L.start = start;
  L.counts = counts;
  L.status = static_cast<int*>(ws);
  return cuda_code(launch_cache_read(L, static_cast<cudaStream_t>(stream)));
}

static int cache_attention(const pisa_paged_cache* cache, const pisa_rows* q, int T, int Hq, const int32_t* lengths,
                           const int32_t* idx, int Ksel, const ScoreDev* score, void* out, int out_f32, void* ws,
                           size_t ws_bytes, void* stream) {
  CacheAttendLaunch L{};
  int st = check_cache(cache, L.cache);
  if (st) return st;
  if (T < 1 || Hq < 1 || !lengths || !out || !ws) return PISA_ERR_INVALID_ARG;
  if ((st = check_rows(q, false, L.q))) return st;
  if (!aligned(out, 16) || !aligned(ws, 256) || !aligned(lengths, 4) || !aligned(idx, 4)) return PISA_ERR_INVALID_ARG;
  if (T > kCacheMaxT || !group_ok(Hq, cache->Hkv)) return PISA_ERR_UNSUPPORTED;
  if (idx && (Ksel < 1 || Ksel > kCacheMaxSel)) return PISA_ERR_UNSUPPORTED;
  if ((long long)cache->B * T * cache->Hkv >= (1LL << 24)) return PISA_ERR_UNSUPPORTED;
  if (ws_bytes < pisa_cache_attention_workspace_bytes()) return PISA_ERR_WORKSPACE_TOO_SMALL;
  L.T = T;
  L.Hq = Hq;
  L.G = Hq / cache->Hkv;
  L.lengths = lengths;
  L.idx = idx;
  L.Ksel = Ksel;
  L.out = out;
  L.out_f32 = out_f32 != 0;
  L.status = static_cast<int*>(ws);
  L.part = reinterpret_cast<float*>(static_cast<char*>(ws) + kCacheStatusBytes);
  const bool bf16 = cache->kind == PISA_CACHE_BF16;
  if (score) {
    L.score = *score;
    const auto launch = score->cap > 0.f ? (bf16 ? launch_cache_cap_bf16 : launch_cache_cap_e2m1)
                        : score->slopes  ? (bf16 ? launch_cache_bias_bf16 : launch_cache_bias_e2m1)
                                         : (bf16 ? launch_cache_window_bf16 : launch_cache_window_e2m1);
    return cuda_code(launch(L, static_cast<cudaStream_t>(stream)));
  }
  const auto launch = bf16 ? launch_cache_attend_bf16 : launch_cache_attend_e2m1;
  return cuda_code(launch(L, static_cast<cudaStream_t>(stream)));
}

int pisa_cache_attention(const pisa_paged_cache* cache, const pisa_rows* q, int T, int Hq, const int32_t* lengths,
                         const int32_t* idx, int Ksel, void* out, int out_f32, void* ws, size_t ws_bytes,
                         void* stream) {
  return cache_attention(cache, q, T, Hq, lengths, idx, Ksel, nullptr, out, out_f32, ws, ws_bytes, stream);
}

int pisa_cache_attention_scored(const pisa_paged_cache* cache, const pisa_rows* q, int T, int Hq,
                                const int32_t* lengths, const int32_t* idx, int Ksel, float cap, const float* slopes,
                                int window, void* out, int out_f32, void* ws, size_t ws_bytes, void* stream) {
  ScoreDev d;
  const int st = check_score(cap, slopes, window, d);
  if (st) return st;
  return cache_attention(cache, q, T, Hq, lengths, idx, Ksel, &d, out, out_f32, ws, ws_bytes, stream);
}

int pisa_cache_prompt_attention(const pisa_paged_cache* cache, const pisa_rows* q, int T, int Hq,
                                const int32_t* start, const int32_t* counts, const int32_t* first,
                                const int32_t* last, float cap, const float* slopes, int window, void* out, void* ws,
                                size_t ws_bytes, void* stream) {
  CachePromptLaunch L{};
  int st = check_cache(cache, L.cache);
  if (st) return st;
  if (T < 1 || Hq < 1 || !start || !out || !ws) return PISA_ERR_INVALID_ARG;
  if ((st = check_rows(q, false, L.q)) || (st = check_score(cap, slopes, window, L.score))) return st;
  if (!aligned(out, 16) || !aligned(ws, 256) || !aligned(start, 4) || !aligned(counts, 4) || !aligned(first, 4) ||
      !aligned(last, 4))
    return PISA_ERR_INVALID_ARG;
  if (!group_ok(Hq, cache->Hkv)) return PISA_ERR_UNSUPPORTED;
  // 32-bit numbers of rows and of row tiles
  if (T > (1 << 27) || (long long)cache->B * T * Hq >= (1LL << 30)) return PISA_ERR_UNSUPPORTED;
  if (ws_bytes < pisa_cache_workspace_bytes()) return PISA_ERR_WORKSPACE_TOO_SMALL;
  L.T = T;
  L.Hq = Hq;
  L.G = Hq / cache->Hkv;
  L.start = start;
  L.counts = counts;
  L.first = first;
  L.last = last;
  L.out = static_cast<__nv_bfloat16*>(out);
  L.status = static_cast<int*>(ws);
  L.plan.piece = reinterpret_cast<PromptPiece*>(static_cast<char*>(ws) + kCacheStatusBytes);
  L.plan.cut = reinterpret_cast<int2*>(L.plan.piece + kPromptUnits + kPromptRuns);
  L.plan.tiles = reinterpret_cast<int32_t*>(L.plan.cut + kPromptRuns);
  L.part = reinterpret_cast<float*>(L.plan.tiles + kPromptUnits);
  return cuda_code(launch_cache_prompt(L, static_cast<cudaStream_t>(stream)));
}

size_t pisa_pool_workspace_bytes(int n_pages, int B) {
  if (n_pages < 1 || n_pages > (1 << 30) || B < 1 || B > 65535) return 0;
  return (kCacheStatusBytes + 4 * (64 + 3 * (size_t)n_pages + 3 * (size_t)B) + 255) / 256 * 256;
}

int pisa_cache_fork(const pisa_page_pool* pool, const int32_t* parents, int32_t* lengths, void* ws, void* stream) {
  PoolForkLaunch L{};
  const int st = check_pool(pool, L.pool);
  if (st) return st;
  if (!parents || !lengths || !aligned(parents, 4) || !aligned(lengths, 4) || !aligned(ws, 4))
    return PISA_ERR_INVALID_ARG;
  if (pool->B > kForkMaxB) return PISA_ERR_UNSUPPORTED;
  if (overlap(parents, pool->B, lengths, pool->B) || in_pool(L.pool, lengths, pool->B)) return PISA_ERR_INVALID_ARG;
  L.parents = parents;
  L.lengths = lengths;
  L.status = static_cast<int*>(ws);
  return cuda_code(launch_pool_fork(L, static_cast<cudaStream_t>(stream)));
}

int pisa_cache_reserve(const pisa_page_pool* pool, const int32_t* lengths, int T, const int32_t* counts,
                       int32_t* granted, void* ws, size_t ws_bytes, void* stream) {
  PoolReserveLaunch L{};
  const int st = check_pool(pool, L.pool);
  if (st) return st;
  if (!lengths || T < 1 || !granted || !ws) return PISA_ERR_INVALID_ARG;
  if (!aligned(lengths, 4) || !aligned(counts, 4) || !aligned(granted, 4) || !aligned(ws, 256))
    return PISA_ERR_INVALID_ARG;
  // (lengths and counts are read again when some grants are written; a grant in its count's place is that count, or is
  // not read again)
  if (overlap(granted, pool->B, lengths, pool->B) ||
      (granted != counts && overlap(granted, pool->B, counts, pool->B)) ||
      in_pool(L.pool, granted, pool->B))
    return PISA_ERR_INVALID_ARG;
  if (ws_bytes < pisa_pool_workspace_bytes(pool->n_pages, pool->B)) return PISA_ERR_WORKSPACE_TOO_SMALL;
  L.ws = pool_scratch(L.pool, ws);
  L.lengths = lengths;
  L.counts = counts;
  L.granted = granted;
  L.T = T;
  L.status = static_cast<int*>(ws);
  return cuda_code(launch_pool_reserve(L, static_cast<cudaStream_t>(stream)));
}

int pisa_cache_compact(const pisa_page_pool* pool, int32_t* used, void* ws, size_t ws_bytes, void* stream) {
  PoolCompactLaunch L{};
  const int st = check_pool(pool, L.pool);
  if (st) return st;
  if (!used || !aligned(used, 4) || !ws || !aligned(ws, 256) || in_pool(L.pool, used, 1)) return PISA_ERR_INVALID_ARG;
  if (ws_bytes < pisa_pool_workspace_bytes(pool->n_pages, pool->B)) return PISA_ERR_WORKSPACE_TOO_SMALL;
  L.ws = pool_scratch(L.pool, ws);
  L.used = used;
  return cuda_code(launch_pool_compact(L, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
