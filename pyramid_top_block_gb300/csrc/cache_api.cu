// cache_api.cu -- the C ABI of the paged KV cache (include/pisa.h): argument checks and
// launches.  No allocation, no exceptions, one stream.
#include "cache.cuh"

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

int cuda_code(cudaError_t e) { return e == cudaSuccess ? PISA_OK : PISA_ERR_CUDA; }

}  // namespace

extern "C" {

size_t pisa_cache_page_bytes(int page_size, int Hkv, int kind) {
  if (page_shift_of(page_size) < 0 || Hkv < 1 || Hkv > 32) return 0;
  if (kind != PISA_CACHE_BF16 && kind != PISA_CACHE_E2M1) return 0;
  return (size_t)page_size * Hkv * (kind == PISA_CACHE_BF16 ? kRowBf16 : kRowE2m1);
}

size_t pisa_cache_workspace_bytes(void) { return kCacheStatusBytes + cache_part_bytes(); }

int pisa_cache_append(const pisa_paged_cache* cache, int T, const pisa_rows* q, int Hq, const pisa_rows* k,
                      const pisa_rows* v, const int32_t* start, const int32_t* counts, const float* rotary,
                      int64_t n_rot, int rot, int interleaved, const pisa_rows* q_out, const pisa_rows* k_out,
                      void* ws, void* stream) {
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
  L.status = static_cast<int*>(ws);
  return cuda_code(launch_cache_append(L, static_cast<cudaStream_t>(stream)));
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

int pisa_cache_attention(const pisa_paged_cache* cache, const pisa_rows* q, int T, int Hq, const int32_t* lengths,
                         const int32_t* idx, int Ksel, void* out, int out_f32, void* ws, size_t ws_bytes,
                         void* stream) {
  CacheAttendLaunch L{};
  int st = check_cache(cache, L.cache);
  if (st) return st;
  if (T < 1 || Hq < 1 || !lengths || !out || !ws) return PISA_ERR_INVALID_ARG;
  if ((st = check_rows(q, false, L.q))) return st;
  if (!aligned(out, 16) || !aligned(ws, 256) || !aligned(lengths, 4) || !aligned(idx, 4)) return PISA_ERR_INVALID_ARG;
  if (T > kCacheMaxT || !group_ok(Hq, cache->Hkv)) return PISA_ERR_UNSUPPORTED;
  if (idx && (Ksel < 1 || Ksel > kCacheMaxSel)) return PISA_ERR_UNSUPPORTED;
  if ((long long)cache->B * T * cache->Hkv >= (1LL << 24)) return PISA_ERR_UNSUPPORTED;
  if (ws_bytes < pisa_cache_workspace_bytes()) return PISA_ERR_WORKSPACE_TOO_SMALL;
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
  const auto launch = cache->kind == PISA_CACHE_BF16 ? launch_cache_attend_bf16 : launch_cache_attend_e2m1;
  return cuda_code(launch(L, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
