// Host-side checks of the paged-cache entry points' arguments (paged_api.cu, prompt_api.cu).
#pragma once

#include <cuda_runtime.h>

#include "api_checks.h"

namespace ditattn {
namespace api {

constexpr long long kMaxSpan = 1LL << 60;  // elements a view may reach, far inside 64-bit bytes
constexpr int kMaxTokens = 1 << 30;        // of a step: token indexes and what is added to them stay in 32 bits

// Sizes of the page pool and of a request's table row.
inline dit_status check_pages(int page_size, int n_pages, int max_pages) {
  if (page_size < 1 || n_pages < 1 || max_pages < 1) return DIT_ERR_INVALID_ARG;
  if (page_size % 16 != 0 || page_size > 1024) return DIT_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page_size > INT_MAX) return DIT_ERR_INVALID_ARG;
  return DIT_OK;
}

inline long long table_bytes(int B, int max_pages, long long stride) {
  return ((B - 1) * stride + max_pages) * 4;
}

inline bool valid_table(const int* table, long long stride, int B, int max_pages) {
  if (!table || !aligned(table, 4)) return false;
  return B == 1 || (stride >= max_pages && stride <= kMaxSpan / B);
}

// The strides of a paged cache [n_pages, H, page_size, D]: the given ones (a size-1 dimension's
// addresses nothing: any valid value will do) or contiguous.
inline dit_strides cache_strides(const dit_strides* s, int n_pages, int H, int page_size, int D) {
  dit_strides x = s ? *s : contiguous(H, page_size, D);
  if (n_pages == 1) x.b = D;
  if (H == 1) x.h = D;
  return x;
}

inline bool valid_cache(const void* p, const dit_strides& s, int n_pages, int H) {
  return p && aligned(p, 16) && valid_strides(s) && s.b <= kMaxSpan / n_pages && s.h <= kMaxSpan / H;
}

inline Range cache_range(const void* p, const dit_strides& s, int n_pages, int H, int page_size, int D) {
  return span(p, view_span(s, n_pages, H, page_size, D, 2));
}

// True if the two caches share no element: apart, or of equal strides and interleaved (pages, rows or
// heads of K and V in turn in one allocation), which the pair as one view with the distance between
// them as a further dimension shows.
inline bool caches_apart(const void* k, const dit_strides& ks, const void* v, const dit_strides& vs, int n_pages,
                  int H, int page_size, int D) {
  if (!overlap(cache_range(k, ks, n_pages, H, page_size, D), cache_range(v, vs, n_pages, H, page_size, D)))
    return true;
  if (ks.b != vs.b || ks.h != vs.h || ks.n != vs.n) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(k), b = reinterpret_cast<uintptr_t>(v);
  return no_self_overlap(ks, n_pages, H, page_size, D, static_cast<long long>((a > b ? a - b : b - a) / 2), 2);
}

// A [B, H, D] query view: its strides (b, h) in the manner of cache_strides.
inline dit_strides query_strides(const dit_strides* s, int B, int H, int D) {
  dit_strides x = s ? *s : dit_strides{static_cast<long long>(H) * D, D, D};
  x.n = D;
  if (B == 1) x.b = D;
  if (H == 1) x.h = D;
  return x;
}

inline bool valid_query(const void* q, const dit_strides& s, int B, int H) {
  return q && aligned(q, 16) && valid_strides(s) && s.b <= kMaxSpan / B && s.h <= kMaxSpan / H;
}

inline dit_status check_heads(int B, int H_q, int H_kv, int D) {
  if (H_kv < 1) return DIT_ERR_INVALID_ARG;
  const dit_status s = check_dims(B, H_q, 1, D);
  if (s != DIT_OK) return s;
  return H_q % H_kv == 0 ? DIT_OK : DIT_ERR_INVALID_ARG;
}

inline dit_status done(cudaError_t e) { return e == cudaSuccess ? DIT_OK : DIT_ERR_CUDA; }

}  // namespace api
}  // namespace ditattn
