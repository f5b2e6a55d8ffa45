// Host-side argument checks shared by the C entry points (ditattn_api.cu, paged_api.cu).
#pragma once

#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <utility>

#include "../../include/ditattn.h"

namespace ditattn {
namespace api {

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};
inline Range span(const void* p, long long bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + static_cast<uintptr_t>(bytes)};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

inline bool valid_dtype(dit_dtype t) { return t == DIT_F32 || t == DIT_BF16; }
inline int dtype_bytes(dit_dtype t) { return t == DIT_F32 ? 4 : 2; }

inline dit_status check_dims(long long B, long long H, long long N, int D) {
  if (B < 1 || H < 1 || N < 1 || D < 1) return DIT_ERR_INVALID_ARG;
  if (B * H > INT_MAX || N > INT_MAX) return DIT_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return DIT_ERR_UNSUPPORTED;
  return DIT_OK;
}

// Bytes spanned by a strided [B, H, N, D] view (from its base to one past its last element).
inline long long view_span(const dit_strides& s, long long B, long long H, long long N, long long D,
                           int esize) {
  return ((B - 1) * s.b + (H - 1) * s.h + (N - 1) * s.n + D) * esize;
}

inline dit_strides contiguous(long long H, long long N, long long D) { return {H * N * D, N * D, D}; }

// A strided view usable by the kernels: strides positive multiples of 8 elements (16-byte
// TMA strides) below 2^39, and the view must fit 64-bit byte offsets comfortably.
inline bool valid_strides(const dit_strides& s) {
  for (long long x : {s.b, s.h, s.n})
    if (x < 8 || x % 8 != 0 || x >= (1LL << 39)) return false;
  return true;
}

// True if no two elements of the view, or of `copies` of it `distance` elements apart, share an
// address: sorted by stride, every stride must clear the span of the dimensions below it.
inline bool no_self_overlap(const dit_strides& s, long long B, long long H, long long N,
                            long long D, long long distance = 0, long long copies = 1) {
  struct Dim {
    long long stride, extent;
  } d[4] = {{s.n, N}, {s.h, H}, {s.b, B}, {distance, copies}};
  for (int i = 0; i < 4; ++i)  // sort by stride
    for (int j = i + 1; j < 4; ++j)
      if (d[j].stride < d[i].stride) std::swap(d[i], d[j]);
  long long span = D;
  for (const Dim& x : d) {
    if (x.extent <= 1) continue;
    if (x.stride < span) return false;
    span = x.stride * (x.extent - 1) + span;
  }
  return true;
}

}  // namespace api
}  // namespace ditattn
