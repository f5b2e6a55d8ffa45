// Tensor maps of the paged operators' tiles (paged_prefill.cu, paged_mass.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "attn_host.cuh"
#include "launch.h"

namespace ditattn {
namespace maps {

// A map of bf16 elements: extents, strides (elements) of all dimensions but the first, box; 128-byte swizzle.
template <int N>
bool encode(CUtensorMap* m, const void* base, const long long (&dims)[N], const long long (&strides)[N - 1],
            const int (&boxes)[N]) {
  EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t d[N], st[N - 1];
  cuuint32_t box[N], elem[N];
  for (int i = 0; i < N; ++i) {
    d[i] = static_cast<cuuint64_t>(dims[i]);
    box[i] = static_cast<cuuint32_t>(boxes[i]);
    elem[i] = 1;
    if (i) st[i - 1] = static_cast<cuuint64_t>(strides[i - 1]) * 2;
  }
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, N, const_cast<void*>(base), d, st, box, elem,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of a page that one copy brings to a tile of 128: the largest power of two that divides the page size.
inline int box_rows(int page_size) {
  int rows = 16;
  while (rows < 128 && page_size % (2 * rows) == 0) rows *= 2;
  return rows;
}

// A paged cache's map of copies of `rows` rows of 64 channels: (D, row, head, page).
inline bool encode_rows(CUtensorMap* m, const void* base, const Strides& s, int d, int page_size, int heads, int n_pages,
                        int rows) {
  return encode<4>(m, base, {d, page_size, heads, n_pages}, {s.n_, s.h_, s.b_}, {64, rows, 1, 1});
}

// A step's queries [T, H_q, D], boxes of the `group` heads of a key/value head of `tokens` tokens: (D, head of the
// group, token, key/value head).
inline bool encode_queries(CUtensorMap* m, const void* q, long long q_n, long long q_h, int d, int group, int n, int h_kv,
                           int tokens) {
  return encode<4>(m, q, {d, group, n, h_kv}, {q_h, q_n, q_h * group}, {64, group, tokens, 1});
}

}  // namespace maps
}  // namespace ditattn
