// Internal launch interface between the paged-cache entry points (paged_api.cu) and their
// kernels.  Arguments arrive here already validated.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>

#include "launch.h"

namespace ditattn {

// Pages of `rows` tokens (0 <= rows < 2^31: the sum may pass 2^31).
__host__ __device__ inline int pages_of(int rows, int page_size) {
  return static_cast<int>((static_cast<unsigned>(rows) + page_size - 1) / page_size);
}

struct PlanLaunch {
  const int* new_lens;
  const int* seq_lens;
  int* table;
  long long table_stride;
  const int* free_pages;
  const int* n_free;
  int* seq_lens_out;
  int* n_free_out;
  int* cu_new;
  long long* slots;
  int batch, max_pages, page_size, n_pages, pool_capacity, max_tokens;
};
constexpr int kPlanMaxBatch = 8192;
cudaError_t launch_paged_plan(const PlanLaunch& a, cudaStream_t st);

struct WriteLaunch {
  const void* k_new;
  const void* v_new;
  long long kn_n, kn_h, vn_n, vn_h;  // token and head strides (elements) of the new rows
  const long long* slots;
  void* k_cache;
  void* v_cache;
  Strides ks, vs;  // page, head, row strides (elements)
  void* summary;   // [n_pages, heads, 2, d] or null
  int tokens, heads, d, page_size, n_pages;
};
cudaError_t launch_paged_write(const WriteLaunch& a, cudaStream_t st);

struct PagedAttnLaunch {
  const void* q;
  long long q_b, q_h;  // request and head strides (elements)
  const void* k_cache;
  const void* v_cache;
  Strides ks, vs;
  const int* table;
  long long table_stride;
  const int* seq_lens;
  const int* selected;  // [batch, h_kv, n_selected] or null
  int n_selected;
  void* out;
  float* lse;  // may be null
  bool out_f32;
  int batch, h_q, h_kv, d, page_size, n_pages, max_pages;
  float scale;
  void* workspace;
  int* status;  // device status word
};
cudaError_t launch_paged_attn(const PagedAttnLaunch& a, cudaStream_t st);
// Workspace bytes on the current device; `keys`: the most that a request can attend to.
size_t paged_attn_workspace(int batch, int h_q, int h_kv, int d, long long keys);

struct SelectLaunch {
  const void* q;
  long long q_b, q_h;
  const void* summary;  // [n_pages, h_kv, 2, d]
  const int* table;
  long long table_stride;
  const int* seq_lens;
  int* selected;
  int batch, h_q, h_kv, d, page_size, n_pages, max_pages, top_k;
  void* workspace;
};
cudaError_t launch_paged_select(const SelectLaunch& a, cudaStream_t st);
size_t paged_select_workspace(int batch, int h_kv, int max_pages);

}  // namespace ditattn
