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

struct RopeLaunch {  // queries, keys (heads 0: none)
  const void* in[2];
  void* out[2];
  Strides is[2], os[2];
  const void* weight[2];  // may be null
  int heads[2];
  bool weight_f32, norm, interleaved;
  float eps, rot_scale;
  const int* positions;  // or cu_new, start_lens
  long long pos_b, pos_axis;
  const int* cu_new;
  const int* start_lens;
  int requests;
  const float* freqs;
  int pairs, axes;  // 0 pairs: no rotation
  int axis_pairs[4];
  int batch, n, d;
};
cudaError_t launch_qk_norm_rope(const RopeLaunch& a, cudaStream_t st);

struct PrefillLaunch {
  const void* q;
  long long q_n, q_h;  // token and head strides (elements)
  const void* k_cache;
  const void* v_cache;
  Strides ks, vs;
  const int* table;
  long long table_stride;
  const int* seq_lens;
  const int* cu_new;
  const int* start_lens;  // may be null
  void* out;
  float* lse;  // may be null
  bool out_f32, causal;
  int tokens, batch, h_q, h_kv, d, page_size, n_pages, max_pages;
  float scale;
  void* workspace;
  int* status;
};
cudaError_t launch_paged_prefill(const PrefillLaunch& a, cudaStream_t st);
// Workspace bytes on the current device; `keys`: the most that a request can hold.
size_t paged_prefill_workspace(int d, long long keys);

struct MassLaunch {
  const void* q;
  long long q_n, q_h;
  const float* lse;
  const void* k_cache;
  Strides ks;
  const int* table;
  long long table_stride;
  const int* seq_lens;
  const int* cu_new;      // null: one token a request
  const int* start_lens;  // may be null
  const float* mass;
  float* mass_out;
  int tokens, batch, h_q, h_kv, d, page_size, n_pages, max_pages, window;
  float scale;
  int* status;
};
cudaError_t launch_paged_mass(const MassLaunch& a, cudaStream_t st);

struct EvictLaunch {
  const float* mass;
  const int* table;
  long long table_stride;
  int* table_out;
  long long out_stride;
  const int* seq_lens;
  int* lens_out;
  int* stack;
  const int* n_free;
  int* n_free_out;
  int batch, h_kv, page_size, n_pages, max_pages, capacity, keep, recent;
  void* workspace;
};
constexpr int kEvictMaxBatch = 8192;
cudaError_t launch_paged_evict(const EvictLaunch& a, cudaStream_t st);
size_t paged_evict_workspace(int batch, int max_pages);

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
