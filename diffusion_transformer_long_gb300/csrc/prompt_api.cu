// C entry points of prompts over the paged key/value cache (declared in include/ditattn.h): argument
// validation and dispatch.  Validation makes no CUDA call but the workspace sizes' look at the device's
// SM count.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/ditattn.h"
#include "paged_checks.h"
#include "paged_launch.h"

using namespace ditattn::api;

namespace {

// A [T, H, D] view of a step's tokens: its strides (n, h) in the manner of cache_strides.
dit_strides token_strides(const dit_strides* s, int T, int H, int D) {
  dit_strides x = s ? *s : dit_strides{D, D, static_cast<long long>(H) * D};
  x.b = D;
  if (H == 1) x.h = D;
  if (T == 1) x.n = D;
  return x;
}

bool valid_tokens(const void* p, const dit_strides& s, int T, int H) {
  return p && aligned(p, 16) && valid_strides(s) && s.n <= kMaxSpan / T && s.h <= kMaxSpan / H;
}

}  // namespace

extern "C" {

size_t dit_paged_prefill_workspace_bytes(int D, int page_size, int max_pages) {
  if (D < 1 || page_size < 1 || max_pages < 1) return 0;
  return ditattn::paged_prefill_workspace(D, static_cast<long long>(max_pages) * page_size);
}

dit_status dit_paged_prefill_fwd(const void* q, const dit_strides* q_strides, const void* k_cache,
                                 const dit_strides* k_strides, const void* v_cache,
                                 const dit_strides* v_strides, const int* block_table,
                                 long long table_stride, const int* seq_lens, const int* cu_new,
                                 const int* start_lens, void* out, float* lse, int T, int B, int H_q,
                                 int H_kv, int D, int page_size, int n_pages, int max_pages, int causal,
                                 float scale, dit_dtype out_dtype, void* workspace,
                                 size_t workspace_bytes, dit_stream stream) {
  if (T < 1 || T > kMaxTokens || B < 1 || B == INT_MAX) return DIT_ERR_INVALID_ARG;
  dit_status s = check_heads(T, H_q, H_kv, D);
  if (s != DIT_OK) return s;
  s = check_pages(page_size, n_pages, max_pages);
  if (s != DIT_OK) return s;
  if (H_q / H_kv > 128) return DIT_ERR_UNSUPPORTED;  // a tile's rows
  const dit_strides qs = token_strides(q_strides, T, H_q, D);
  const dit_strides ks = cache_strides(k_strides, n_pages, H_kv, page_size, D);
  const dit_strides vs = cache_strides(v_strides, n_pages, H_kv, page_size, D);
  if (!valid_tokens(q, qs, T, H_q) || qs.h >= (1LL << 39) / (H_q / H_kv) ||
      !valid_cache(k_cache, ks, n_pages, H_kv) || !valid_cache(v_cache, vs, n_pages, H_kv))
    return DIT_ERR_INVALID_ARG;
  if (!valid_table(block_table, table_stride, B, max_pages) || !seq_lens || !aligned(seq_lens, 4) || !cu_new ||
      !aligned(cu_new, 4) || !aligned(start_lens, 4) || !out || !aligned(out, 16) || !aligned(lse, 4))
    return DIT_ERR_INVALID_ARG;
  if ((causal != 0 && causal != 1) || !(scale > 0.f) || !std::isfinite(scale * 1.4426950408889634f) ||  // (base 2)
      !valid_dtype(out_dtype))
    return DIT_ERR_INVALID_ARG;
  const size_t need = dit_paged_prefill_workspace_bytes(D, page_size, max_pages);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return DIT_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(T) * H_q;
  const Range outs[] = {span(out, rows * D * dtype_bytes(out_dtype)), span(lse, lse ? rows * 4 : 0),
                        span(workspace, static_cast<long long>(need))};
  const Range ins[] = {span(q, view_span(qs, 1, H_q, T, D, 2)),
                       cache_range(k_cache, ks, n_pages, H_kv, page_size, D),
                       cache_range(v_cache, vs, n_pages, H_kv, page_size, D),
                       span(block_table, table_bytes(B, max_pages, table_stride)),
                       span(seq_lens, 4LL * B), span(cu_new, 4LL * (B + 1LL)),
                       span(start_lens, start_lens ? 4LL * B : 0)};
  for (int i = 0; i < 3; ++i) {
    for (int j = i + 1; j < 3; ++j)
      if (overlap(outs[i], outs[j])) return DIT_ERR_INVALID_ARG;
    for (const Range& in : ins)
      if (overlap(outs[i], in)) return DIT_ERR_INVALID_ARG;
  }
  ditattn::PrefillLaunch a;
  a.q = q;
  a.q_n = qs.n;
  a.q_h = qs.h;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.ks = {ks.b, ks.h, ks.n};
  a.vs = {vs.b, vs.h, vs.n};
  a.table = block_table;
  a.table_stride = table_stride;
  a.seq_lens = seq_lens;
  a.cu_new = cu_new;
  a.start_lens = start_lens;
  a.out = out;
  a.lse = lse;
  a.out_f32 = out_dtype == DIT_F32;
  a.causal = causal != 0;
  a.tokens = T;
  a.batch = B;
  a.h_q = H_q;
  a.h_kv = H_kv;
  a.d = D;
  a.page_size = page_size;
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  a.scale = scale;
  a.workspace = workspace;
  a.status = ditattn::status_word();
  if (!a.status) return DIT_ERR_CUDA;
  return done(ditattn::launch_paged_prefill(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
