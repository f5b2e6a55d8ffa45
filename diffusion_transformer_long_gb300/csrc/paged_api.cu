// C entry points of the paged key/value cache (declared in include/ditattn.h): argument
// validation and dispatch.  Validation makes no CUDA call but the workspace sizes' look at the device's
// SM count.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/ditattn.h"
#include "api_checks.h"
#include "paged_launch.h"

namespace {

using namespace ditattn::api;

constexpr long long kMaxSpan = 1LL << 60;  // elements a view may reach, far inside 64-bit bytes
constexpr int kMaxTokens = 1 << 30;        // of a step: token indexes and what is added to them stay in 32 bits

// Sizes of the page pool and of a request's table row.
dit_status check_pages(int page_size, int n_pages, int max_pages) {
  if (page_size < 1 || n_pages < 1 || max_pages < 1) return DIT_ERR_INVALID_ARG;
  if (page_size % 16 != 0 || page_size > 1024) return DIT_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page_size > INT_MAX) return DIT_ERR_INVALID_ARG;
  return DIT_OK;
}

long long table_bytes(int B, int max_pages, long long stride) {
  return ((B - 1) * stride + max_pages) * 4;
}

bool valid_table(const int* table, long long stride, int B, int max_pages) {
  if (!table || !aligned(table, 4)) return false;
  return B == 1 || (stride >= max_pages && stride <= kMaxSpan / B);
}

// The strides of a paged cache [n_pages, H, page_size, D]: the given ones (a size-1 dimension's
// addresses nothing: any valid value will do) or contiguous.
dit_strides cache_strides(const dit_strides* s, int n_pages, int H, int page_size, int D) {
  dit_strides x = s ? *s : contiguous(H, page_size, D);
  if (n_pages == 1) x.b = D;
  if (H == 1) x.h = D;
  return x;
}

bool valid_cache(const void* p, const dit_strides& s, int n_pages, int H) {
  return p && aligned(p, 16) && valid_strides(s) && s.b <= kMaxSpan / n_pages && s.h <= kMaxSpan / H;
}

Range cache_range(const void* p, const dit_strides& s, int n_pages, int H, int page_size, int D) {
  return span(p, view_span(s, n_pages, H, page_size, D, 2));
}

// True if the two caches share no element: apart, or of equal strides and interleaved (pages, rows or
// heads of K and V in turn in one allocation), which the pair as one view with the distance between
// them as a further dimension shows.
bool caches_apart(const void* k, const dit_strides& ks, const void* v, const dit_strides& vs, int n_pages,
                  int H, int page_size, int D) {
  if (!overlap(cache_range(k, ks, n_pages, H, page_size, D), cache_range(v, vs, n_pages, H, page_size, D)))
    return true;
  if (ks.b != vs.b || ks.h != vs.h || ks.n != vs.n) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(k), b = reinterpret_cast<uintptr_t>(v);
  return no_self_overlap(ks, n_pages, H, page_size, D, static_cast<long long>((a > b ? a - b : b - a) / 2), 2);
}

// A [B, H, D] query view: its strides (b, h) in the manner of cache_strides.
dit_strides query_strides(const dit_strides* s, int B, int H, int D) {
  dit_strides x = s ? *s : dit_strides{static_cast<long long>(H) * D, D, D};
  x.n = D;
  if (B == 1) x.b = D;
  if (H == 1) x.h = D;
  return x;
}

bool valid_query(const void* q, const dit_strides& s, int B, int H) {
  return q && aligned(q, 16) && valid_strides(s) && s.b <= kMaxSpan / B && s.h <= kMaxSpan / H;
}

dit_status check_heads(int B, int H_q, int H_kv, int D) {
  if (H_kv < 1) return DIT_ERR_INVALID_ARG;
  const dit_status s = check_dims(B, H_q, 1, D);
  if (s != DIT_OK) return s;
  return H_q % H_kv == 0 ? DIT_OK : DIT_ERR_INVALID_ARG;
}

dit_status done(cudaError_t e) { return e == cudaSuccess ? DIT_OK : DIT_ERR_CUDA; }

}  // namespace

extern "C" {

dit_status dit_paged_plan(const int* new_lens, const int* seq_lens, int* block_table,
                          long long table_stride, const int* free_pages, const int* n_free,
                          int* seq_lens_out, int* n_free_out, int* cu_new, long long* slots, int B,
                          int max_pages, int page_size, int n_pages, int pool_capacity,
                          int max_tokens, dit_stream stream) {
  if (B < 1 || max_tokens < 1 || max_tokens > kMaxTokens || pool_capacity < 0)
    return DIT_ERR_INVALID_ARG;
  const dit_status s = check_pages(page_size, n_pages, max_pages);
  if (s != DIT_OK) return s;
  if (B > ditattn::kPlanMaxBatch) return DIT_ERR_UNSUPPORTED;
  if (!new_lens || !seq_lens || !n_free || !seq_lens_out || !n_free_out || !cu_new || !slots ||
      (!free_pages && pool_capacity > 0))
    return DIT_ERR_INVALID_ARG;
  for (const void* p : std::initializer_list<const void*>{new_lens, seq_lens, free_pages, n_free,
                                                          seq_lens_out, n_free_out, cu_new})
    if (!aligned(p, 4)) return DIT_ERR_INVALID_ARG;
  if (!aligned(slots, 8) || !valid_table(block_table, table_stride, B, max_pages))
    return DIT_ERR_INVALID_ARG;
  const Range outs[] = {span(block_table, table_bytes(B, max_pages, table_stride)),
                        span(seq_lens_out, 4LL * B), span(n_free_out, 4), span(cu_new, 4LL * (B + 1)),
                        span(slots, 8LL * max_tokens)};
  const Range ins[] = {span(new_lens, 4LL * B), span(free_pages, 4LL * pool_capacity),
                       span(seq_lens, 4LL * B), span(n_free, 4)};
  for (int i = 0; i < 5; ++i) {
    for (int j = i + 1; j < 5; ++j)
      if (overlap(outs[i], outs[j])) return DIT_ERR_INVALID_ARG;
    for (int j = 0; j < 4; ++j) {
      const bool in_place = (i == 1 && j == 2 && seq_lens_out == seq_lens) ||
                            (i == 2 && j == 3 && n_free_out == n_free);
      if (!in_place && overlap(outs[i], ins[j])) return DIT_ERR_INVALID_ARG;
    }
  }
  ditattn::PlanLaunch a{new_lens,  seq_lens, block_table, table_stride, free_pages, n_free,
                        seq_lens_out, n_free_out, cu_new,  slots,        B,          max_pages,
                        page_size, n_pages,  pool_capacity, max_tokens};
  return done(ditattn::launch_paged_plan(a, static_cast<cudaStream_t>(stream)));
}

dit_status dit_paged_kv_write(const void* k_new, const dit_strides* k_new_strides,
                              const void* v_new, const dit_strides* v_new_strides,
                              const long long* slots, void* k_cache,
                              const dit_strides* k_strides, void* v_cache,
                              const dit_strides* v_strides, void* summary, int T, int H, int D,
                              int page_size, int n_pages, dit_stream stream) {
  dit_status s = check_dims(1, H, T, D);
  if (s != DIT_OK) return s;
  if (T > kMaxTokens) return DIT_ERR_INVALID_ARG;
  s = check_pages(page_size, n_pages, 1);
  if (s != DIT_OK) return s;
  auto rows = [&](const dit_strides* p) {
    dit_strides x = p ? *p : dit_strides{D, D, static_cast<long long>(H) * D};
    x.b = D;
    if (H == 1) x.h = D;
    if (T == 1) x.n = D;
    return x;
  };
  const dit_strides kn = rows(k_new_strides), vn = rows(v_new_strides);
  const dit_strides ks = cache_strides(k_strides, n_pages, H, page_size, D);
  const dit_strides vs = cache_strides(v_strides, n_pages, H, page_size, D);
  if (!k_new || !v_new || !aligned(k_new, 16) || !aligned(v_new, 16) || !valid_strides(kn) ||
      !valid_strides(vn) || kn.n > kMaxSpan / T || vn.n > kMaxSpan / T || kn.h > kMaxSpan / H ||
      vn.h > kMaxSpan / H)
    return DIT_ERR_INVALID_ARG;
  if (!slots || !aligned(slots, 8) || !valid_cache(k_cache, ks, n_pages, H) ||
      !valid_cache(v_cache, vs, n_pages, H) || !aligned(summary, 16) ||
      H > kMaxSpan / (static_cast<long long>(n_pages) * D))
    return DIT_ERR_INVALID_ARG;
  if (!no_self_overlap(ks, n_pages, H, page_size, D) ||
      !no_self_overlap(vs, n_pages, H, page_size, D))
    return DIT_ERR_INVALID_ARG;
  const Range outs[] = {cache_range(k_cache, ks, n_pages, H, page_size, D),
                        cache_range(v_cache, vs, n_pages, H, page_size, D),
                        span(summary, summary ? 4LL * n_pages * H * D : 0)};
  const Range ins[] = {span(k_new, view_span(kn, 1, H, T, D, 2)),
                       span(v_new, view_span(vn, 1, H, T, D, 2)), span(slots, 8LL * T)};
  const int n_out = summary ? 3 : 2;
  if (!caches_apart(k_cache, ks, v_cache, vs, n_pages, H, page_size, D)) return DIT_ERR_INVALID_ARG;
  for (int i = 0; i < n_out; ++i) {
    if (i < 2 && summary && overlap(outs[i], outs[2])) return DIT_ERR_INVALID_ARG;
    for (const Range& in : ins)
      if (overlap(outs[i], in)) return DIT_ERR_INVALID_ARG;
  }
  ditattn::WriteLaunch a;
  a.k_new = k_new;
  a.v_new = v_new;
  a.kn_n = kn.n;
  a.kn_h = kn.h;
  a.vn_n = vn.n;
  a.vn_h = vn.h;
  a.slots = slots;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.ks = {ks.b, ks.h, ks.n};
  a.vs = {vs.b, vs.h, vs.n};
  a.summary = summary;
  a.tokens = T;
  a.heads = H;
  a.d = D;
  a.page_size = page_size;
  a.n_pages = n_pages;
  return done(ditattn::launch_paged_write(a, static_cast<cudaStream_t>(stream)));
}

size_t dit_paged_attn_workspace_bytes(int B, int H_q, int H_kv, int D, int page_size, int pages) {
  if (B < 1 || H_kv < 1 || H_q < H_kv || D < 1 || page_size < 1 || pages < 1) return 0;
  return ditattn::paged_attn_workspace(B, H_q, H_kv, D, static_cast<long long>(pages) * page_size);
}

dit_status dit_paged_attn_fwd(const void* q, const dit_strides* q_strides, const void* k_cache,
                              const dit_strides* k_strides, const void* v_cache,
                              const dit_strides* v_strides, const int* block_table,
                              long long table_stride, const int* seq_lens, const int* selected,
                              int n_selected, void* out, float* lse, int B, int H_q, int H_kv,
                              int D, int page_size, int n_pages, int max_pages, float scale,
                              dit_dtype out_dtype, void* workspace, size_t workspace_bytes,
                              dit_stream stream) {
  dit_status s = check_heads(B, H_q, H_kv, D);
  if (s != DIT_OK) return s;
  s = check_pages(page_size, n_pages, max_pages);
  if (s != DIT_OK) return s;
  const dit_strides qs = query_strides(q_strides, B, H_q, D);
  const dit_strides ks = cache_strides(k_strides, n_pages, H_kv, page_size, D);
  const dit_strides vs = cache_strides(v_strides, n_pages, H_kv, page_size, D);
  if (!valid_query(q, qs, B, H_q) || !valid_cache(k_cache, ks, n_pages, H_kv) ||
      !valid_cache(v_cache, vs, n_pages, H_kv))
    return DIT_ERR_INVALID_ARG;
  if (!valid_table(block_table, table_stride, B, max_pages) || !seq_lens || !aligned(seq_lens, 4) ||
      !aligned(selected, 4) || !out || !aligned(out, 16) || !aligned(lse, 4))
    return DIT_ERR_INVALID_ARG;
  if (selected && (n_selected < 1 || n_selected > max_pages)) return DIT_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale * 1.4426950408889634f) || !valid_dtype(out_dtype))  // (used in base 2)
    return DIT_ERR_INVALID_ARG;
  const size_t need = dit_paged_attn_workspace_bytes(B, H_q, H_kv, D, page_size, selected ? n_selected : max_pages);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return DIT_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(B) * H_q;
  const Range outs[] = {span(out, rows * D * dtype_bytes(out_dtype)), span(lse, lse ? rows * 4 : 0),
                        span(workspace, static_cast<long long>(need))};
  const Range ins[] = {span(q, view_span(qs, B, H_q, 1, D, 2)),
                       cache_range(k_cache, ks, n_pages, H_kv, page_size, D),
                       cache_range(v_cache, vs, n_pages, H_kv, page_size, D),
                       span(block_table, table_bytes(B, max_pages, table_stride)),
                       span(seq_lens, 4LL * B),
                       span(selected, selected ? 4LL * B * H_kv * n_selected : 0)};
  for (int i = 0; i < 3; ++i) {
    for (int j = i + 1; j < 3; ++j)
      if (overlap(outs[i], outs[j])) return DIT_ERR_INVALID_ARG;
    for (const Range& in : ins)
      if (overlap(outs[i], in)) return DIT_ERR_INVALID_ARG;
  }
  ditattn::PagedAttnLaunch a;
  a.q = q;
  a.q_b = qs.b;
  a.q_h = qs.h;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.ks = {ks.b, ks.h, ks.n};
  a.vs = {vs.b, vs.h, vs.n};
  a.table = block_table;
  a.table_stride = table_stride;
  a.seq_lens = seq_lens;
  a.selected = selected;
  a.n_selected = selected ? n_selected : 0;
  a.out = out;
  a.lse = lse;
  a.out_f32 = out_dtype == DIT_F32;
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
  return done(ditattn::launch_paged_attn(a, static_cast<cudaStream_t>(stream)));
}

size_t dit_paged_select_workspace_bytes(int B, int H_kv, int max_pages) {
  if (B < 1 || H_kv < 1 || max_pages < 1) return 0;
  return ditattn::paged_select_workspace(B, H_kv, max_pages);
}

dit_status dit_paged_select(const void* q, const dit_strides* q_strides, const void* summary,
                            const int* block_table, long long table_stride, const int* seq_lens,
                            int* selected, int B, int H_q, int H_kv, int D, int page_size,
                            int n_pages, int max_pages, int top_k, void* workspace,
                            size_t workspace_bytes, dit_stream stream) {
  dit_status s = check_heads(B, H_q, H_kv, D);
  if (s != DIT_OK) return s;
  s = check_pages(page_size, n_pages, max_pages);
  if (s != DIT_OK) return s;
  const dit_strides qs = query_strides(q_strides, B, H_q, D);
  if (!valid_query(q, qs, B, H_q) || !summary || !aligned(summary, 16) ||
      H_kv > kMaxSpan / (static_cast<long long>(n_pages) * D))
    return DIT_ERR_INVALID_ARG;
  if (!valid_table(block_table, table_stride, B, max_pages) || !seq_lens || !aligned(seq_lens, 4) ||
      !selected || !aligned(selected, 4))
    return DIT_ERR_INVALID_ARG;
  if (top_k < 1 || top_k > max_pages) return DIT_ERR_INVALID_ARG;
  const size_t need = dit_paged_select_workspace_bytes(B, H_kv, max_pages);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return DIT_ERR_INVALID_ARG;
  const Range outs[] = {span(selected, 4LL * B * H_kv * top_k),
                        span(workspace, static_cast<long long>(need))};
  const Range ins[] = {span(q, view_span(qs, B, H_q, 1, D, 2)), span(summary, 4LL * n_pages * H_kv * D),
                       span(block_table, table_bytes(B, max_pages, table_stride)),
                       span(seq_lens, 4LL * B)};
  if (overlap(outs[0], outs[1])) return DIT_ERR_INVALID_ARG;
  for (const Range& out : outs)
    for (const Range& in : ins)
      if (overlap(out, in)) return DIT_ERR_INVALID_ARG;
  ditattn::SelectLaunch a{q,   qs.b, qs.h, summary,   block_table, table_stride, seq_lens, selected,
                          B,   H_q,  H_kv, D,         page_size,   n_pages,      max_pages, top_k,
                          workspace};
  return done(ditattn::launch_paged_select(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
