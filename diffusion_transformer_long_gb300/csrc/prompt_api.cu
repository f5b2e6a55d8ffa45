// C entry points of norms with rotary positions and of prompts over the paged key/value cache (declared in include/ditattn.h): argument
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

// Each block adds the requests' lengths up for itself, 32 at a time: 20 ms at this many.
constexpr int kMaxRequests = 1 << 20;

// Whether the kernels' 32-bit key indexes reach past a full table row's last tile.
bool room_counts(int page_size, int max_pages) { return static_cast<long long>(max_pages) * page_size <= 1 << 30; }

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

// A [B, H, N, D] view's strides; a size-1 dimension's addresses nothing.
dit_strides row_strides(const dit_strides* s, int B, int H, int N, int D) {
  dit_strides x = s ? *s : contiguous(H, N, D);
  if (B == 1) x.b = D;
  if (H == 1) x.h = D;
  if (N == 1) x.n = D;
  return x;
}

struct View {
  const void* p;
  dit_strides s;
  int H;
  bool valid(int B, int N) const {
    return p && aligned(p, 16) && valid_strides(s) && s.b <= kMaxSpan / B && s.h <= kMaxSpan / H && s.n <= kMaxSpan / N;
  }
  Range range(int B, int N, int D) const { return span(p, view_span(s, B, H, N, D, 2)); }
  bool same(const View& v) const {
    return p == v.p && H == v.H && s.b == v.s.b && s.h == v.s.h && s.n == v.s.n;
  }
};

// A view's dimensions of more than one element, the longest strides first, over runs of `run` elements.
struct Grid {
  struct {
    long long stride, extent;
  } dim[3];
  int dims = 0;
  long long run;
  void add(long long stride, long long extent) {
    if (extent <= 1) return;
    int i = dims++;
    for (; i > 0 && dim[i - 1].stride < stride; --i) dim[i] = dim[i - 1];
    dim[i] = {stride, extent};
  }
  // Elements from the first to behind the last of dimensions `from` on.
  long long span(int from) const {
    long long x = run;
    for (int i = from; i < dims; ++i) x += dim[i].stride * (dim[i].extent - 1);
    return x;
  }
};

constexpr int kMostSteps = 1 << 14;  // of telling two grids apart (0.1 ms)

// Whether a, from its dimension i on, and b, from its j on and `gap` elements further, share no element: where their
// spans meet, the longest stride's elements one by one (of both grids together if it is in both, so that only their
// difference counts), as far as they can meet.  Grids that nest, as the slices of one allocation do, are told apart in a
// few steps; what takes more than `steps` counts as shared.
bool grids_apart(const Grid& a, int i, const Grid& b, int j, long long gap, int& steps) {
  const long long sa = a.span(i), sb = b.span(j);
  if (gap >= sa || gap + sb <= 0) return true;
  if ((i == a.dims && j == b.dims) || --steps < 0) return false;
  const long long ta = i < a.dims ? a.dim[i].stride : 0, tb = j < b.dims ? b.dim[j].stride : 0, s = ta > tb ? ta : tb;
  // b's elements less a's: x strides apart.
  const long long lo = ta == s ? 1 - a.dim[i].extent : 0, hi = tb == s ? b.dim[j].extent - 1 : 0;
  i += ta == s;
  j += tb == s;
  const long long ra = a.span(i), rb = b.span(j);
  // The least x with gap + x s > -rb.
  const long long y = -rb - gap, least = (y >= 0 ? y / s : -((-y + s - 1) / s)) + 1;
  for (long long x = least > lo ? least : lo; x <= hi && gap + x * s < ra; ++x)
    if (!grids_apart(a, i, b, j, gap + x * s, steps)) return false;
  return true;
}

// True if the two views share no element, whichever way they interleave.
bool views_apart(const View& a, const View& b, int B, int N, int D) {
  if (!overlap(a.range(B, N, D), b.range(B, N, D))) return true;
  Grid g[2];
  for (int i = 0; i < 2; ++i) {
    const View& v = i ? b : a;
    g[i].run = D;
    g[i].add(v.s.b, B);
    g[i].add(v.s.h, v.H);
    g[i].add(v.s.n, N);
  }
  const long long gap = (static_cast<long long>(reinterpret_cast<uintptr_t>(b.p)) - static_cast<long long>(reinterpret_cast<uintptr_t>(a.p))) / 2;
  int steps = kMostSteps;
  return grids_apart(g[0], 0, g[1], 0, gap, steps);
}

// True if two tables of B rows of n ints share none.
bool rows_apart(const int* a, long long a_stride, const int* b, long long b_stride, int B, int n) {
  Grid g[2];
  for (int i = 0; i < 2; ++i) {
    g[i].run = n;
    g[i].add(i ? b_stride : a_stride, B);
  }
  int steps = kMostSteps;
  return grids_apart(g[0], 0, g[1], 0, b - a, steps);
}

}  // namespace

extern "C" {

dit_status dit_qk_norm_rope(const void* q, const dit_strides* q_strides, void* q_out,
                            const dit_strides* q_out_strides, int H_q, const void* k,
                            const dit_strides* k_strides, void* k_out, const dit_strides* k_out_strides,
                            int H_k, int norm, float eps, const void* q_weight, const void* k_weight,
                            dit_dtype weight_dtype, const float* freqs, const int* axis_pairs, int axes,
                            int interleaved, float rot_scale, const int* positions, long long pos_b,
                            long long pos_axis, const int* cu_new, const int* start_lens, int requests, int B,
                            int N, int D, dit_stream stream) {
  dit_status s = check_dims(B, H_q, N, D);
  if (s != DIT_OK) return s;
  if (H_k < 0 || (H_k > 0) != (k != nullptr) || (!k && (k_out || k_weight))) return DIT_ERR_INVALID_ARG;
  if (k && (s = check_dims(B, H_k, N, D)) != DIT_OK) return s;
  if (static_cast<long long>(B) * N > kMaxTokens) return DIT_ERR_INVALID_ARG;
  const int sides = k ? 2 : 1;
  const View in[2] = {{q, row_strides(q_strides, B, H_q, N, D), H_q}, {k, row_strides(k_strides, B, H_k, N, D), H_k}};
  const View out[2] = {{q_out, row_strides(q_out_strides, B, H_q, N, D), H_q},
                       {k_out, row_strides(k_out_strides, B, H_k, N, D), H_k}};
  const void* weight[2] = {q_weight, k_weight};
  if ((norm != 0 && norm != 1) || (!norm && (q_weight || k_weight)) || (norm && !(eps >= 0.f && std::isfinite(eps))) ||
      !valid_dtype(weight_dtype))
    return DIT_ERR_INVALID_ARG;
  const int wsize = dtype_bytes(weight_dtype);
  // The rotation: frequencies of all pairs, and positions given, or packed requests.
  if ((axes > 0) != (freqs != nullptr) || axes < 0 || (!norm && !freqs)) return DIT_ERR_INVALID_ARG;
  if (axes > 4) return DIT_ERR_UNSUPPORTED;
  long long pairs = 0;
  if (freqs) {
    if (!axis_pairs || !aligned(freqs, 4) || (interleaved != 0 && interleaved != 1) || !std::isfinite(rot_scale))
      return DIT_ERR_INVALID_ARG;
    for (int a = 0; a < axes; ++a) {
      if (axis_pairs[a] < 0) return DIT_ERR_INVALID_ARG;
      pairs += axis_pairs[a];
    }
    if (pairs < 1 || 2 * pairs > D) return DIT_ERR_INVALID_ARG;
    if (pairs % 8 != 0) return DIT_ERR_UNSUPPORTED;
    const bool packed = !positions;
    if (!aligned(positions, 4) || !aligned(cu_new, 4) || !aligned(start_lens, 4)) return DIT_ERR_INVALID_ARG;
    if (packed && (!cu_new || !start_lens || requests < 1 || requests > kMaxRequests || B != 1 || axes != 1))
      return DIT_ERR_INVALID_ARG;
    if (!packed && (cu_new || start_lens || pos_b < 0 || pos_axis < 0 || pos_b > kMaxSpan / B || pos_axis > kMaxSpan / 4))
      return DIT_ERR_INVALID_ARG;
  } else if (positions || cu_new || start_lens) {
    return DIT_ERR_INVALID_ARG;
  }
  for (int i = 0; i < sides; ++i) {
    if (!in[i].valid(B, N) || !out[i].valid(B, N) || !aligned(weight[i], wsize)) return DIT_ERR_INVALID_ARG;
    if (!no_self_overlap(out[i].s, B, out[i].H, N, D)) return DIT_ERR_INVALID_ARG;
  }
  const long long pos_span = positions ? ((B - 1) * pos_b + (axes - 1) * pos_axis + N) * 4 : 0;
  const Range reads[] = {span(q_weight, q_weight ? D * wsize : 0), span(k_weight, k_weight ? D * wsize : 0),
                         span(freqs, freqs ? pairs * 4 : 0), span(positions, pos_span),
                         span(cu_new, cu_new ? 4LL * (requests + 1LL) : 0), span(start_lens, start_lens ? 4LL * requests : 0)};
  for (int i = 0; i < sides; ++i) {
    for (const Range& r : reads)
      if (overlap(out[i].range(B, N, D), r)) return DIT_ERR_INVALID_ARG;
    // In place, or apart.
    for (int j = 0; j < sides; ++j)
      if (!(i == j && out[i].same(in[j])) && !views_apart(out[i], in[j], B, N, D)) return DIT_ERR_INVALID_ARG;
  }
  if (sides == 2 && !views_apart(out[0], out[1], B, N, D)) return DIT_ERR_INVALID_ARG;
  ditattn::RopeLaunch a{};
  for (int i = 0; i < sides; ++i) {
    a.in[i] = in[i].p;
    a.out[i] = const_cast<void*>(out[i].p);
    a.is[i] = {in[i].s.b, in[i].s.h, in[i].s.n};
    a.os[i] = {out[i].s.b, out[i].s.h, out[i].s.n};
    a.weight[i] = weight[i];
    a.heads[i] = in[i].H;
  }
  a.weight_f32 = weight_dtype == DIT_F32;
  a.norm = norm != 0;
  a.interleaved = interleaved != 0;
  a.eps = eps;
  a.rot_scale = rot_scale;
  a.positions = positions;
  a.pos_b = pos_b;
  a.pos_axis = pos_axis;
  a.cu_new = cu_new;
  a.start_lens = start_lens;
  a.requests = requests;
  a.freqs = freqs;
  a.pairs = static_cast<int>(pairs);
  a.axes = axes;
  for (int i = 0; i < axes; ++i) a.axis_pairs[i] = axis_pairs[i];
  a.batch = B;
  a.n = N;
  a.d = D;
  return done(ditattn::launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream)));
}

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
  if (T < 1 || T > kMaxTokens || B < 1 || B > kMaxRequests) return DIT_ERR_INVALID_ARG;
  dit_status s = check_heads(T, H_q, H_kv, D);
  if (s != DIT_OK) return s;
  s = check_pages(page_size, n_pages, max_pages);
  if (s != DIT_OK) return s;
  if (H_q / H_kv > 128 /* a tile's rows */ || !room_counts(page_size, max_pages)) return DIT_ERR_UNSUPPORTED;
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

dit_status dit_paged_page_mass(const void* q, const dit_strides* q_strides, const float* lse, const void* k_cache,
                               const dit_strides* k_strides, const int* block_table, long long table_stride,
                               const int* seq_lens, const int* cu_new, const int* start_lens, const float* mass,
                               float* mass_out, int T, int B, int H_q, int H_kv, int D, int page_size,
                               int n_pages, int max_pages, int window, float scale, dit_stream stream) {
  if (T < 1 || T > kMaxTokens || B < 1 || B > kMaxRequests || window < 0) return DIT_ERR_INVALID_ARG;
  if (!cu_new && (T != B || start_lens)) return DIT_ERR_INVALID_ARG;
  dit_status s = check_heads(T, H_q, H_kv, D);
  if (s != DIT_OK) return s;
  s = check_pages(page_size, n_pages, max_pages);
  if (s != DIT_OK) return s;
  if (H_q / H_kv > 256 /* a product's columns */ || !room_counts(page_size, max_pages)) return DIT_ERR_UNSUPPORTED;
  const dit_strides qs = token_strides(q_strides, T, H_q, D);
  const dit_strides ks = cache_strides(k_strides, n_pages, H_kv, page_size, D);
  if (!valid_tokens(q, qs, T, H_q) || qs.h >= (1LL << 39) / (H_q / H_kv) || !valid_cache(k_cache, ks, n_pages, H_kv) || !lse || !aligned(lse, 4) ||
      !valid_table(block_table, table_stride, B, max_pages) || !seq_lens || !aligned(seq_lens, 4) ||
      !aligned(cu_new, 4) || !aligned(start_lens, 4) || !mass || !aligned(mass, 4) || !mass_out || !aligned(mass_out, 4))
    return DIT_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale * 1.4426950408889634f)) return DIT_ERR_INVALID_ARG;
  const Range out = span(mass_out, 4LL * n_pages * H_kv);
  const Range ins[] = {span(q, view_span(qs, 1, H_q, T, D, 2)), span(lse, 4LL * T * H_q),
                       cache_range(k_cache, ks, n_pages, H_kv, page_size, D),
                       span(block_table, table_bytes(B, max_pages, table_stride)), span(seq_lens, 4LL * B),
                       span(cu_new, cu_new ? 4LL * (B + 1LL) : 0), span(start_lens, start_lens ? 4LL * B : 0)};
  for (const Range& in : ins)
    if (overlap(out, in)) return DIT_ERR_INVALID_ARG;
  if (mass != mass_out && overlap(out, span(mass, 4LL * n_pages * H_kv))) return DIT_ERR_INVALID_ARG;
  ditattn::MassLaunch a;
  a.q = q;
  a.q_n = qs.n;
  a.q_h = qs.h;
  a.lse = lse;
  a.k_cache = k_cache;
  a.ks = {ks.b, ks.h, ks.n};
  a.table = block_table;
  a.table_stride = table_stride;
  a.seq_lens = seq_lens;
  a.cu_new = cu_new;
  a.start_lens = start_lens;
  a.mass = mass;
  a.mass_out = mass_out;
  a.tokens = T;
  a.batch = B;
  a.h_q = H_q;
  a.h_kv = H_kv;
  a.d = D;
  a.page_size = page_size;
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  a.window = window;
  a.scale = scale;
  a.status = ditattn::status_word();
  if (!a.status) return DIT_ERR_CUDA;
  return done(ditattn::launch_paged_mass(a, static_cast<cudaStream_t>(stream)));
}

size_t dit_paged_evict_workspace_bytes(int B, int max_pages) {
  if (B < 1 || max_pages < 1) return 0;
  return ditattn::paged_evict_workspace(B, max_pages);
}

dit_status dit_paged_evict(const float* mass, const int* block_table, long long table_stride, int* table_out,
                           long long table_out_stride, const int* seq_lens, int* seq_lens_out, int* free_pages,
                           const int* n_free, int* n_free_out, int B, int H_kv, int page_size, int n_pages,
                           int max_pages, int pool_capacity, int keep, int recent, void* workspace,
                           size_t workspace_bytes, dit_stream stream) {
  if (B < 1 || H_kv < 1 || pool_capacity < 0 || keep < 1 || recent < 1 || recent > keep) return DIT_ERR_INVALID_ARG;
  const dit_status s = check_pages(page_size, n_pages, max_pages);
  if (s != DIT_OK) return s;
  if (B > ditattn::kEvictMaxBatch) return DIT_ERR_UNSUPPORTED;
  if (!mass || !seq_lens || !seq_lens_out || !n_free || !n_free_out || (!free_pages && pool_capacity > 0))
    return DIT_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(mass), static_cast<const void*>(seq_lens),
                        static_cast<const void*>(seq_lens_out), static_cast<const void*>(free_pages),
                        static_cast<const void*>(n_free), static_cast<const void*>(n_free_out)})
    if (!aligned(p, 4)) return DIT_ERR_INVALID_ARG;
  if (!valid_table(block_table, table_stride, B, max_pages) || !valid_table(table_out, table_out_stride, B, max_pages))
    return DIT_ERR_INVALID_ARG;
  const bool in_place = table_out == block_table && (B == 1 || table_out_stride == table_stride);
  const size_t need = dit_paged_evict_workspace_bytes(B, max_pages);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return DIT_ERR_INVALID_ARG;
  const Range table = span(block_table, table_bytes(B, max_pages, table_stride));
  const Range outs[] = {span(table_out, table_bytes(B, max_pages, table_out_stride)), span(seq_lens_out, 4LL * B),
                        span(free_pages, 4LL * pool_capacity), span(n_free_out, 4),
                        span(workspace, static_cast<long long>(need))};
  const Range ins[] = {table, span(seq_lens, 4LL * B), span(mass, 4LL * n_pages * H_kv), span(n_free, 4)};
  // (Rows of the two tables may lie in turn, in one allocation.)
  const bool tables_apart = rows_apart(block_table, table_stride, table_out, table_out_stride, B, max_pages);
  const bool same[5] = {in_place, seq_lens_out == seq_lens, false, n_free_out == n_free, false};
  const int of[5] = {0, 1, -1, 3, -1};  // the input that an output may be
  for (int i = 0; i < 5; ++i) {
    for (int j = i + 1; j < 5; ++j)
      if (overlap(outs[i], outs[j])) return DIT_ERR_INVALID_ARG;
    for (int j = 0; j < 4; ++j)
      if (!(same[i] && j == of[i]) && overlap(outs[i], ins[j]) && !(i == 0 && j == 0 && tables_apart))
        return DIT_ERR_INVALID_ARG;
  }
  ditattn::EvictLaunch a{mass,   block_table, table_stride, table_out, table_out_stride, seq_lens,  seq_lens_out, free_pages,
                         n_free, n_free_out,  B,            H_kv,      page_size,        n_pages,   max_pages,    pool_capacity,
                         keep,   recent,      workspace};
  return done(ditattn::launch_paged_evict(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
