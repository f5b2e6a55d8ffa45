// The pages whose keys can score highest for one query token of each request:
//   score_i = max_h sum_d max(q_hd lo_id, q_hd hi_id)
// over the query heads h of a key/value head's group, in 64 bits; listed are the newest page
// and the top_k - 1 others with the highest scores, ties to the lower index.
//
// A block per (request, key/value head) scores its pages, ranks each against all others and
// writes those of the first top_k in ascending order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "paged_launch.h"

namespace ditattn {
namespace {

constexpr int kSelThreads = 256;

__global__ void __launch_bounds__(kSelThreads) paged_select_simple(const SelectLaunch a) {
  __shared__ int written;
  const int b = blockIdx.x / a.h_kv, g = blockIdx.x % a.h_kv, group = a.h_q / a.h_kv;
  const int P = a.page_size;
  const int len = min(max(0, a.seq_lens[b]), a.max_pages * P);
  const int n = pages_of(len, P);
  int* out = a.selected + static_cast<long long>(blockIdx.x) * a.top_k;
  double* score = static_cast<double*>(a.workspace) + static_cast<long long>(blockIdx.x) * a.max_pages;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + b * a.q_b + g * group * a.q_h;
  for (int i = threadIdx.x; i < n; i += kSelThreads) {
    double best = -INFINITY;
    const int page = a.table[b * a.table_stride + i];
    if (i == n - 1) {
      best = INFINITY;
    } else if (page >= 0 && page < a.n_pages) {
      const __nv_bfloat16* lo = static_cast<const __nv_bfloat16*>(a.summary) + (static_cast<long long>(page) * a.h_kv + g) * 2 * a.d;
      for (int h = 0; h < group; ++h) {
        double s = 0;
        for (int d = 0; d < a.d; ++d) {
          const double x = static_cast<double>(__bfloat162float(q[h * a.q_h + d]));
          const double u = x * static_cast<double>(__bfloat162float(lo[d])), v = x * static_cast<double>(__bfloat162float(lo[a.d + d]));
          s += u != u ? u : v != v ? v : fmax(u, v);
        }
        if (s != s) s = INFINITY;
        best = fmax(best, s);
      }
    }
    score[i] = best;
  }
  if (threadIdx.x == 0) written = 0;
  __syncthreads();
  for (int i0 = 0; i0 < n; i0 += kSelThreads) {
    const int i = i0 + threadIdx.x;
    int in = 0;
    if (i < n) {
      int better = i == n - 1 ? 0 : 1;  // the newest page comes first, whatever the others score
      for (int j = 0; j < n - 1 && i < n - 1; ++j)
        better += score[j] > score[i] || (score[j] == score[i] && j < i);
      in = better < a.top_k;
    }
    __shared__ int warp_n[kSelThreads / 32];
    const unsigned bal = __ballot_sync(~0u, in);
    if ((threadIdx.x & 31) == 0) warp_n[threadIdx.x >> 5] = __popc(bal);
    __syncthreads();
    int at = written + __popc(bal & ((1u << (threadIdx.x & 31)) - 1));
    for (int w = 0; w < static_cast<int>(threadIdx.x >> 5); ++w) at += warp_n[w];
    if (in) out[at] = i;
    __syncthreads();
    if (threadIdx.x == 0)
      for (int w = 0; w < kSelThreads / 32; ++w) written += warp_n[w];
    __syncthreads();
  }
  for (int k = written + threadIdx.x; k < a.top_k; k += kSelThreads) out[k] = -1;
}

}  // namespace

size_t paged_select_workspace(int batch, int h_kv, int max_pages) {
  return static_cast<size_t>(batch) * h_kv * max_pages * 8;
}

cudaError_t launch_paged_select(const SelectLaunch& a, cudaStream_t st) {
  paged_select_simple<<<static_cast<unsigned>(a.batch) * a.h_kv, kSelThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace ditattn
