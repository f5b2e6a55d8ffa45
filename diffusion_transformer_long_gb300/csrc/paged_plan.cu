// Block tables and slot maps of one step of a batch, from the requests' lengths.
//
// With s_b cached and n_b new tokens, P rows a page, F free pages:
//   cu_b   = sum_{a<b} n_a                      first row of request b in the step's batch
//   need_b = ceil((s_b + n_b) / P) - ceil(s_b / P),  off_b = sum_{a<b} need_a
//   grant j = 0 .. min(F, sum need) - 1 is free_pages[F - 1 - j]; it becomes page
//             ceil(s_b / P) + j - off_b of the request b with off_b <= j < off_b + need_b
//   token t of request b sits at position s_b + t - cu_b of its request
// Both sums are 32-bit and saturate (they are bounded by max_tokens and the grants).
//
// Every block scans all lengths for itself (B <= 8192) into shared memory and takes its share of
// the tokens and the grants; a token finds its request by bisection of the prefix sums.  One
// block serves up to kTokensPerBlock tokens alone.  Where several blocks share the tokens and
// the lengths or the count are updated in place, those are written by a second launch, since
// no block may overwrite what another has yet to read.  Bound by latency: the launch, one
// dependent read of the lengths, two block scans, one dependent read of the table (256 requests
// of one token 3.9 us, 63 of 75569 tokens 5.0 us, in a captured graph).
#include <cuda_runtime.h>

#include <algorithm>

#include "paged_device.cuh"
#include "paged_launch.h"

namespace ditattn {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kTokensPerBlock = 2048;

struct PlanParams {
  PlanLaunch a;
  int cap;  // tokens a table row can hold
  int fill, commit;  // what this launch writes: slots, table and first tokens; lengths and count
};

__device__ __forceinline__ int sat_add(int x, int y) {
  return static_cast<int>(min(static_cast<unsigned>(x) + static_cast<unsigned>(y), 0x7fffffffu));
}

// Sum of the block's lower threads' values, saturating at 2^31 - 1 (all values >= 0).
__device__ int block_exclusive(int x, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(~0u, x, d);
    if (lane >= d) x = sat_add(x, y);
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = lane < static_cast<int>(blockDim.x >> 5) ? warp_sums[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(~0u, w, d);
      if (lane >= d) w = sat_add(w, y);
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  x = __shfl_up_sync(~0u, x, 1);
  if (lane == 0) x = 0;
  return warp > 0 ? sat_add(x, warp_sums[warp - 1]) : x;
}

// The request r with first[r] <= x < first[r + 1], for x < first[n].
__device__ __forceinline__ int find(const int* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PlanParams p) {
  extern __shared__ int sm[];
  wait_for_inputs();
  __shared__ int warp_sums[32];
  const int B = p.a.batch, P = p.a.page_size;
  int* cu = sm;               // [B + 1]
  int* off = cu + B + 1;      // [B + 1]
  int* old = off + B + 1;     // [B]
  const int per = (B + blockDim.x - 1) / blockDim.x;
  const int b0 = min(B, static_cast<int>(threadIdx.x) * per), b1 = min(B, b0 + per);

  // first tokens, capped at max_tokens: every n_b below counts kept tokens only
  int sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = max(0, p.a.new_lens[b]);
    cu[b + 1] = n;
    sum = sat_add(sum, n);
    old[b] = min(max(0, p.a.seq_lens[b]), p.cap);
  }
  const int free = min(max(0, *p.a.n_free), p.a.pool_capacity);
  int run = block_exclusive(sum, warp_sums);
  for (int b = b0; b < b1; ++b) {
    run = sat_add(run, cu[b + 1]);
    cu[b + 1] = min(run, p.a.max_tokens);
  }
  if (threadIdx.x == 0) cu[0] = off[0] = 0;
  __syncthreads();
  sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int want = min(sat_add(old[b], cu[b + 1] - cu[b]), p.cap);
    const int need = pages_of(want, P) - pages_of(old[b], P);
    off[b + 1] = need;
    sum = sat_add(sum, need);
  }
  run = block_exclusive(sum, warp_sums);
  for (int b = b0; b < b1; ++b) {
    run = sat_add(run, off[b + 1]);
    off[b + 1] = run;
  }
  __syncthreads();  // this block has read seq_lens and n_free: alone, it may write them in place

  const int step = gridDim.x * blockDim.x, first = blockIdx.x * blockDim.x + threadIdx.x;
  const int grants = min(free, off[B]);
  if (p.commit) {
    for (int b = first; b < B; b += step) {
      const int have = pages_of(old[b], P);
      const int got = min(max(0, free - off[b]), off[b + 1] - off[b]);
      const int want = min(sat_add(old[b], cu[b + 1] - cu[b]), p.cap);
      p.a.seq_lens_out[b] =
          static_cast<int>(min(static_cast<long long>(want), static_cast<long long>(have + got) * P));
    }
    if (first == 0) *p.a.n_free_out = free - grants;
  }
  if (!p.fill) return;
  for (int b = first; b <= B; b += step) p.a.cu_new[b] = cu[b];
  for (int j = first; j < grants; j += step) {
    const int b = find(off, B, j);
    p.a.table[b * p.a.table_stride + pages_of(old[b], P) + j - off[b]] = p.a.free_pages[free - 1 - j];
  }
  const int total = cu[B];
  for (int t = first; t < p.a.max_tokens; t += step) {
    long long slot = -1;
    if (t < total) {
      const int b = find(cu, B, t);
      const long long pos = static_cast<long long>(old[b]) + (t - cu[b]);
      if (pos < p.cap) {
        const int i = static_cast<int>(pos) / P, have = pages_of(old[b], P);
        int page = -1;
        if (i < have) {
          page = p.a.table[b * p.a.table_stride + i];  // in the row before this step: not written here
        } else {
          const int j = off[b] + i - have;
          if (j < grants) page = p.a.free_pages[free - 1 - j];
        }
        if (page >= 0 && page < p.a.n_pages)
          slot = static_cast<long long>(page) * P + (static_cast<int>(pos) - i * P);
      }
    }
    p.a.slots[t] = slot;
  }
}

}  // namespace

cudaError_t launch_paged_plan(const PlanLaunch& a, cudaStream_t st) {
  PlanParams p;
  p.a = a;
  p.cap = a.max_pages * a.page_size;
  const int smem = (3 * a.batch + 2) * static_cast<int>(sizeof(int));
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (3 * kPlanMaxBatch + 2) * static_cast<int>(sizeof(int)));
    if (e != cudaSuccess) return e;
  }
  // Few requests and tokens: a small block, whose scans and barriers are shorter.
  const int threads = std::max(a.batch, std::min(a.max_tokens, kTokensPerBlock)) <= 512 ? 256 : kPlanThreads;
  const int blocks = std::min((a.max_tokens + kTokensPerBlock - 1) / kTokensPerBlock, 256);
  const bool in_place = a.seq_lens_out == a.seq_lens || a.n_free_out == a.n_free;
  p.fill = 1;
  p.commit = blocks == 1 || !in_place;
  cudaError_t e = launch_after(paged_plan_kernel, dim3(blocks), dim3(threads), smem, st, p);
  if (e == cudaSuccess && !p.commit) {
    p.fill = 0;
    p.commit = 1;
    e = launch_after(paged_plan_kernel, dim3(1), dim3(kPlanThreads), smem, st, p);
  }
  return e;
}

}  // namespace ditattn
