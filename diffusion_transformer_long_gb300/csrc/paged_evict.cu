// Eviction: the pages of long requests that drew least attention weight leave the block table and go back to the
// stack of free pages.
//
// Request b of n = ceil(len / page_size) pages, n > keep, keeps its newest `recent` pages and, of the others, the
// keep - recent of most weight, x_i = sum_h mass[page_i, h] in 64 bits (ties: the lowest index).  The kept ones close
// up in order, the entries behind them become -1, and the length falls by page_size a page: the newest page stays, so
// that all that go are full.  Freed pages follow each other on the stack by request and column.
//
// Two launches.  The first turns weights into 64-bit keys whose order is the numbers' (NaN above all, an entry without
// a page below all), over the whole GPU: an SM adds two numbers of 64 bits a clock.  It also counts what a request can
// give back, and keeps the lengths and the stack's height as they were.  In the second a block a request finds the
// border key digit by digit, eight bits a pass (from the first bit that not all share, and no further than tells the
// kept ones from the others), places what is kept and what goes by scans over flags, and knows from the counts where on
// the stack its pages go.  Bound by latency: the bytes would take 0.3 us (16 x 75600 keys in pages of 16, 8 heads) and
// 0.1 us (256 requests of up to 4608 in pages of 64, 24 heads), the two launches take 23 and 14 us in a graph
// (28.8 and 14.7 with 512 columns placed at a time and the search begun at the top digit; chunks of 256 columns in the
// first launch and 1024 threads in the second change nothing).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "paged_device.cuh"
#include "paged_launch.h"

namespace ditattn {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kChunk = 1024;  // table columns of a scoring block
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 4;  // table columns a thread places at a time
constexpr int kShared = 12288;  // keys that stay in shared memory

struct EvictParams {
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
  // workspace
  int* height;     // the stack's, before
  int* lens;       // [batch], before
  int* counts;     // [batch][chunks]: pages of the pool among the columns in front of the newest
  uint64_t* keys;  // [batch][max_pages]
  int batch, h_kv, page_size, n_pages, max_pages, chunks, capacity, keep, recent;
};

// x's place in the order of the numbers, as a whole number: NaN above all, -0 as 0.
__device__ __forceinline__ uint64_t ordered(double x) {
  if (x != x) return ~0ull;
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return bits >> 63 ? ~bits : bits | 0x8000000000000000ull;
}

__device__ __forceinline__ int length_of(const EvictParams& p, int b) {
  return min(max(p.seq_lens[b], 0), p.max_pages * p.page_size);
}

__global__ void __launch_bounds__(kScoreThreads) score_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int part[kScoreThreads / 32];
  const int chunk = blockIdx.x, b = blockIdx.y;
  wait_for_inputs();
  const int len = length_of(p, b), n = pages_of(len, p.page_size);
  if (chunk == 0 && threadIdx.x == 0) {
    p.lens[b] = len;
    if (b == 0) *p.height = min(max(*p.n_free, 0), p.capacity);
  }
  if (n <= p.keep) return;
  const int old = n - p.recent;
  int count = 0;
  for (int i = chunk * kChunk + threadIdx.x; i < min(old, (chunk + 1) * kChunk); i += kScoreThreads) {
    const int page = p.table[b * p.table_stride + i];
    uint64_t x = 0;  // below every number's
    if (page >= 0 && page < p.n_pages) {
      const float* m = p.mass + static_cast<long long>(page) * p.h_kv;
      double sum = 0;
#pragma unroll 8
      for (int h = 0; h < p.h_kv; ++h) sum += m[h];
      x = ordered(sum);
      ++count;
    }
    p.keys[static_cast<long long>(b) * p.max_pages + i] = x;
  }
  count = __reduce_add_sync(~0u, count);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = count;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kScoreThreads / 32; ++w) count += part[w];
    p.counts[static_cast<long long>(b) * p.chunks + chunk] = count;
  }
}

// Exclusive sum over the block of a number of each thread, and the total.
__device__ __forceinline__ int scan(int x, int* warps, int& total) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int upto = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, upto, o);
    if (lane >= o) upto += y;
  }
  __syncthreads();  // the last use of `warps` is over
  if (lane == 31) warps[warp] = upto;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? warps[w] : 0;
    total += warps[w];
  }
  return before + upto - x;
}

// Pages that request b gives back.
__device__ __forceinline__ int gives(const EvictParams& p, int b) {
  const int n = pages_of(p.lens[b], p.page_size);
  if (n <= p.keep) return 0;
  int have = 0;
  for (int c = 0; c * kChunk < n - p.recent; ++c) have += p.counts[static_cast<long long>(b) * p.chunks + c];
  return max(0, have - (p.keep - p.recent));  // (entries without a page go first)
}

__global__ void __launch_bounds__(kThreads) evict_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(8) unsigned char smem[];
  __shared__ int hist[256];
  __shared__ int warps[kWarps];
  __shared__ unsigned spread[2];  // bits in which keys differ
  __shared__ int found[3];  // the border's digit, how many to take among those that share it, and whether that is all
  const int b = blockIdx.x;
  wait_for_inputs();
  const int len = p.lens[b], n = pages_of(len, p.page_size);
  const int* const row = p.table + b * p.table_stride;
  int* const out = p.table_out + b * p.out_stride;
  const bool last = b == p.batch - 1;
  if (n <= p.keep && !last) {
    if (out != row)
      for (int i = threadIdx.x; i < p.max_pages; i += kThreads) out[i] = row[i];
    if (threadIdx.x == 0) p.lens_out[b] = len;
    return;
  }
  // Where on the stack the request's pages go.
  if (threadIdx.x < 2) spread[threadIdx.x] = 0;
  int before = 0;
  for (int i = threadIdx.x; i < b; i += kThreads) before += gives(p, i);
  int all;
  scan(before, warps, all);
  const long long height = static_cast<long long>(*p.height) + all;
  if (last && threadIdx.x == 0)
    *p.n_free_out = static_cast<int>(min(height + gives(p, b), static_cast<long long>(p.capacity)));
  if (n <= p.keep) {
    if (out != row)
      for (int i = threadIdx.x; i < p.max_pages; i += kThreads) out[i] = row[i];
    if (threadIdx.x == 0) p.lens_out[b] = len;
    return;
  }

  const int old = n - p.recent, want = p.keep - p.recent;  // 0 <= want < old
  const uint64_t* key = p.keys + static_cast<long long>(b) * p.max_pages;
  const uint64_t first = key[0];
  uint64_t differ = 0;
  uint64_t* const mine = reinterpret_cast<uint64_t*>(smem);
  for (int i = threadIdx.x; i < old; i += kThreads) {
    const uint64_t x = key[i];
    differ |= x ^ first;
    if (old <= kShared) mine[i] = x;
  }
  if (old <= kShared) key = mine;
  for (int half = 0; half < 2; ++half) {
    const unsigned x = __reduce_or_sync(~0u, static_cast<unsigned>(differ >> (32 * half)));
    if (threadIdx.x % 32 == 0) atomicOr(&spread[half], x);
  }
  __syncthreads();
  // The search starts with the first bit in which some differ: what all share would have every thread count in one
  // place (weights of one sign and few exponents do for ten bits).
  int rest = 64 - __clzll(static_cast<long long>(static_cast<uint64_t>(spread[1]) << 32 | spread[0]));
  // Taken are the keys above the border, and the first `left` of those equal to it.
  uint64_t border = want == 0 ? ~0ull : rest < 64 ? first & ~0ull << rest : 0;
  int left = want;
  while (want > 0 && rest > 0) {
    if (threadIdx.x < 256) hist[threadIdx.x] = 0;
    __syncthreads();
    const uint64_t above = rest == 64 ? 0 : ~0ull << rest;
    const int width = min(rest, 8), shift = rest - width;
    for (int i = threadIdx.x; i < old; i += kThreads)
      if ((key[i] & above) == border) atomicAdd(&hist[key[i] >> shift & ((1 << width) - 1)], 1);
    __syncthreads();
    if (threadIdx.x < 32) {
      // Lane l: digits 255 - 8 l and the seven below it.
      int mine = 0;
      for (int d = 0; d < 8; ++d) mine += hist[255 - 8 * threadIdx.x - d];
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, upto, o);
        if (threadIdx.x >= o) upto += y;
      }
      int more = upto - mine;  // keys of larger digits
      if (more < left && upto >= left)
        for (int d = 0;; ++d) {
          const int digit = 255 - 8 * threadIdx.x - d;
          if (more + hist[digit] >= left) {
            found[0] = digit;
            found[1] = left - more;
            found[2] = more + hist[digit] == left;
            break;
          }
          more += hist[digit];
        }
    }
    __syncthreads();
    border |= static_cast<uint64_t>(found[0]) << shift;
    left = found[1];
    rest = shift;
    if (found[2]) {  // all that begin like this are taken: those not below it (it is not 0: some key is not taken)
      --border;
      left = 0;
      break;
    }
    __syncthreads();
  }
  __syncthreads();
  // In chunks of kPer neighbours a thread, each chunk read before its places, which are never behind it, are written.
  int kept = 0, dropped = 0, equal = 0;
  for (int i0 = 0; i0 < n; i0 += kThreads * kPer) {
    const int i = i0 + threadIdx.x * kPer;
    int page[kPer], total;
    unsigned same = 0, stays = 0, goes = 0;  // a bit a neighbour
#pragma unroll
    for (int j = 0; j < kPer; ++j) page[j] = i + j < n ? row[i + j] : -1;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint64_t x = i + j < old ? key[i + j] : 0;
      same |= static_cast<unsigned>(i + j < old && left > 0 && x == border) << j;
      stays |= static_cast<unsigned>(i + j < n && (i + j >= old || x > border)) << j;
    }
    if (left > 0) {
      int rank = equal + scan(__popc(same), warps, total);
      equal += total;
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (same >> j & 1 && rank++ < left) stays |= 1u << j;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      goes |= static_cast<unsigned>(!(stays >> j & 1) && page[j] >= 0 && page[j] < p.n_pages) << j;
    const int at = scan(__popc(stays) | __popc(goes) << 16, warps, total);
    int place = kept + (at & 0xffff);
    long long top = height + dropped + (at >> 16);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (stays >> j & 1) out[place++] = page[j];
      if (goes >> j & 1) {
        if (top < p.capacity) p.stack[top] = page[j];
        ++top;
      }
    }
    kept += total & 0xffff;
    dropped += total >> 16;
  }
  __syncthreads();
  for (int i = p.keep + threadIdx.x; i < p.max_pages; i += kThreads)
    if (i < n || out != row) out[i] = i < n ? -1 : row[i];
  if (threadIdx.x == 0) p.lens_out[b] = len - (n - p.keep) * p.page_size;
}

long long aligned16(long long x) { return (x + 15) / 16 * 16; }

}  // namespace

size_t paged_evict_workspace(int batch, int max_pages) {
  const long long chunks = (max_pages + kChunk - 1) / kChunk;
  return 16 + aligned16(4LL * batch) + aligned16(4LL * batch * chunks) + 8LL * batch * max_pages;
}

cudaError_t launch_paged_evict(const EvictLaunch& a, cudaStream_t st) {
  EvictParams p;
  p.mass = a.mass;
  p.table = a.table;
  p.table_stride = a.table_stride;
  p.table_out = a.table_out;
  p.out_stride = a.out_stride;
  p.seq_lens = a.seq_lens;
  p.lens_out = a.lens_out;
  p.stack = a.stack;
  p.n_free = a.n_free;
  p.n_free_out = a.n_free_out;
  p.batch = a.batch;
  p.h_kv = a.h_kv;
  p.page_size = a.page_size;
  p.n_pages = a.n_pages;
  p.max_pages = a.max_pages;
  p.chunks = (a.max_pages + kChunk - 1) / kChunk;
  p.capacity = a.capacity;
  p.keep = a.keep;
  p.recent = a.recent;
  char* w = static_cast<char*>(a.workspace);
  p.height = reinterpret_cast<int*>(w);
  p.lens = reinterpret_cast<int*>(w += 16);
  p.counts = reinterpret_cast<int*>(w += aligned16(4LL * a.batch));
  p.keys = reinterpret_cast<uint64_t*>(w += aligned16(4LL * a.batch * p.chunks));
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared * 8);
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  e = launch_after(score_kernel, dim3(p.chunks, a.batch), dim3(kScoreThreads), 0, st, p);
  if (e != cudaSuccess) return e;
  const size_t smem = 8 * static_cast<size_t>(std::min(a.max_pages, kShared));
  return launch_after(evict_kernel, dim3(a.batch), dim3(kThreads), smem, st, p);
}

}  // namespace ditattn
