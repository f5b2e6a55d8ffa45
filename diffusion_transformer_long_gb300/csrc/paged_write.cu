// Keys and values of new tokens into their slots of the paged caches, and the touched pages'
// summaries (per channel minimum and maximum of the keys).
//
// A copy of T * H rows of 2 D bytes twice over: bound by HBM for long prefills, by latency
// for a decode step.  Without a summary every (token, head) row stands alone: a thread moves 16
// bytes of it, in the order of the new rows.  With one, a page's extremes need all its new rows
// together: the tokens of a page follow each other, so each maximal run of consecutive slots in
// one page has exactly one owner, the window of tokens in which it begins.  A thread of that
// window has 8 channels of one head: it moves them for all of the run's tokens, keeps their
// running extremes in registers and merges them with the page's earlier summary (or starts it
// anew, where the run holds row 0): no atomics, no exchange between threads, and neighbouring
// threads read whole tokens, as without a summary.  Measured: 27280 tokens of 24 heads of 128, pages
// of 64: 110 us, 6.1 TB/s (without summaries 104 us; a copy's rate here is 6.8 TB/s); 64 tokens of 8
// heads 2.4 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "paged_device.cuh"
#include "paged_launch.h"

namespace ditattn {
namespace {

constexpr int kWriteThreads = 128;  // (256: 0.5 to 1 % slower for long prefills)

struct WriteParams {
  const char* k_new;
  const char* v_new;
  long long kn_n, kn_h, vn_n, vn_h;  // bytes
  const long long* slots;
  char* k_cache;
  char* v_cache;
  long long ks_p, ks_h, ks_r, vs_p, vs_h, vs_r;  // page, head, row strides (bytes)
  char* summary;
  long long n_slots;
  long long threads;  // with a summary: windows * columns (16 bytes of a head), or * heads (blocks)
  int tokens, heads, page_size, window, few;
};

// kVpr: 16-byte vectors per row.  One thread per vector of a (token, head) row.
template <int kVpr>
__global__ void __launch_bounds__(kWriteThreads) paged_write_rows(const __grid_constant__ WriteParams p) {
  wait_for_inputs();
  const long long i = static_cast<long long>(blockIdx.x) * kWriteThreads + threadIdx.x;
  const long long row = i / kVpr;
  const int t = static_cast<int>(row / p.heads), h = static_cast<int>(row - static_cast<long long>(t) * p.heads);
  if (t >= p.tokens) return;
  const int vec = static_cast<int>(i % kVpr) * 16;
  const long long slot = p.slots[t];
  if (slot < 0 || slot >= p.n_slots) return;
  const long long page = slot / p.page_size, r = slot - page * p.page_size;
  const uint4 k = load_once(p.k_new + t * p.kn_n + h * p.kn_h + vec);
  const uint4 v = load_once(p.v_new + t * p.vn_n + h * p.vn_h + vec);
  *reinterpret_cast<uint4*>(p.k_cache + page * p.ks_p + h * p.ks_h + r * p.ks_r + vec) = k;
  *reinterpret_cast<uint4*>(p.v_cache + page * p.vs_p + h * p.vs_h + r * p.vs_r + vec) = v;
}

// Extremes of 8 bf16 channels; NaN in either operand gives NaN.
struct Ext {
  __nv_bfloat162 lo[4], hi[4];
  __device__ __forceinline__ void take(const uint4& x, bool first) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 y;
      memcpy(&y, &w[i], 4);
      lo[i] = first ? y : __hmin2_nan(lo[i], y);
      hi[i] = first ? y : __hmax2_nan(hi[i], y);
    }
  }
  __device__ __forceinline__ void take(const Ext& e) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = __hmin2_nan(lo[i], e.lo[i]);
      hi[i] = __hmax2_nan(hi[i], e.hi[i]);
    }
  }
  __device__ __forceinline__ Ext shuffled(int d) const {
    Ext e;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e.lo[i] = __shfl_xor_sync(~0u, lo[i], d);
      e.hi[i] = __shfl_xor_sync(~0u, hi[i], d);
    }
    return e;
  }
};

__device__ __forceinline__ uint4 pack(const __nv_bfloat162 (&x)[4]) {
  uint4 r;
  memcpy(&r, x, 16);
  return r;
}

// The next token of a run at (page, row), or a token without a slot (row < 0).
struct Place {
  long long page;
  int row;
};
__device__ __forceinline__ Place place_of(long long slot, long long n_slots, int page_size) {
  if (slot < 0 || slot >= n_slots) return {0, -1};
  if (n_slots <= 0xffffffffLL) {  // a 32-bit division is several times cheaper
    const unsigned s = static_cast<unsigned>(slot), page = s / page_size;
    return {static_cast<long long>(page), static_cast<int>(s - page * page_size)};
  }
  const long long page = slot / page_size;
  return {page, static_cast<int>(slot - page * page_size)};
}

template <int kVpr>
__global__ void __launch_bounds__(kWriteThreads) paged_write_runs(const __grid_constant__ WriteParams p) {
  constexpr int kAhead = 4;  // tokens in flight
  wait_for_inputs();
  const long long id = static_cast<long long>(blockIdx.x) * kWriteThreads + threadIdx.x;
  if (id >= p.threads) return;
  const int columns = p.heads * kVpr;
  const int window = p.threads <= 0xffffffffLL ? static_cast<int>(static_cast<unsigned>(id) / columns)
                                               : static_cast<int>(id / columns);
  const int column = static_cast<int>(id - static_cast<long long>(window) * columns);
  const int h = column / kVpr, vec = column % kVpr * 16;
  const char* k_src = p.k_new + h * p.kn_h + vec;
  const char* v_src = p.v_new + h * p.vn_h + vec;
  int t = window * p.window;
  const int t_end = min(p.tokens, t + p.window);
  Place at = place_of(p.slots[t], p.n_slots, p.page_size);
  // a run that began before this window belongs to an earlier one
  if (t > 0 && at.row > 0 && p.slots[t - 1] == p.slots[t] - 1) {
    long long slot = p.slots[t];
    do {
      ++t;
      ++at.row;
      ++slot;
    } while (t < t_end && at.row < p.page_size && p.slots[t] == slot);
    if (t < t_end) at = place_of(p.slots[t], p.n_slots, p.page_size);
  }
  while (t < t_end) {
    if (at.row < 0) {
      if (++t < t_end) at = place_of(p.slots[t], p.n_slots, p.page_size);
      continue;
    }
    char* k_dst = p.k_cache + at.page * p.ks_p + h * p.ks_h + at.row * p.ks_r + vec;
    char* v_dst = p.v_cache + at.page * p.vs_p + h * p.vs_h + at.row * p.vs_r + vec;
    uint4* lo = reinterpret_cast<uint4*>(p.summary + (at.page * p.heads + h) * (2 * 16 * kVpr) + vec);
    uint4* hi = lo + kVpr;
    Ext e;
    if (at.row > 0) {
      const uint4 a = *lo, b = *hi;
      memcpy(e.lo, &a, 16);
      memcpy(e.hi, &b, 16);
    } else {
      e.take(load_once(k_src + t * p.kn_n), true);
    }
    const long long first = p.slots[t] - t;  // slot - token along the run
    const int most = min(p.page_size - at.row, p.tokens - t);
    for (int n = 0;; n += kAhead) {
      uint4 k[kAhead], v[kAhead];
      int m = 0;  // tokens of the run among the next kAhead
#pragma unroll
      for (int i = 0; i < kAhead; ++i) m += m == i && n + i < most && p.slots[t + i] - t - i == first;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (i < m) {
          k[i] = load_once(k_src + (t + i) * p.kn_n);
          v[i] = load_once(v_src + (t + i) * p.vn_n);
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (i < m) {
          *reinterpret_cast<uint4*>(k_dst + i * p.ks_r) = k[i];
          *reinterpret_cast<uint4*>(v_dst + i * p.vs_r) = v[i];
          e.take(k[i], false);
        }
      }
      t += m;
      k_dst += kAhead * p.ks_r;
      v_dst += kAhead * p.vs_r;
      if (m < kAhead) break;
    }
    *lo = pack(e.lo);
    *hi = pack(e.hi);
    if (t < t_end) at = place_of(p.slots[t], p.n_slots, p.page_size);
  }
}

// The same for launches that a thread per column would leave with too few threads: a block for each
// window and head shares out a run's rows over its warps and lanes.  Short runs (decoded tokens)
// go to every kWarps-th head's block, a head to each warp.
template <int kVpr, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, 32 / kWarps) paged_write_few(const __grid_constant__ WriteParams p) {
  constexpr int kRows = 32 / kVpr;  // rows a warp moves at once
  __shared__ Ext of_warp[kWarps][kVpr];
  wait_for_inputs();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = static_cast<int>(blockIdx.x % p.heads), t0 = static_cast<int>(blockIdx.x / p.heads) * p.window;
  const int sub = lane / kVpr, column = lane % kVpr, vec = column * 16;
  // the runs that begin in this window (every warp finds them for itself)
  bool begins = false;
  const int t = t0 + lane;
  if (lane < p.window && t < p.tokens) {
    const long long slot = p.slots[t];
    const Place at = place_of(slot, p.n_slots, p.page_size);
    begins = at.row == 0 || (at.row > 0 && (t == 0 || p.slots[t - 1] != slot - 1));
  }
  for (unsigned todo = __ballot_sync(~0u, begins); todo; todo &= todo - 1) {
    const int tb = t0 + __ffs(todo) - 1;
    const long long slot = p.slots[tb];
    const Place at = place_of(slot, p.n_slots, p.page_size);
    const int most = min(p.page_size - at.row, p.tokens - tb);
    int n = 0;  // the run's length: up to the first token that is not in the next slot
    while (n < most) {
      const unsigned ok = __ballot_sync(~0u, n + lane < most && p.slots[tb + n + lane] == slot + n + lane);
      n += ok == ~0u ? 32 : __ffs(~ok) - 1;
      if (ok != ~0u) break;
    }
    const bool alone = n <= 2 * kRows;  // a warp needs no help
    if (alone && (h % kWarps != 0 || h + warp >= p.heads)) continue;
    const int head = alone ? h + warp : h, first = alone ? 0 : warp * kRows, step = alone ? kRows : kWarps * kRows;
    const char* ks = p.k_new + tb * p.kn_n + head * p.kn_h + vec;
    const char* vs = p.v_new + tb * p.vn_n + head * p.vn_h + vec;
    char* kd = p.k_cache + at.page * p.ks_p + head * p.ks_h + at.row * p.ks_r + vec;
    char* vd = p.v_cache + at.page * p.vs_p + head * p.vs_h + at.row * p.vs_r + vec;
    uint4* lo = reinterpret_cast<uint4*>(p.summary + (at.page * p.heads + head) * (2 * 16 * kVpr) + vec);
    uint4* hi = lo + kVpr;
    const bool writes = sub == 0 && (alone || warp == 0);  // the summary's 16 bytes of this lane
    Ext old;
    if (writes && at.row > 0) {
      const uint4 x = *lo, y = *hi;
      memcpy(old.lo, &x, 16);
      memcpy(old.hi, &y, 16);
    }
    const int r0 = first + sub;
    Ext e;
    e.take(*reinterpret_cast<const uint4*>(ks + (r0 < n ? r0 : 0) * p.kn_n), true);  // any row of the run
#pragma unroll 2
    for (int r = r0; r < n; r += step) {
      const uint4 k = *reinterpret_cast<const uint4*>(ks + r * p.kn_n);
      const uint4 v = *reinterpret_cast<const uint4*>(vs + r * p.vn_n);
      *reinterpret_cast<uint4*>(kd + r * p.ks_r) = k;
      *reinterpret_cast<uint4*>(vd + r * p.vs_r) = v;
      e.take(k, false);
    }
#pragma unroll
    for (int d = kVpr; d < 32; d <<= 1) e.take(e.shuffled(d));
    if (!alone) {
      if (sub == 0) of_warp[warp][column] = e;
      __syncthreads();
#pragma unroll
      for (int w = 1; w < kWarps; ++w)
        if (writes) e.take(of_warp[w][column]);
      __syncthreads();  // of_warp is free for the window's next run
    }
    if (writes) {
      if (at.row > 0) e.take(old);
      *lo = pack(e.lo);
      *hi = pack(e.hi);
    }
  }
}

template <int kVpr>
cudaError_t launch(const WriteParams& p, cudaStream_t st) {
  const long long threads = p.summary ? p.threads : static_cast<long long>(p.tokens) * p.heads * kVpr;
  const long long blocks = p.few ? threads : (threads + kWriteThreads - 1) / kWriteThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks)), block(kWriteThreads);
  if (!p.summary) return launch_after(paged_write_rows<kVpr>, grid, block, 0, st, p);
  if (!p.few) return launch_after(paged_write_runs<kVpr>, grid, block, 0, st, p);
  // Four warps for a run of up to 64 rows (24 heads of 128, 64 decoded tokens: 4.0 us, eight warps 5.3),
  // eight for longer ones (8 heads, 300 tokens, pages of 512: 8.8 us, four warps 12.0).
  return p.page_size <= 64 ? launch_after(paged_write_few<kVpr, 4>, grid, dim3(128), 0, st, p)
                           : launch_after(paged_write_few<kVpr, 8>, grid, dim3(256), 0, st, p);
}

}  // namespace

cudaError_t launch_paged_write(const WriteLaunch& a, cudaStream_t st) {
  WriteParams p;
  p.k_new = static_cast<const char*>(a.k_new);
  p.v_new = static_cast<const char*>(a.v_new);
  p.kn_n = a.kn_n * 2;
  p.kn_h = a.kn_h * 2;
  p.vn_n = a.vn_n * 2;
  p.vn_h = a.vn_h * 2;
  p.slots = a.slots;
  p.k_cache = static_cast<char*>(a.k_cache);
  p.v_cache = static_cast<char*>(a.v_cache);
  p.ks_p = a.ks.b_ * 2;
  p.ks_h = a.ks.h_ * 2;
  p.ks_r = a.ks.n_ * 2;
  p.vs_p = a.vs.b_ * 2;
  p.vs_h = a.vs.h_ * 2;
  p.vs_r = a.vs.n_ * 2;
  p.summary = static_cast<char*>(a.summary);
  p.n_slots = static_cast<long long>(a.n_pages) * a.page_size;
  p.tokens = a.tokens;
  p.heads = a.heads;
  p.page_size = a.page_size;
  const long long columns = static_cast<long long>(a.heads) * a.d / 8;
  // Threads that would hold a run each: the two forms meet at 30 to 50 thousand (8 heads of 128, pages
  // of 64: 18432 tokens; at 300 tokens the block form takes 5 us, the other 16; at 27280, 51 and 44).
  // Runs of at most 16 tokens are short enough for one thread at any size.
  p.few = a.summary && a.page_size > 16 && a.tokens * columns / a.page_size < 32768;
  // A window per token (and head) where there are few, longer ones where every SM has work anyway.
  p.window = 1;
  if (p.few)
    while (p.window < 32 && static_cast<long long>(a.tokens) * a.heads > 2048LL * p.window) p.window *= 2;
  else
    while (p.window < 16 && a.tokens * columns > 65536LL * p.window) p.window *= 2;
  p.threads = (static_cast<long long>(a.tokens) + p.window - 1) / p.window * (p.few ? a.heads : columns);
  return a.d == 64 ? launch<8>(p, st) : launch<16>(p, st);
}

}  // namespace ditattn
