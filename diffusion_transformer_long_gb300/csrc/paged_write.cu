// Keys and values of new tokens into their slots of the paged caches, and the touched pages'
// summaries (per channel minimum and maximum of the keys).
//
// A copy of T * H rows of 2 D bytes twice over: bound by HBM for long prefills, by latency
// for a decode step.  Without a summary every (token, head) row stands alone.  With one, a
// page's extremes need all its new rows together and no atomics: the tokens of a page follow
// each other, so each maximal run of consecutive slots in one page has exactly one owner, the
// warp in whose window of tokens it begins, which copies the run's rows of one head, keeps the
// running extremes in registers and merges them with the page's earlier summary (or starts it
// anew, where the run holds row 0).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "paged_device.cuh"
#include "paged_launch.h"

namespace ditattn {
namespace {

constexpr int kWriteThreads = 256;

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
  long long warps;  // with a summary: windows * heads
  int tokens, heads, page_size, window;
};

// kVpr: 16-byte vectors per row.  One thread per vector of a (token, head) row.
template <int kVpr>
__global__ void __launch_bounds__(kWriteThreads) paged_write_rows(const __grid_constant__ WriteParams p) {
  launch_dependents();
  wait_for_inputs();
  const long long i = static_cast<long long>(blockIdx.x) * kWriteThreads + threadIdx.x;
  const long long row = i / kVpr;
  const int t = static_cast<int>(row / p.heads), h = static_cast<int>(row - static_cast<long long>(t) * p.heads);
  if (t >= p.tokens) return;
  const int vec = static_cast<int>(i % kVpr) * 16;
  const long long slot = p.slots[t];
  if (slot < 0 || slot >= p.n_slots) return;
  const long long page = slot / p.page_size, r = slot - page * p.page_size;
  const uint4 k = __ldcs(reinterpret_cast<const uint4*>(p.k_new + t * p.kn_n + h * p.kn_h + vec));
  const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p.v_new + t * p.vn_n + h * p.vn_h + vec));
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

template <int kVpr>
__global__ void __launch_bounds__(kWriteThreads, 4) paged_write_runs(const __grid_constant__ WriteParams p) {
  launch_dependents();
  wait_for_inputs();
  constexpr int kRows = 32 / kVpr;  // rows a warp moves at once
  const long long w = (static_cast<long long>(blockIdx.x) * kWriteThreads + threadIdx.x) >> 5;
  if (w >= p.warps) return;
  const int lane = threadIdx.x & 31;
  const int h = static_cast<int>(w % p.heads);
  const int t0 = static_cast<int>(w / p.heads) * p.window;
  const int sub = lane / kVpr, vec = (lane % kVpr) * 16;
  // the runs that begin in this window
  bool begins = false;
  const int t = t0 + lane;
  if (lane < p.window && t < p.tokens) {
    const long long slot = p.slots[t];
    if (slot >= 0 && slot < p.n_slots)
      begins = t == 0 || p.slots[t - 1] != slot - 1 || slot % p.page_size == 0;
  }
  for (unsigned todo = __ballot_sync(~0u, begins); todo; todo &= todo - 1) {
    const int tb = t0 + __ffs(todo) - 1;
    const long long slot = p.slots[tb];
    const long long page = slot / p.page_size;
    const int r0 = static_cast<int>(slot - page * p.page_size);
    const int most = min(p.page_size - r0, p.tokens - tb);
    int n = 0;  // the run's length: up to the first token that is not in the next slot
    while (n < most) {
      const unsigned ok = __ballot_sync(~0u, n + lane < most && p.slots[tb + n + lane] == slot + n + lane);
      n += ok == ~0u ? 32 : __ffs(~ok) - 1;
      if (ok != ~0u) break;
    }
    const char* ks = p.k_new + tb * p.kn_n + h * p.kn_h + vec;
    const char* vs = p.v_new + tb * p.vn_n + h * p.vn_h + vec;
    char* kd = p.k_cache + page * p.ks_p + h * p.ks_h + r0 * p.ks_r + vec;
    char* vd = p.v_cache + page * p.vs_p + h * p.vs_h + r0 * p.vs_r + vec;
    Ext e;
    // row sub of the run, or (a run shorter than a warp's rows) row 0 again: every lane
    // starts from a row of the run
    {
      const uint4 k = *reinterpret_cast<const uint4*>(ks + (sub < n ? sub : 0) * p.kn_n);
      e.take(k, true);
    }
#pragma unroll 2
    for (int r = sub; r < n; r += kRows) {
      const uint4 k = *reinterpret_cast<const uint4*>(ks + r * p.kn_n);
      const uint4 v = *reinterpret_cast<const uint4*>(vs + r * p.vn_n);
      *reinterpret_cast<uint4*>(kd + r * p.ks_r) = k;
      *reinterpret_cast<uint4*>(vd + r * p.vs_r) = v;
      e.take(k, false);
    }
#pragma unroll
    for (int d = kVpr; d < 32; d <<= 1) e.take(e.shuffled(d));
    if (sub == 0) {
      uint4* lo = reinterpret_cast<uint4*>(p.summary + (page * p.heads + h) * (2 * 16 * kVpr) + vec);
      uint4* hi = lo + kVpr;
      if (r0 > 0) {
        Ext old;
        const uint4 a = *lo, b = *hi;
        memcpy(old.lo, &a, 16);
        memcpy(old.hi, &b, 16);
        e.take(old);
      }
      *lo = pack(e.lo);
      *hi = pack(e.hi);
    }
  }
}

template <int kVpr>
cudaError_t launch(const WriteParams& p, cudaStream_t st) {
  const long long threads = p.summary ? p.warps * 32 : static_cast<long long>(p.tokens) * p.heads * kVpr;
  const long long blocks = (threads + kWriteThreads - 1) / kWriteThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks));
  return p.summary ? launch_after(paged_write_runs<kVpr>, grid, dim3(kWriteThreads), 0, st, p)
                   : launch_after(paged_write_rows<kVpr>, grid, dim3(kWriteThreads), 0, st, p);
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
  p.window = 1;
  while (p.window < 32 && static_cast<long long>(a.tokens) * a.heads > 16384LL * p.window) p.window *= 2;
  p.warps = (static_cast<long long>(a.tokens) + p.window - 1) / p.window * a.heads;
  return a.d == 64 ? launch<8>(p, st) : launch<16>(p, st);
}

}  // namespace ditattn
