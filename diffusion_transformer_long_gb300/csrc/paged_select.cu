// The pages whose keys can score highest for one query token of each request:
//   score_i = max_h sum_d max(q_hd lo_id, q_hd hi_id)
// over the query heads h of a key/value head's group; listed are the newest page and the
// top_k - 1 others with the highest scores, ties to the lower index, by the scores in 64 bits.
//
// Scoring.  max(q lo, q hi) = max(q, 0) hi + min(q, 0) lo for lo <= hi, so the scores of 16 pages against 8
// heads are a matrix product over 2 D channels, on mma.sync straight from the summaries in
// global memory: a lane's 16-byte loads hold its operands once the channels are renumbered (the
// order of a sum's terms is free).  4 D bytes per page and head: bound by HBM, or by latency.
//
// Choosing.  Products of bf16 are exact in 32 bits but their sums are not, and two pages at the
// border may differ by less.  A second product, of the magnitudes, bounds a score's error by
// kErr sum |q| |k| =: e.  One block per (request, key/value head) narrows the score of the last
// page in down to a histogram bin; a page more than 2 e above the bin is in, one more than 2 e
// below is out, and those between, a handful, are scored again in 64 bits and ranked.  A score
// that is not finite in 32 bits sends all pages of its row that way.
//
// Measured (in a captured graph): 8 rows of 4725 pages 14 us; 256 rows of up to 853 pages 24 us, of
// which 14 for 56 MB of summaries; 14 rows of up to 427 pages 8 us.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attn_host.cuh"
#include "paged_device.cuh"
#include "paged_launch.h"
#include "sm103_ptx.cuh"

namespace ditattn {
namespace {

constexpr int kScoreWarps = 8;
constexpr int kChunk = 16;          // pages of a warp
constexpr int kPickThreads = 512, kPickWarps = kPickThreads / 32;
constexpr int kBins = 1024;
constexpr int kRanked = kPickThreads;  // pages between that are ranked pair by pair
constexpr int kCached = 8192;       // keys held in shared memory
constexpr int kFewPages = 2048;     // pages of a row that a cluster scores; it holds their 64-bit scores too
static_assert(kFewPages * 4 + kFewPages * 8 <= kCached * 4, "keys and 64-bit scores");
// A 32-bit score is summed in 2 D / 16 <= 16 steps of 16 products and the running sum, each of
// the 17 terms cut to within 2^-23 of the step's largest: at most 16 * 17 * 2^-23 of sum |q| |k|.
constexpr float kErr = 16 * 17 / 8388608.f;
constexpr uint32_t kLowest = 0x007FFFFFu;    // the key of -inf: a page without keys
constexpr uint32_t kInfKey = 0xFF800000u;    // the key of +inf
constexpr uint32_t kUnknown = 0xFFFFFFFFu;   // not finite in 32 bits

struct PickParams {
  SelectLaunch a;
  uint32_t* keys;   // [batch * h_kv][max_pages]: scores, as integers of the same order
  float* bounds;    // [batch * h_kv][chunks]: the largest sum |q| |k| of 16 pages
  unsigned long long* exact;  // [batch * h_kv][max_pages]: 64-bit scores of the pages between, in order
  uint32_t* masks;  // [batch * h_kv][mask_words]: a bit for every page, where shared memory has no room
  int chunks, mask_words;
};

// Unsigned integers in the order of the floating-point numbers (no NaN, no -0).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long key_of(double x) {
  const unsigned long long b = __double_as_longlong(x == 0.0 ? 0.0 : x);  // -0 ties with +0
  return b >> 63 ? ~b : b | 1ull << 63;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t half_of(uint32_t w, bool positive) {
  __nv_bfloat162 x, z = __float2bfloat162_rn(0.f);
  memcpy(&x, &w, 4);
  x = positive ? __hmax2_nan(x, z) : __hmin2_nan(x, z);
  memcpy(&w, &x, 4);
  return w;
}

__device__ __forceinline__ void sort_pair(uint32_t& lo, uint32_t& hi) {
  __nv_bfloat162 x, y;
  memcpy(&x, &lo, 4);
  memcpy(&y, &hi, 4);
  const __nv_bfloat162 least = __hmin2_nan(x, y), most = __hmax2_nan(x, y);
  memcpy(&lo, &least, 4);
  memcpy(&hi, &most, 4);
}
__device__ __forceinline__ void sort_pair(uint4& lo, uint4& hi) {
  sort_pair(lo.x, hi.x);
  sort_pair(lo.y, hi.y);
  sort_pair(lo.z, hi.z);
  sort_pair(lo.w, hi.w);
}

__device__ __forceinline__ int pages_now(const SelectLaunch& a, int b) {
  return pages_of(min(max(0, a.seq_lens[b]), a.max_pages * a.page_size), a.page_size);
}

// A lane's table entry of a warp's chunk.  It is read before the request's length is known, or while
// the chunk before is scored: one latency less in the chain (any entry of the row may be read).
__device__ __forceinline__ int entry_of(const SelectLaunch& a, int b, long long chunk) {
  const long long i = chunk * kChunk + (threadIdx.x & 31);
  return (threadIdx.x & 31) < kChunk && i < a.max_pages ? a.table[b * a.table_stride + i] : -1;
}

// A warp scores 16 pages of one (request, key/value head), the n table columns' from 16 chunk on, of
// whose entries every lane brings its own: store(i, key) gets each one's, by one lane.  Returns the
// largest sum |q| |k|.
template <int D, typename Store>
__device__ __forceinline__ float score_pages(const SelectLaunch& a, int b, int g, int n, int chunk, int entry,
                                             Store store) {
  constexpr int kLoads = 2 * D / 32;  // 64-byte pieces of a page's [lo | hi]
  const int lane = threadIdx.x & 31, j = lane & 3, i0 = chunk * kChunk;
  const int page = i0 + lane < n && entry < a.n_pages ? entry : -1;
  const int p0 = __shfl_sync(~0u, page, lane >> 2), p1 = __shfl_sync(~0u, page, (lane >> 2) + 8);
  uint4 x0[kLoads], x1[kLoads];
  const uint4* s0 = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.summary) +
                                                   (static_cast<long long>(max(p0, 0)) * a.h_kv + g) * 2 * D) + j;
  const uint4* s1 = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.summary) +
                                                   (static_cast<long long>(max(p1, 0)) * a.h_kv + g) * 2 * D) + j;
  const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    x0[i] = p0 >= 0 ? s0[4 * i] : none;
    x1[i] = p1 >= 0 ? s1[4 * i] : none;
  }
  // the smaller value first, whichever half holds it (NaN: both), so that the product below is max(q lo, q hi)
#pragma unroll
  for (int i = 0; i < kLoads / 2; ++i) {
    sort_pair(x0[i], x0[i + kLoads / 2]);
    sort_pair(x1[i], x1[i + kLoads / 2]);
  }
  const int group = a.h_q / a.h_kv;
  float best0 = -INFINITY, best1 = -INFINITY, mag = 0.f;
  bool odd0 = false, odd1 = false;
  for (int h0 = 0; h0 < group; h0 += 8) {
    const int h = h0 + (lane >> 2);
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + b * a.q_b +
                                                    static_cast<long long>(g * group + min(h, group - 1)) * a.q_h) + j;
    float s[4] = {0.f, 0.f, 0.f, 0.f}, m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      // lane j's words of piece i: channels 8 j .. 8 j + 7 of 32, two products of 16
      const bool hi = i >= kLoads / 2;
      uint4 y = q[4 * (i % (kLoads / 2))];
      y.x = half_of(y.x, hi);
      y.y = half_of(y.y, hi);
      y.z = half_of(y.z, hi);
      y.w = half_of(y.w, hi);
      constexpr uint32_t kAbs = 0x7fff7fffu;
      mma16816(s, x0[i].x, x1[i].x, x0[i].y, x1[i].y, y.x, y.y);
      mma16816(s, x0[i].z, x1[i].z, x0[i].w, x1[i].w, y.z, y.w);
      mma16816(m, x0[i].x & kAbs, x1[i].x & kAbs, x0[i].y & kAbs, x1[i].y & kAbs, y.x & kAbs, y.y & kAbs);
      mma16816(m, x0[i].z & kAbs, x1[i].z & kAbs, x0[i].w & kAbs, x1[i].w & kAbs, y.z & kAbs, y.w & kAbs);
    }
    // columns past the group repeat its last head: they change neither maximum
    odd0 |= !(fabsf(s[0]) < INFINITY && fabsf(s[1]) < INFINITY);
    odd1 |= !(fabsf(s[2]) < INFINITY && fabsf(s[3]) < INFINITY);
    best0 = fmaxf(best0, fmaxf(s[0], s[1]));
    best1 = fmaxf(best1, fmaxf(s[2], s[3]));
    mag = fmaxf(fmaxf(mag, fmaxf(m[0], m[1])), fmaxf(m[2], m[3]));
  }
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    best0 = fmaxf(best0, __shfl_xor_sync(~0u, best0, d));
    best1 = fmaxf(best1, __shfl_xor_sync(~0u, best1, d));
    odd0 |= __shfl_xor_sync(~0u, static_cast<int>(odd0), d) != 0;
    odd1 |= __shfl_xor_sync(~0u, static_cast<int>(odd1), d) != 0;
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) mag = fmaxf(mag, __shfl_xor_sync(~0u, mag, d));
  if (j == 0) {
    const int i = i0 + (lane >> 2);
    if (i < n) store(i, p0 < 0 ? kLowest : odd0 ? kUnknown : key_of(best0 + 0.f));
    if (i + 8 < n) store(i + 8, p1 < 0 ? kLowest : odd1 ? kUnknown : key_of(best1 + 0.f));
  }
  return mag;
}

template <int D>
__global__ void __launch_bounds__(kScoreWarps * 32) paged_score_kernel(const __grid_constant__ PickParams p) {
  wait_for_inputs();
  const SelectLaunch& a = p.a;
  const int bg = blockIdx.y + blockIdx.z * gridDim.y;
  if (bg >= a.batch * a.h_kv) return;
  const int b = bg / a.h_kv, g = bg - b * a.h_kv;
  int chunk = blockIdx.x * kScoreWarps + (threadIdx.x >> 5);
  int entry = entry_of(a, b, chunk);
  const int n = pages_now(a, b);
  if (n <= a.top_k) return;  // nothing to choose
  uint32_t* keys = p.keys + static_cast<long long>(bg) * a.max_pages;
  while (chunk * kChunk < n) {
    const int next = chunk + gridDim.x * kScoreWarps, entry2 = entry_of(a, b, next);
    const float mag = score_pages<D>(a, b, g, n, chunk, entry, [&](int i, uint32_t key) { keys[i] = key; });
    if ((threadIdx.x & 31) == 0) p.bounds[static_cast<long long>(bg) * p.chunks + chunk] = mag;
    chunk = next;
    entry = entry2;
  }
}

// Sum over the block; `sm` is free again at the next barrier.
__device__ __forceinline__ int block_sum(int x, int* sm) {
  x = __reduce_add_sync(~0u, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = x;
  __syncthreads();
  return __reduce_add_sync(~0u, (threadIdx.x & 31) < kPickWarps ? sm[threadIdx.x & 31] : 0);
}
// Sum over the lower threads, and over all.
__device__ __forceinline__ int block_below(int x, int* sm, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int up = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(~0u, up, d);
    if (lane >= d) up += y;
  }
  __syncthreads();
  if (lane == 31) sm[warp] = up;
  __syncthreads();
  int w = lane < kPickWarps ? sm[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(~0u, w, d);
    if (lane >= d) w += y;
  }
  all = __shfl_sync(~0u, w, kPickWarps - 1);
  const int before = __shfl_sync(~0u, w, max(warp - 1, 0));
  return up - x + (warp > 0 ? before : 0);
}

// Sum * 2^(e - 54), |sum| < 2^62, rounded to fp64's 53 bits (halves away from zero) and as an integer
// of the same order as the fp64 numbers, by integer arithmetic: an fp64 instruction costs a block 16 clocks a warp.
__device__ __forceinline__ unsigned long long key_of(long long sum, int e) {
  const unsigned long long sign = static_cast<unsigned long long>(sum >> 63);
  const unsigned long long m = (static_cast<unsigned long long>(sum) ^ sign) - sign;
  const int lead = __clzll(m);
  const unsigned long long top = m << (lead & 63);  // its highest bit is bit 63: what goes over is the exponent's last 1
  const unsigned long long bits =
      (static_cast<unsigned long long>(1023 - 54 + 63 - 1 + e - lead) << 52) + (top >> 11) + (top >> 10 & 1);
  return sum == 0 ? 1ull << 63 : bits ^ sign ^ 1ull << 63;
}

// The warp's sum of the lanes' four terms, |t| < 2^(e + 1), -72 <= e < 128, each rounded to a whole number of units of
// 2^(e - 54): in three pieces of 18 bits, whose sums stay in 32.  Adding 1.5 * 2^23 rounds to a whole number (a
// conversion to 64 bits costs as much as an fp64 instruction).
__device__ __forceinline__ long long warp_sum(const float (&t)[4], int e) {
  constexpr float kRound = 12582912.f;
  const float unit = __uint_as_float(static_cast<uint32_t>(18 - e + 127) << 23);
  int p[3] = {0, 0, 0};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float y = t[k] * unit;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const float z = y + kRound;
      p[i] += __float_as_int(z) - __float_as_int(kRound);
      y = (y - (z - kRound)) * 262144.f;  // the rest, exactly
    }
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) p[i] = __reduce_add_sync(~0u, p[i]);
  return static_cast<long long>(p[0]) * (1ll << 36) + static_cast<long long>(p[1]) * (1ll << 18) + p[2];
}

// The 64-bit score of table column i, over heads h_first .. h_end - 1 of the group, as an integer of
// the same order, by one warp: a lane takes two channels in every 64.  A head's sum is of 64-bit
// integers in units of 2^(e - 54), 2^e the power of two in its own largest term (the pages' scales may be far apart):
// each of the up to 128 terms, products exact in 32 bits, is rounded once, to 2^-55 of the largest, so that the
// sum is as good as one in fp64, in any order, and far cheaper: this GPU does two fp64 operations a clock
// and SM.  A term that is not finite in 32 bits, or all of them below 2^-72 but not 0 (near the underflow
// of the products): fp64 after all.
__device__ unsigned long long exact_key(const SelectLaunch& a, int b, int g, int i, int h_first, int h_end) {
  const int lane = threadIdx.x & 31;
  const int page = a.table[b * a.table_stride + i];
  if (page < 0 || page >= a.n_pages) return key_of(-static_cast<double>(INFINITY));  // as a page that scores -inf
  const uint32_t* lo = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.summary) +
                                                         (static_cast<long long>(page) * a.h_kv + g) * 2 * a.d) + lane;
  const uint32_t* hi = lo + a.d / 2;
  const int parts = a.d / 64;
  const uint32_t lo0 = lo[0], hi0 = hi[0], lo1 = parts > 1 ? lo[32] : 0, hi1 = parts > 1 ? hi[32] : 0;
  const float l[4] = {ptx::bf16lo(lo0), ptx::bf16hi(lo0), ptx::bf16lo(lo1), ptx::bf16hi(lo1)};
  const float r[4] = {ptx::bf16lo(hi0), ptx::bf16hi(hi0), ptx::bf16lo(hi1), ptx::bf16hi(hi1)};
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + b * a.q_b + static_cast<long long>(g) * (a.h_q / a.h_kv) * a.q_h;
  const uint32_t* qh = reinterpret_cast<const uint32_t*>(q) + lane;
  const long long q_step = a.q_h / 2;
  auto larger = [](float x, float l, float h) {  // NaN in either product is NaN
    const double u = static_cast<double>(x) * l, v = static_cast<double>(x) * h;
    return u != u ? u : v != v ? v : fmax(u, v);
  };
  unsigned long long best = 0;  // below every score
#pragma unroll 4
  for (int h = h_first; h < h_end; ++h) {
    const uint32_t q0 = qh[h * q_step], q1 = parts > 1 ? qh[h * q_step + 32] : 0;
    const float x[4] = {ptx::bf16lo(q0), ptx::bf16hi(q0), ptx::bf16lo(q1), ptx::bf16hi(q1)};
    float t[4], most = 0.f, odd = 0.f;  // odd: NaN where a product is not finite
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float u = x[k] * l[k], v = x[k] * r[k];
      odd = fmaf(u, 0.f, fmaf(v, 0.f, odd));
      t[k] = fmaxf(u, v);
      most = fmaxf(most, fabsf(t[k]));
    }
    const int e = static_cast<int>(__reduce_max_sync(~0u, odd == 0.f ? __float_as_uint(most) : 0x7f800000u) >> 23) - 127;
    if (e >= -72 && e < 128) {
      best = max(best, key_of(warp_sum(t, e), e));
      continue;
    }
    // all terms 0, none of them a product that underflowed: zeroed keys, or a query of zeros
    bool none = odd == 0.f && most == 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      none &= x[k] == 0.f || ((l[k] == 0.f || x[k] * l[k] != 0.f) && (r[k] == 0.f || x[k] * r[k] != 0.f));
    if (__all_sync(~0u, none)) {
      best = max(best, 1ull << 63);
      continue;
    }
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < 4; ++k) s += larger(x[k], l[k], r[k]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    best = max(best, key_of(s != s ? static_cast<double>(INFINITY) : s));
  }
  return best;
}

struct PickSmem {
  uint32_t cache[kCached];  // the pages' keys
  uint32_t mask[kCached / 32];
  int bins[kBins];
  int between[kRanked];
  unsigned long long ranked[kRanked];
  uint32_t extremes[3][kPickWarps];
  int red[kPickWarps];
  int count, bin_found, bin_above;
};

// Chooses top_k of one row's n > top_k > 1 pages, by a whole block.  kHeld: the keys are in sm.cache
// (the block has met since) and mag_bits is this thread's share of the magnitudes; else both are
// read from the workspace.
template <bool kHeld>
__device__ __forceinline__ void pick_pages(const PickParams& p, PickSmem& sm, int bg, int b, int g, int n, int* out,
                                           uint32_t mag_bits) {
  const SelectLaunch& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t* const cache = sm.cache;
  uint32_t* const mask_sm = sm.mask;
  int* const bins = sm.bins;
  int* const between = sm.between;
  unsigned long long* const ranked = sm.ranked;
  auto& extremes = sm.extremes;
  int* const red = sm.red;
  int &count = sm.count, &bin_found = sm.bin_found, &bin_above = sm.bin_above;
  const int others = n - 1, want = a.top_k - 1;  // 1 <= want < others
  const uint32_t* all_keys = p.keys + static_cast<long long>(bg) * a.max_pages;
  const bool cached = kHeld || others <= kCached;
  uint32_t lo = ~0u, hi = 0;  // magnitudes are >= 0 (or NaN): their bits are in order
#pragma unroll 4
  for (int i = tid; i < others; i += kPickThreads) {
    const uint32_t k = kHeld ? cache[i] : all_keys[i];
    if (!kHeld && cached) cache[i] = k;
    lo = min(lo, k);
    hi = max(hi, k);
  }
  if constexpr (!kHeld)
    for (int i = tid; i < (n + kChunk - 1) / kChunk; i += kPickThreads)
      mag_bits = max(mag_bits, __float_as_uint(p.bounds[static_cast<long long>(bg) * p.chunks + i]));
  lo = __reduce_min_sync(~0u, lo);
  hi = __reduce_max_sync(~0u, hi);
  mag_bits = __reduce_max_sync(~0u, mag_bits);
  if (lane == 0) {
    extremes[0][warp] = lo;
    extremes[1][warp] = hi;
    extremes[2][warp] = mag_bits;
  }
  for (int i = tid; i < kBins; i += kPickThreads) bins[i] = 0;
  __syncthreads();
  lo = __reduce_min_sync(~0u, extremes[0][lane % kPickWarps]);
  hi = __reduce_max_sync(~0u, extremes[1][lane % kPickWarps]);
  const float mag = __uint_as_float(__reduce_max_sync(~0u, extremes[2][lane % kPickWarps]));
  const uint32_t* keys = cached ? cache : all_keys;
  // bit i: page i is in
  uint32_t* mask = cached ? mask_sm : p.masks + static_cast<long long>(bg) * p.mask_words;
  // twice the error (the magnitudes' own sum may be short by as much; 2^-110: terms below 32 bits'
  // range), rounded up; in 32 bits, since every fp64 instruction costs a block 16 clocks a warp
  const float wide = __fmul_ru(2.002f, __fmaf_ru(kErr, mag, 0x1p-110f));
  const bool unknown = hi >= kInfKey || !(mag < INFINITY);
  uint32_t from = 0, to = ~0u;  // pages whose key is above `to` are in, below `from` out
  int above = 0;                // pages above the range [lo, hi]
  int sure;                     // pages above `to`
  for (;;) {
    if (!unknown) {
      // the bin that holds the want-th highest key
      const int shift = max(0, 32 - __clz(hi - lo) - 10);
#pragma unroll 4
      for (int i = tid; i < others; i += kPickThreads) {
        const uint32_t k = keys[i] - lo;
        if (k <= hi - lo) atomicAdd(bins + (k >> shift), 1);
      }
      if (tid == 0) count = 0;
      __syncthreads();
      // thread t holds bins 1023 - 2 t and 1022 - 2 t: sums run from the highest scores down
      const int first = bins[kBins - 1 - 2 * tid], second = bins[kBins - 2 - 2 * tid];
      int all;
      const int over = above + block_below(first + second, red, all);
      if (over < want && over + first + second >= want) {
        const bool in_first = over + first >= want;
        bin_found = in_first ? kBins - 1 - 2 * tid : kBins - 2 - 2 * tid;
        bin_above = in_first ? over : over + first;
      }
      __syncthreads();
      const uint32_t lo2 = lo + (static_cast<uint32_t>(bin_found) << shift);
      hi = min(hi, lo2 + ((1u << shift) - 1));
      lo = lo2;
      above = bin_above;
      from = key_of(__fsub_rd(value_of(lo), wide) + 0.f);
      to = key_of(__fadd_ru(value_of(hi), wide) + 0.f);
    } else {
      if (tid == 0) count = 0;
      __syncthreads();
    }
    // the pages in for sure, and a list of those between
    sure = 0;
#pragma unroll 2
    for (int i = tid; i - lane < others; i += kPickThreads) {
      const uint32_t k = i < others ? keys[i] : 0;
      const unsigned in = __ballot_sync(~0u, i < others && k > to);
      if (lane == 0) mask[i >> 5] = in;
      sure += __popc(in);
      if (i < others && k - from <= to - from) {
        const int x = atomicAdd(&count, 1);
        if (x < kRanked) between[x] = i;
      }
    }
    for (int i = tid; i < kBins; i += kPickThreads) bins[i] = 0;
    sure = block_sum(lane == 0 ? sure : 0, red);
    // all between are in, or a narrower bin would not part them
    if (unknown || count == want - sure || lo == hi || (count <= kRanked && value_of(hi) - value_of(lo) <= wide)) break;
    __syncthreads();
  }
  const int mids = count, rest = want - sure;  // 1 <= rest <= mids
  if (mids <= kRanked) {
    // scored in 64 bits and ranked pair by pair
    if (rest < mids) {
      const int group = a.h_q / a.h_kv;
      if (tid < mids) ranked[tid] = 0;
      __syncthreads();
      for (long long x = warp; x < static_cast<long long>(mids) * group; x += kPickWarps) {
        const int i = static_cast<int>(x / group), h = static_cast<int>(x - static_cast<long long>(i) * group);
        const unsigned long long k = exact_key(a, b, g, between[i], h, h + 1);
        if (lane == 0) atomicMax(ranked + i, k);
      }
      __syncthreads();
    }
    if (tid < mids) {
      const int i = between[tid];
      int better = 0;
      if (rest < mids) {
        const unsigned long long k = ranked[tid];
        for (int x = 0; x < mids; ++x) better += ranked[x] > k || (ranked[x] == k && between[x] < i);
      }
      if (better < rest) atomicOr(mask + (i >> 5), 1u << (i & 31));
    }
  } else if (rest == mids) {
    for (int i = tid; i < others; i += kPickThreads)
      if (keys[i] - from <= to - from) atomicOr(mask + (i >> 5), 1u << (i & 31));
  } else {
    // many alike (or not finite): the border by bisection of the 64-bit keys, ties in order
    unsigned long long* exact = kHeld ? reinterpret_cast<unsigned long long*>(cache + kFewPages)
                                      : p.exact + static_cast<long long>(bg) * a.max_pages;
    for (int i = warp; i < others; i += kPickWarps) {
      if (keys[i] - from > to - from) continue;
      const unsigned long long k = exact_key(a, b, g, i, 0, a.h_q / a.h_kv);
      if (lane == 0) exact[i] = k;
    }
    __syncthreads();
    auto at_least = [&](unsigned long long k) {
      int c = 0;
      for (int i = tid; i < others; i += kPickThreads)
        if (keys[i] - from <= to - from) c += exact[i] >= k;
      return block_sum(c, red);
    };
    unsigned long long border = 0;
    for (int bit = 63; bit >= 0; --bit) {
      const unsigned long long k = border | 1ull << bit;
      if (at_least(k) >= rest) border = k;
    }
    const int higher = border == ~0ull ? 0 : at_least(border + 1);
    __syncthreads();
    if (warp == 0) {
      int ties = rest - higher;  // to take, from the lowest columns up
      for (int i0 = 0; i0 < others; i0 += 32) {
        const int i = i0 + lane;
        const bool mid = i < others && keys[i] - from <= to - from;
        const unsigned long long k = mid ? exact[i] : 0;
        const unsigned tied = __ballot_sync(~0u, mid && k == border);
        const bool takes = mid && (k > border || (k == border && __popc(tied & ((1u << lane) - 1)) < ties));
        const unsigned in = __ballot_sync(~0u, takes);
        if (lane == 0) mask[i0 >> 5] |= in;
        ties -= min(ties, __popc(tied));
      }
    }
  }
  __syncthreads();
  // the columns of the mask's bits, in ascending order
  int done = 0;
  for (int w0 = 0; w0 * 32 < others; w0 += kPickThreads) {
    const int w = w0 + tid;
    uint32_t bits = w * 32 < others ? mask[w] : 0;
    int all;
    int at = done + block_below(__popc(bits), red, all);
    for (; bits; bits &= bits - 1) out[at++] = w * 32 + __ffs(bits) - 1;
    done += all;
  }
  if (tid == 0) out[a.top_k - 1] = n - 1;
}

// The list of a row that has nothing to choose: all its pages, or (top_k = 1) the newest alone.
__device__ __forceinline__ void list_all(const SelectLaunch& a, int n, int* out, int threads) {
  for (int i = threadIdx.x; i < a.top_k; i += threads) out[i] = a.top_k == 1 ? n - 1 : i < n ? i : -1;
}

__global__ void __launch_bounds__(kPickThreads) paged_pick_kernel(const __grid_constant__ PickParams p) {
  __shared__ PickSmem sm;
  wait_for_inputs();
  const SelectLaunch& a = p.a;
  const int bg = blockIdx.x, b = bg / a.h_kv, g = bg - b * a.h_kv;
  const int n = pages_now(a, b);
  int* out = a.selected + static_cast<long long>(bg) * a.top_k;
  if (n <= a.top_k || a.top_k == 1) list_all(a, n, out, kPickThreads);
  else pick_pages<false>(p, sm, bg, b, g, n, out, 0);
}

// Few rows: a cluster of eight blocks scores a row's pages, the keys going straight to the first
// block's shared memory, which then chooses.  One launch, and nothing through the workspace.
constexpr int kSelectCluster = 8;
template <int D>
__global__ void __launch_bounds__(kPickThreads) paged_select_few_kernel(const __grid_constant__ PickParams p) {
  __shared__ PickSmem sm;
  __shared__ uint32_t mags[kSelectCluster * kPickWarps];
  const auto cluster = cooperative_groups::this_cluster();
  cluster.sync();  // the first block's shared memory is there
  const SelectLaunch& a = p.a;
  const int bg = blockIdx.x / kSelectCluster, rank = blockIdx.x % kSelectCluster;
  const int b = bg / a.h_kv, g = bg - b * a.h_kv, warp = threadIdx.x >> 5;
  int chunk = warp * kSelectCluster + rank;
  int entry = entry_of(a, b, chunk);
  const int n = pages_now(a, b);
  int* out = a.selected + static_cast<long long>(bg) * a.top_k;
  if (n <= a.top_k || a.top_k == 1) {
    if (rank == 0) list_all(a, n, out, kPickThreads);
    return;
  }
  uint32_t* keys = cluster.map_shared_rank(sm.cache, 0);
  float mag = 0.f;
  while (chunk * kChunk < n) {
    const int next = chunk + kSelectCluster * kPickWarps, entry2 = entry_of(a, b, next);
    const float x = score_pages<D>(a, b, g, n, chunk, entry, [&](int i, uint32_t key) { keys[i] = key; });
    mag = x > mag || x != x ? x : mag;
    chunk = next;
    entry = entry2;
  }
  if ((threadIdx.x & 31) == 0) cluster.map_shared_rank(mags, 0)[rank * kPickWarps + warp] = __float_as_uint(mag);
  cluster.sync();
  if (rank == 0)
    pick_pages<true>(p, sm, bg, b, g, n, out, threadIdx.x < kSelectCluster * kPickWarps ? mags[threadIdx.x] : 0);
}

size_t aligned256(size_t x) { return (x + 255) / 256 * 256; }
size_t mask_words(int max_pages) { return (static_cast<size_t>(max_pages) + 31) / 32; }

// One block of 512 threads and their registers fits an SM: clusters for all rows at once, or none.
// Against two launches (in a graph; each launch also costs the host 2 us): 8 rows of 500 pages 7.4
// and 8.7 us, of 1705 pages 10.8 and 12.3, of 3000 pages 12.7 and 12.4, of 4725 pages 15.4 and 13.8;
// 16 rows of 3000 pages 15.8 and 14.9, of 4725 pages 23.9 and 19.7.
bool few_rows(size_t rows, int max_pages) {
  return rows * kSelectCluster <= static_cast<size_t>(host::sm_count()) && max_pages <= kFewPages;
}

}  // namespace

// Keys, bounds and 64-bit scores of every (request, key/value head).  Clusters need none.
size_t paged_select_workspace(int batch, int h_kv, int max_pages) {
  if (few_rows(static_cast<size_t>(batch) * h_kv, max_pages)) return 0;
  const size_t rows = static_cast<size_t>(batch) * h_kv, chunks = (static_cast<size_t>(max_pages) + kChunk - 1) / kChunk;
  return aligned256(rows * max_pages * 8) + aligned256(rows * max_pages * 4) + aligned256(rows * chunks * 4) +
         aligned256(rows * mask_words(max_pages) * 4);
}

cudaError_t launch_paged_select(const SelectLaunch& a, cudaStream_t st) {
  PickParams p;
  p.a = a;
  p.chunks = static_cast<int>((static_cast<long long>(a.max_pages) + kChunk - 1) / kChunk);
  const size_t rows = static_cast<size_t>(a.batch) * a.h_kv;
  char* ws = static_cast<char*>(a.workspace);
  p.exact = reinterpret_cast<unsigned long long*>(ws);
  p.keys = reinterpret_cast<uint32_t*>(ws + aligned256(rows * a.max_pages * 8));
  p.bounds = reinterpret_cast<float*>(ws + aligned256(rows * a.max_pages * 8) + aligned256(rows * a.max_pages * 4));
  p.mask_words = static_cast<int>(mask_words(a.max_pages));
  p.masks = reinterpret_cast<uint32_t*>(reinterpret_cast<char*>(p.bounds) + aligned256(rows * p.chunks * 4));
  if (rows > 0x7fffffffu) return cudaErrorInvalidConfiguration;
  if (few_rows(rows, a.max_pages)) {
    const dim3 grid(static_cast<unsigned>(rows * kSelectCluster));
    return a.d == 64 ? launch_after<kSelectCluster>(paged_select_few_kernel<64>, grid, dim3(kPickThreads), 0, st, p)
                     : launch_after<kSelectCluster>(paged_select_few_kernel<128>, grid, dim3(kPickThreads), 0, st, p);
  }
  const unsigned rows_y = static_cast<unsigned>(std::min<size_t>(rows, 32768));
  // A block for every 128 pages that the table has room for, up to 32 an SM: tables are often far wider
  // than the requests are long, and each empty block costs its start.
  const size_t most = std::max<size_t>(1, 32 * static_cast<size_t>(host::sm_count()) / rows);
  const size_t needed = (static_cast<size_t>(p.chunks) + kScoreWarps - 1) / kScoreWarps;
  const dim3 grid(static_cast<unsigned>(std::min(needed, most)), rows_y,
                  static_cast<unsigned>((rows + rows_y - 1) / rows_y));
  cudaError_t e = cudaSuccess;
  if (a.top_k > 1)  // (else the newest page alone is listed, whatever the scores)
    e = a.d == 64 ? launch_after(paged_score_kernel<64>, grid, dim3(kScoreWarps * 32), 0, st, p)
                  : launch_after(paged_score_kernel<128>, grid, dim3(kScoreWarps * 32), 0, st, p);
  return e != cudaSuccess ? e : launch_after(paged_pick_kernel, dim3(static_cast<unsigned>(rows)), dim3(kPickThreads), 0, st, p);
}

}  // namespace ditattn
