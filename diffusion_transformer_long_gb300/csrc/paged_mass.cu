// The attention weight that each page has drawn, brought up to date by a step's queries.
//
//   mass[page, h] = (0 where the page's first key is new, else mass[page, h])
//                   + sum over the page's keys j, the last `window` new tokens t that see them, the heads of h's
//                     group: exp(scale q_t . k_j - lse_t)
// The keys are read once for all rows (tokens x heads of a group) and no values are: half the attention's bytes,
// bound by HBM for a few rows (48 requests of 0 to 4608 keys, 24 heads on 8: %s us, %s TB/s), and towards 128 rows by the
// instructions (2 x 75600 keys, 40 heads on 8, 16 tokens: %s us, %s TB/s).
//
// Scores are S = K Q^T on mma.sync m16n8k16, keys as rows and (token, head) rows as columns, as the decode
// attention has them.  A product's sum over channels may take them in any order, so that a lane's operands are
// 16 neighbouring bytes of two keys, read straight from the cache into registers, and 16 bytes of a query row, from
// shared memory; tiles need no staging.  A block takes a run of one request's pages for one key/value head, its
// warps a page each (or a part of one, of large pages); the lanes' sums meet by shuffles in a fixed order, and every
// page is written by one block: no atomics, equal calls give equal bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "attn_host.cuh"
#include "paged_device.cuh"
#include "paged_launch.h"
#include "sm103_ptx.cuh"

namespace ditattn {
namespace {

constexpr int kWarps = 8;
constexpr int kTile = 16;       // keys of a product
constexpr int kTiles = 2;       // whose loads a warp has in flight
constexpr int kRows = 128;      // (token, head) rows in shared memory at once
constexpr int kSums = 128;      // sums of a run: pages x warps of a page
constexpr int kFewRows = 16;    // up to so many rows a warp takes a run by itself
constexpr int kFewKeys = 256;   // keys of such a run (or a page's)
constexpr int kManyKeys = 1024;  // keys of a block's run

struct MassParams {
  const __nv_bfloat16* q;
  long long q_n, q_h;
  const float* lse;
  const __nv_bfloat16* k;
  Strides ks;
  const int* table;
  long long table_stride;
  const int* seq_lens;
  const int* cu_new;      // or null: token b is request b's
  const int* start_lens;  // or null
  const float* mass;
  float* out;
  int batch, tokens, h_q, h_kv, group, page_size, n_pages, max_len, window;
  int page_warps, run_pages;  // warps of a page, pages of a run
  float scale_log2;
};

template <int D>
struct Smem {
  static constexpr int kQ = 0;                        // [rows / 8][D / 32][32 lanes] 16 bytes
  static constexpr int kLse = kQ + kRows * D * 2;     // per row: base-2 lse, then the keys that it sees
  static constexpr int kLimit = kLse + kRows * 4;
  static constexpr int kSum = kLimit + kRows * 4;
  static constexpr int kBytes = kSum + kSums * 4;
};

struct Request {
  int row0, n, len;
  long long start;
  __device__ __forceinline__ void load(const MassParams& p, int b) {
    if (p.cu_new) {
      row0 = min(max(p.cu_new[b], 0), p.tokens);
      n = max(0, min(max(p.cu_new[b + 1], 0), p.tokens) - row0);
    } else {
      row0 = b;
      n = 1;
    }
    len = min(max(p.seq_lens[b], 0), p.max_len);
    start = p.start_lens ? p.start_lens[b] : static_cast<long long>(len) - n;
  }
  __device__ __forceinline__ int pages(const MassParams& p) const { return n > 0 ? pages_of(len, p.page_size) : 0; }
  __device__ __forceinline__ int runs(const MassParams& p) const {
    return (pages(p) + p.run_pages - 1) / p.run_pages;
  }
};

// The request that holds run `run`, from request b on, before which there are `base` runs; b = batch: none does.
__device__ __forceinline__ void seek(const MassParams& p, long long run, int& b, long long& base, int lane) {
  Request rq;
  for (; b < p.batch; b += 32) {
    long long mine = 0;
    if (b + lane < p.batch) {
      rq.load(p, b + lane);
      mine = static_cast<long long>(rq.runs(p)) * p.h_kv;
    }
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += y;
    }
    const unsigned past = __ballot_sync(~0u, base + upto > run);
    if (past) {
      const int l = __ffs(past) - 1;
      base += __shfl_sync(~0u, upto - mine, l);
      b += l;
      return;
    }
    base += __shfl_sync(~0u, upto, 31);
  }
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The sum of a lane's four weights of a tile's keys (first, at rows g and g + 8) and two (token, head) rows, whose base-2
// lse and limits are given; `all`: keys that every row sees.
__device__ __forceinline__ float weights(const float (&d)[4], float scale, float2 lse, int first, int g, int all,
                                         const int* limit) {
  float e[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) e[c] = ptx::ex2_approx(fmaf(d[c], scale, c & 1 ? -lse.y : -lse.x));
  if (first + kTile > all) {
    const int2 lim = *reinterpret_cast<const int2*>(limit);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (first + g + (c & 2 ? 8 : 0) >= (c & 1 ? lim.y : lim.x)) e[c] = 0.f;
  }
  return (e[0] + e[1]) + (e[2] + e[3]);
}

// Many rows: a block for each run.
template <int D>
__global__ void __launch_bounds__(kWarps * 32, 2) paged_mass_kernel(const __grid_constant__ MassParams p) {
  using S = Smem<D>;
  constexpr int kPieces = D / 32;  // 16-byte pieces of a lane and row
  extern __shared__ __align__(16) unsigned char smem[];
  uint4* const qs = reinterpret_cast<uint4*>(smem + S::kQ);
  float* const lse2 = reinterpret_cast<float*>(smem + S::kLse);
  int* const limit = reinterpret_cast<int*>(smem + S::kLimit);
  float* const sums = reinterpret_cast<float*>(smem + S::kSum);
  __shared__ int least;  // keys that all rows in shared memory see (0 where a row takes no part)
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  wait_for_inputs();

  int b = 0;
  long long base = 0;  // runs of the requests before b
  for (long long run = blockIdx.x;; run += gridDim.x) {
    Request rq;
    seek(p, run, b, base, lane);
    if (b >= p.batch) return;
    rq.load(p, b);
    const int runs = rq.runs(p);
    const int h = static_cast<int>((run - base) / runs), first = static_cast<int>((run - base) - static_cast<long long>(h) * runs) * p.run_pages;
    const int pages = min(p.run_pages, rq.pages(p) - first);
    const int* const row = p.table + b * p.table_stride + first;
    const int w = p.window > 0 ? min(rq.n, p.window) : rq.n;
    const long long rows = static_cast<long long>(w) * p.group;
    const int tiles = p.page_size / kTile;

    // This warp's tiles: of page warp / page_warps + i (kWarps / page_warps) those of its part.
    const int part = warp % p.page_warps;
    for (int i = threadIdx.x; i < kSums; i += kWarps * 32) sums[i] = 0.f;
    for (long long r0 = 0; r0 < rows; r0 += kRows) {
      const int here = static_cast<int>(min(rows - r0, static_cast<long long>(kRows)));
      const int blocks = (here + 7) / 8;
      __syncthreads();  // the rows before are done with
      if (threadIdx.x == 0) least = 0x7fffffff;
      __syncthreads();
      for (int i = threadIdx.x; i < blocks * 8; i += kWarps * 32) {
        int lim = 0;
        float x = 0.f;
        if (i < here) {
          const long long r = r0 + i;
          const int tok = static_cast<int>(r / p.group), head = static_cast<int>(r - static_cast<long long>(tok) * p.group);
          x = p.lse[static_cast<long long>(rq.row0 + rq.n - w + tok) * p.h_q + h * p.group + head] * 1.4426950408889634f;
          // (lse = -inf: the token saw no key above -inf)
          if (x != -INFINITY)
            lim = static_cast<int>(min(max(rq.start + (rq.n - w) + tok + 1, 0LL), static_cast<long long>(rq.len)));
        }
        lse2[i] = x;
        limit[i] = lim;
        atomicMin(&least, lim);
      }
      for (int i = threadIdx.x; i < blocks * kPieces * 32; i += kWarps * 32) {
        const int l = i % 32, piece = i / 32 % kPieces, r = i / 32 / kPieces * 8 + l / 4;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < here) {
          const long long rr = r0 + r;
          const int tok = static_cast<int>(rr / p.group), head = static_cast<int>(rr - static_cast<long long>(tok) * p.group);
          x = *reinterpret_cast<const uint4*>(p.q + (rq.row0 + rq.n - w + tok) * p.q_n + (h * p.group + head) * p.q_h +
                                              8 * (4 * piece + l % 4));
        }
        qs[i] = x;
      }
      __syncthreads();
      const int all = least;

      for (int pg = warp / p.page_warps; pg < pages; pg += kWarps / p.page_warps) {
        const int page = row[pg];
        if (page < 0 || page >= p.n_pages) continue;
        const int key0 = (first + pg) * p.page_size;
        const __nv_bfloat16* const at = p.k + page * p.ks.b_ + h * p.ks.h_ + 8 * t;
        const int live = min(tiles, (rq.len - key0 + kTile - 1) / kTile);  // tiles with keys
        float sum = 0.f;
        for (int i0 = part; i0 < live; i0 += kTiles * p.page_warps) {
          uint4 ka[kTiles][kPieces][2];
#pragma unroll
          for (int i = 0; i < kTiles; ++i) {
            const int tile = i0 + i * p.page_warps;
            if (tile < live) {
#pragma unroll
              for (int s = 0; s < kPieces; ++s)
#pragma unroll
                for (int e = 0; e < 2; ++e) ka[i][s][e] = load_once(at + (tile * kTile + g + 8 * e) * p.ks.n_ + 32 * s);
            }
          }
          // (A query row's operands serve all tiles in flight: read for each, shared memory's rate bounded the window.)
          for (int nb = 0; nb < blocks; ++nb) {
            float d[kTiles][4] = {};
#pragma unroll
            for (int s = 0; s < kPieces; ++s) {
              const uint4 x = qs[(nb * kPieces + s) * 32 + lane];
#pragma unroll
              for (int i = 0; i < kTiles; ++i) {
                mma16816(d[i], ka[i][s][0].x, ka[i][s][1].x, ka[i][s][0].y, ka[i][s][1].y, x.x, x.y);
                mma16816(d[i], ka[i][s][0].z, ka[i][s][1].z, ka[i][s][0].w, ka[i][s][1].w, x.z, x.w);
              }
            }
            const float2 m = *reinterpret_cast<const float2*>(lse2 + nb * 8 + 2 * t);
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
              const int tile = i0 + i * p.page_warps;
              if (tile >= live) break;
              sum += weights(d[i], p.scale_log2, m, key0 + tile * kTile, g, all, limit + nb * 8 + 2 * t);
            }
          }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        if (lane == 0) sums[pg * p.page_warps + part] += sum;
      }
    }
    __syncthreads();
    for (int pg = threadIdx.x; pg < pages; pg += kWarps * 32) {
      const int page = row[pg];
      if (page < 0 || page >= p.n_pages) continue;
      const long long at = static_cast<long long>(page) * p.h_kv + h;
      const bool begun = static_cast<long long>(first + pg) * p.page_size >= rq.start;
      float sum = begun ? 0.f : p.mass[at];
      for (int i = 0; i < p.page_warps; ++i) sum += sums[pg * p.page_warps + i];
      p.out[at] = sum;
    }
    __syncthreads();  // the sums are free
  }
}

// Up to 8 kNb rows (tokens x heads of a group): a warp for each run, the query rows' operands in registers, and each piece
// of a tile's registers filled again as soon as it is used, so that a tile is always in flight.
template <int D, int kNb>
__global__ void __launch_bounds__(kWarps * 32, kNb == 1 ? 3 : 2) paged_mass_few_kernel(const __grid_constant__ MassParams p) {
  constexpr int kPieces = D / 32;
  __shared__ float lse2[kWarps][8 * kNb];
  __shared__ int limit[kWarps][8 * kNb];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  wait_for_inputs();
  int b = 0;
  long long base = 0;
  for (long long run = blockIdx.x * kWarps + warp;; run += gridDim.x * kWarps) {
    seek(p, run, b, base, lane);
    if (b >= p.batch) return;
    Request rq;
    rq.load(p, b);
    const int runs = rq.runs(p);
    const int h = static_cast<int>((run - base) / runs);
    const int first = static_cast<int>((run - base) - static_cast<long long>(h) * runs) * p.run_pages;
    const int pages = min(p.run_pages, rq.pages(p) - first);  // at most 32
    int mine = lane < pages ? p.table[b * p.table_stride + first + lane] : -1;
    if (mine >= p.n_pages) mine = -1;
    const int w = p.window > 0 ? min(rq.n, p.window) : rq.n, rows = w * p.group;
    const int tiles = p.page_size / kTile;
    const int keys = min(pages * p.page_size, rq.len - first * p.page_size);  // of the run
    // The tile that is loaded next: tile `tile` of the run's page `pg`.
    int pg = 0, tile = 0;
    const __nv_bfloat16* at = nullptr;
    auto settle = [&]() {  // on to a page that there is
      for (;; ++pg, tile = 0) {
        if (pg >= pages) return;
        const int page = __shfl_sync(~0u, mine, pg);
        if (page < 0) continue;
        at = p.k + page * p.ks.b_ + h * p.ks.h_ + g * p.ks.n_ + 8 * t;
        return;
      }
    };
    settle();
    uint4 ka[kPieces][2];
    const bool any = pg < pages;
    if (any) {
#pragma unroll
      for (int s = 0; s < kPieces; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) ka[s][e] = load_once(at + 8 * e * p.ks.n_ + 32 * s);
    }
    // The rows: lane r < 8 kNb knows row r's lse and limit; lane (g, t) has row 8 nb + g's pieces.
    int all = 0x7fffffff;
    for (int r = lane; r < 8 * kNb; r += 32) {
      int lim = 0;
      float x = 0.f;
      if (r < rows) {
        const int tok = r / p.group;
        x = p.lse[static_cast<long long>(rq.row0 + rq.n - w + tok) * p.h_q + h * p.group + (r - tok * p.group)] *
            1.4426950408889634f;
        if (x != -INFINITY)  // (else the token saw no key above -inf)
          lim = static_cast<int>(min(max(rq.start + (rq.n - w) + tok + 1, 0LL), static_cast<long long>(rq.len)));
      }
      lse2[warp][r] = x;
      limit[warp][r] = lim;
      all = min(all, lim);
    }
    all = __reduce_min_sync(~0u, all);
    uint4 q[kNb][kPieces];
#pragma unroll
    for (int nb = 0; nb < kNb; ++nb) {
      const int r = 8 * nb + g, tok = r / p.group;
#pragma unroll
      for (int s = 0; s < kPieces; ++s)
        q[nb][s] = r < rows ? *reinterpret_cast<const uint4*>(p.q + (rq.row0 + rq.n - w + tok) * p.q_n +
                                                              (h * p.group + r - tok * p.group) * p.q_h + 8 * (4 * s + t))
                            : make_uint4(0, 0, 0, 0);
    }
    __syncwarp();
    float2 m[kNb];
#pragma unroll
    for (int nb = 0; nb < kNb; ++nb) m[nb] = *reinterpret_cast<const float2*>(&lse2[warp][nb * 8 + 2 * t]);

    float sum = 0.f;
    while (pg < pages) {
      const int now = pg, first_key = pg * p.page_size + tile * kTile;  // in the run
      // The next tile: of this page, if it has more keys, or of the next.
      if (++tile == tiles || first_key + kTile >= keys) {
        ++pg;
        tile = 0;
        settle();
      }
      const bool more = pg < pages;
      const __nv_bfloat16* const next = at + static_cast<long long>(tile) * kTile * p.ks.n_;
      float d[kNb][4] = {};
#pragma unroll
      for (int s = 0; s < kPieces; ++s) {
#pragma unroll
        for (int nb = 0; nb < kNb; ++nb) {
          mma16816(d[nb], ka[s][0].x, ka[s][1].x, ka[s][0].y, ka[s][1].y, q[nb][s].x, q[nb][s].y);
          mma16816(d[nb], ka[s][0].z, ka[s][1].z, ka[s][0].w, ka[s][1].w, q[nb][s].z, q[nb][s].w);
        }
        if (more) {
#pragma unroll
          for (int e = 0; e < 2; ++e) ka[s][e] = load_once(next + 8 * e * p.ks.n_ + 32 * s);
        }
      }
#pragma unroll
      for (int nb = 0; nb < kNb; ++nb)
        sum += weights(d[nb], p.scale_log2, m[nb], first * p.page_size + first_key, g, all, &limit[warp][nb * 8 + 2 * t]);
      if (pg != now) {  // the page's last tile
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        const int page = __shfl_sync(~0u, mine, now);
        if (lane == 0) {
          const long long out = static_cast<long long>(page) * p.h_kv + h;
          const bool begun = static_cast<long long>(first + now) * p.page_size >= rq.start;
          p.out[out] = (begun ? 0.f : p.mass[out]) + sum;
        }
        sum = 0.f;
      }
    }
    __syncwarp();  // the rows' words are free
  }
}

template <int D>
cudaError_t launch(const MassParams& p, cudaStream_t st) {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      e = cudaFuncSetAttribute(paged_mass_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  return launch_after(paged_mass_kernel<D>, dim3(2 * host::sm_count()), dim3(kWarps * 32), Smem<D>::kBytes, st, p);
}

}  // namespace

cudaError_t launch_paged_mass(const MassLaunch& a, cudaStream_t st) {
  MassParams p;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.q_n = a.q_n;
  p.q_h = a.q_h;
  p.lse = a.lse;
  p.k = static_cast<const __nv_bfloat16*>(a.k_cache);
  p.ks = a.ks;
  p.table = a.table;
  p.table_stride = a.table_stride;
  p.seq_lens = a.seq_lens;
  p.cu_new = a.cu_new;
  p.start_lens = a.start_lens;
  p.mass = a.mass;
  p.out = a.mass_out;
  p.batch = a.batch;
  p.tokens = a.tokens;
  p.h_q = a.h_q;
  p.h_kv = a.h_kv;
  p.group = a.h_q / a.h_kv;
  p.page_size = a.page_size;
  p.n_pages = a.n_pages;
  p.max_len = a.max_pages * a.page_size;
  p.window = a.window;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  const long long rows = std::min(a.cu_new ? a.window > 0 ? a.window : a.tokens : 1, a.tokens) * static_cast<long long>(p.group);
  if (rows <= kFewRows) {
    p.page_warps = 1;
    p.run_pages = std::max(1, kFewKeys / a.page_size);
    const dim3 block(kWarps * 32);
    auto run = [&](auto kernel, int blocks) { return launch_after(kernel, dim3(blocks * host::sm_count()), block, 0, st, p); };
    if (a.d == 64)
      return rows <= 8 ? run(paged_mass_few_kernel<64, 1>, 3) : run(paged_mass_few_kernel<64, 2>, 2);
    return rows <= 8 ? run(paged_mass_few_kernel<128, 1>, 3) : run(paged_mass_few_kernel<128, 2>, 2);
  }
  // Pages of more than 64 keys go to several warps.
  p.page_warps = 1;
  while (p.page_warps < kWarps && a.page_size > 64 * p.page_warps) p.page_warps *= 2;
  p.run_pages = std::min(kSums / p.page_warps, std::max(kWarps / p.page_warps, kManyKeys / a.page_size));
  return a.d == 64 ? launch<64>(p, st) : launch<128>(p, st);
}

}  // namespace ditattn
