// The attention weight that each page has drawn, brought up to date by a step's queries.
//
//   mass[page, h] = (0 where the page's first key is new, else mass[page, h])
//                   + sum over the page's keys j, the last `window` new tokens t that see them, the heads of h's
//                     group: exp(scale q_t . k_j - lse_t)
// The keys are read once for all rows (tokens x heads of a group) and no values are: half the attention's bytes.
//
// Up to 16 rows are bound by HBM (48 requests of 0 to 4608 keys, 24 heads on 8: 44 us, 5.2 TB/s): scores S = K Q^T on
// mma.sync m16n8k16, keys as rows.  A product's sum over channels may take them in any order, so that a lane's operands
// are 16 neighbouring bytes of two keys, read straight from the cache into registers, and of a query row: no staging,
// and every warp walks over runs of pages by itself.  More rows are multiplied on tcgen05 (mma.sync in blocks
// that shared the rows: 2 x 75600 keys, 40 heads on 8, 16 tokens: 107 us, 230 TFLOP/s, near that instruction's rate; now
// 54).
//
// The lanes' sums meet by shuffles in a fixed order, and a page is written by one warp or block: no atomics in a sum, equal
// calls give equal bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <mutex>

#include "attn_host.cuh"
#include "paged_device.cuh"
#include "paged_maps.cuh"
#include "paged_launch.h"
#include "sm103_ptx.cuh"

namespace ditattn {
namespace {

constexpr int kWarps = 8;
constexpr int kTile = 16;      // keys of an mma.sync product
constexpr int kFewRows = 16;   // up to so many rows a warp takes a run by itself
constexpr int kFewKeys = 256;  // keys of such a run (or a page's)

struct MassParams {
  CUtensorMap tm_q, tm_k;  // many rows: boxes of chunk_tokens tokens, and of box_rows rows of a page
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
  int run_pages;  // pages of a run
  int chunk_tokens, box_rows;
  int* status;
  long long wait_limit;
  int stall;
  float scale_log2;
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

// ---------------------------------------------------------------- many rows

constexpr int kTileN = 128;      // keys of a tile: rows of the product, so that a thread has one key's scores
constexpr int kCols = 256;       // (token, head) rows at once: its columns
constexpr int kRing = 4;         // key tiles in shared memory
constexpr int kManyThreads = 384;
constexpr int kEpilogue0 = 4;    // warps 4-7 and 8-11: a tensor-memory buffer each
constexpr int kRunTiles = 32;    // a run's tiles, at most: 256 pieces of 16 keys
constexpr int kRunCost = 256;    // what a run costs beside its keys, in keys (1.5 us)

template <int D>
struct ManySmem {
  static constexpr uint32_t kRegion = 128 * 128;             // 128 rows of one 64-channel block
  static constexpr uint32_t kTileBytes = kTileN * D * 2;
  static constexpr uint32_t kQRegion = kCols * 128;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + kCols * D * 2;
  static constexpr uint32_t kBars = kK + kRing * kTileBytes;
  static constexpr int bQFull = 0, bQEmpty = 1, bKFull = 2, bKEmpty = bKFull + kRing, bDFull = bKEmpty + kRing,
                       bDEmpty = bDFull + 2, bBoth = bDEmpty + 2, bDrain = bBoth + 1, kNumBars = bDrain + 1;
  static constexpr uint32_t kTmem = kBars + kNumBars * 8;
  static constexpr uint32_t kAbort = kTmem + 4;
  static constexpr uint32_t kLse = (kAbort + 4 + 15) & ~15u;        // [2][256] base-2 lse
  static constexpr uint32_t kLimit = kLse + 2 * kCols * 4;          // [2][256] keys that the row sees
  static constexpr uint32_t kPieces = kLimit + 2 * kCols * 4;       // [2][128] sums of 16 keys
  static constexpr uint32_t kLeast = kPieces + 2 * kRunTiles * 8 * 4;  // [2]
  static constexpr uint32_t kBytes = kLeast + 8 + 1024;
  static_assert(kBytes <= 232448, "shared memory budget");
};

__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, uint32_t abort_flag, long long limit) {
  if (ptx::mbar_test_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!ptx::mbar_try_wait(bar, parity)) {
    int stop;
    asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(stop) : "r"(abort_flag) : "memory");
    if (stop || clock64() - t0 > limit) return false;
  }
  return true;
}
__device__ __forceinline__ void raise_abort(const MassParams& p, uint32_t abort_flag) {
  asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(abort_flag), "r"(1) : "memory");
  atomicOr(p.status, kStatusTimeout);
}

// A block's run, which every role's warps find for themselves: some pages of one request, for one key/value head.
struct Run {
  int b = 0;
  long long base = 0;  // runs of the requests before b
  Request rq;
  int h, first, pages, keys, tiles, rows, chunks;  // first page, pages; keys in them; rows; column blocks
  __device__ __forceinline__ bool find(const MassParams& p, long long run, int lane) {
    seek(p, run, b, base, lane);
    if (b >= p.batch) return false;
    rq.load(p, b);
    const int runs = rq.runs(p);
    h = static_cast<int>((run - base) / runs);
    first = static_cast<int>((run - base) - static_cast<long long>(h) * runs) * p.run_pages;
    pages = min(p.run_pages, rq.pages(p) - first);
    keys = min(pages * p.page_size, rq.len - first * p.page_size);
    tiles = (keys + kTileN - 1) / kTileN;
    const int w = p.window > 0 ? min(rq.n, p.window) : rq.n;
    rows = w;  // tokens
    chunks = (w + p.chunk_tokens - 1) / p.chunk_tokens;
    return true;
  }
  __device__ __forceinline__ int token0() const { return rq.n - rows; }  // the first observing one
  __device__ __forceinline__ int tokens(const MassParams& p, int chunk) const {
    return min(p.chunk_tokens, rows - chunk * p.chunk_tokens);
  }
};

// The weights of 16 columns for the thread's key: scores u, the columns' lse and limits in shared memory.
__device__ __forceinline__ float sum16(const uint32_t (&u)[16], float scale, uint32_t lse, uint32_t limit, int key,
                                       bool whole) {
  float sum[4] = {};
#pragma unroll
  for (int c = 0; c < 16; c += 4) {
    float m[4];
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(m[0]), "=f"(m[1]), "=f"(m[2]), "=f"(m[3])
                 : "r"(lse + 4 * c)
                 : "memory");
    float e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = ptx::ex2_approx(fmaf(__uint_as_float(u[c + i]), scale, -m[i]));
    if (!whole) {
      int lim[4];
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(lim[0]), "=r"(lim[1]), "=r"(lim[2]), "=r"(lim[3])
                   : "r"(limit + 4 * c)
                   : "memory");
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (key >= lim[i]) e[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] += e[i];
  }
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

// S^T = K Q^T on tcgen05, keys as rows, so that a thread of the epilogue has a key's scores for all columns and sums
// their weights without a word to its neighbours.  One warp copies Q and the key tiles page by page, one thread
// multiplies, two warpgroups take the tiles in turn out of two tensor-memory buffers.
template <int D>
__global__ void __launch_bounds__(kManyThreads, 1) paged_mass_many_kernel(const __grid_constant__ MassParams p) {
  using S = ManySmem<D>;
  constexpr int kRegions = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = ptx::smem_addr(smem);
  const uint32_t abort_flag = sbase + S::kAbort;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  auto bar = [&](int i) { return sbase + S::kBars + 8u * i; };
  auto wait = [&](int i, uint32_t parity) { return wait_or_abort(bar(i), parity, abort_flag, p.wait_limit); };
  // (lane 0 waits for its warp)
  auto wait_warp = [&](int i, uint32_t parity) {
    bool done = true;
    if (lane == 0) done = wait(i, parity);
    return __shfl_sync(~0u, done, 0) != 0;
  };

  if (threadIdx.x == 0) {
    ptx::mbar_init(bar(S::bQFull), 1);
    ptx::mbar_init(bar(S::bQEmpty), 1);
    for (int s = 0; s < kRing; ++s) {
      ptx::mbar_init(bar(S::bKFull + s), 1);
      ptx::mbar_init(bar(S::bKEmpty + s), 1);
    }
    for (int e = 0; e < 2; ++e) {
      ptx::mbar_init(bar(S::bDFull + e), 1);
      ptx::mbar_init(bar(S::bDEmpty + e), 128);
    }
    ptx::mbar_init(bar(S::bBoth), 256);
    ptx::mbar_init(bar(S::bDrain), 1);
    *reinterpret_cast<volatile int*>(smem + S::kAbort) = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(sbase + S::kTmem, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + S::kTmem);
  wait_for_inputs_and_copies();

  Run r;
  bool ok = true;
  if (warp == 0) {
    const int boxes = kTileN / p.box_rows, box = lane % boxes, block = lane / boxes;
    const uint32_t q_bytes = static_cast<uint32_t>(p.group * p.chunk_tokens) * 128 * kRegions;
    int it = 0, loads = 0;  // tiles, Q loads
    for (long long run = blockIdx.x; ok && r.find(p, run, lane); run += gridDim.x) {
      const int* const row = p.table + r.b * p.table_stride + r.first;
      for (int c = 0; ok && c < r.chunks; ++c) {
        if (!(ok = wait_warp(S::bQEmpty, (loads & 1) ^ 1))) break;
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(bar(S::bQFull), q_bytes);
          for (int x = 0; x < kRegions; ++x)
            ptx::tma_load_4d(sbase + S::kQ + x * S::kQRegion, &p.tm_q, bar(S::bQFull), x * 64, 0,
                             r.rq.row0 + r.token0() + c * p.chunk_tokens, r.h);
        }
        ++loads;
        if (p.stall) break;
        // Each lane looks up the box that it copies, a tile ahead.
        auto look_up = [&](int j, int& page, int& at) {
          const int key = j * kTileN + box * p.box_rows, col = key / p.page_size;
          at = key - col * p.page_size;
          page = p.n_pages;  // past the pool: zeros
          if (col < r.pages) {
            const int x = row[col];
            if (x >= 0 && x < p.n_pages) page = x;
          }
        };
        int page, at, next_page, next_at;
        look_up(0, page, at);
        for (int j = 0; j < r.tiles; ++j, ++it) {
          const int s = it % kRing;
          look_up(j + 1, next_page, next_at);
          if (!(ok = wait_warp(S::bKEmpty + s, ((it / kRing) & 1) ^ 1))) break;
          if (lane == 0) ptx::mbar_arrive_expect_tx(bar(S::bKFull + s), S::kTileBytes);
          if (block < kRegions)
            ptx::tma_load_4d(sbase + S::kK + s * S::kTileBytes + block * S::kRegion + box * p.box_rows * 128, &p.tm_k,
                             bar(S::bKFull + s), block * 64, at, r.h, page);
          page = next_page;
          at = next_at;
        }
      }
      if (p.stall) break;  // test only: the products' first wait for keys will expire
    }
    if (!ok || p.stall) {
      if (!ok && lane == 0) raise_abort(p, abort_flag);
      // Let every copy land before the block can exit.
      if (loads > 0) ptx::mbar_wait(bar(S::bQFull), (loads - 1) & 1, p.wait_limit);
      for (int s = 0; s < kRing; ++s) {
        const int n = (it + kRing - 1 - s) / kRing;  // copies into the slot
        if (n > 0) ptx::mbar_wait(bar(S::bKFull + s), (n - 1) & 1, p.wait_limit);
      }
    }
  } else if (warp == 1) {
    int it = 0, loads = 0;
    for (long long run = blockIdx.x; ok && r.find(p, run, lane); run += gridDim.x) {
      if (lane == 0) {
        for (int c = 0; ok && c < r.chunks; ++c) {
          const int cols = (r.tokens(p, c) * p.group + 15) / 16 * 16;
          const uint32_t idesc = ptx::idesc_bf16_f32(kTileN, cols, false, false);
          if (!(ok = wait(S::bQFull, loads & 1))) break;
          ++loads;
          for (int j = 0; j < r.tiles; ++j, ++it) {
            const int s = it % kRing, e = it & 1;
            if (!(ok = wait(S::bKFull + s, (it / kRing) & 1) && wait(S::bDEmpty + e, ((it / 2) & 1) ^ 1))) break;
            ptx::tc_fence_after();
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
              const uint32_t a = (sbase + S::kK + s * S::kTileBytes + (k / 4) * S::kRegion + (k % 4) * 32) >> 4;
              const uint32_t q = (sbase + S::kQ + (k / 4) * S::kQRegion + (k % 4) * 32) >> 4;
              ptx::mma_bf16_ss(tmem + e * kCols, static_cast<uint64_t>(hi) << 32 | a | 1u << 16,
                               static_cast<uint64_t>(hi) << 32 | q | 1u << 16, idesc, k > 0);
            }
            ptx::mma_commit(bar(S::bDFull + e));
            ptx::mma_commit(bar(S::bKEmpty + s));
          }
          if (ok) ptx::mma_commit(bar(S::bQEmpty));
        }
        if (!ok) {
          raise_abort(p, abort_flag);
          ptx::mma_commit(bar(S::bDrain));
          ptx::mbar_wait(bar(S::bDrain), 0, p.wait_limit);
        }
      }
      ok = __shfl_sync(~0u, ok, 0) != 0;
    }
  } else if (warp >= kEpilogue0) {
    const int e = (warp - kEpilogue0) / 4, quarter = warp & 3, key_row = quarter * 32 + lane;
    const int thread = threadIdx.x - kEpilogue0 * 32;  // of both warpgroups
    const uint32_t tD = tmem + e * kCols + (static_cast<uint32_t>(quarter * 32) << 16);
    uint32_t phase = 0;
    auto both = [&]() {  // both warpgroups meet (a bounded wait)
      ptx::mbar_arrive(bar(S::bBoth));
      ok = __all_sync(~0u, wait(S::bBoth, phase));
      phase ^= 1;
      return ok;
    };
    int it = 0, chunk = 0, count = 0;  // tiles, column blocks, runs
    for (long long run = blockIdx.x; ok && r.find(p, run, lane); run += gridDim.x, ++count) {
      float* const pieces = reinterpret_cast<float*>(smem + S::kPieces) + (count & 1) * kRunTiles * 8;
      if (thread < kRunTiles * 8) pieces[thread] = 0.f;
      for (int c = 0; c < r.chunks; ++c, ++chunk) {
        // Lse and limits of the columns, in turn in two places: who writes them has seen the barrier behind which all
        // were through with the place.
        const uint32_t lse = sbase + S::kLse + (chunk & 1) * kCols * 4, limit = sbase + S::kLimit + (chunk & 1) * kCols * 4;
        int* const least = reinterpret_cast<int*>(smem + S::kLeast) + (chunk & 1);
        const int cols = r.tokens(p, c) * p.group;
        {
          const int tok = thread / p.group;
          int lim = 0;
          float x = 0.f;
          if (thread < cols) {
            const int t = r.token0() + c * p.chunk_tokens + tok;  // of the request's new tokens
            x = p.lse[static_cast<long long>(r.rq.row0 + t) * p.h_q + r.h * p.group + (thread - tok * p.group)] *
                1.4426950408889634f;
            if (x != -INFINITY)  // (else the token saw no key above -inf)
              lim = static_cast<int>(min(max(r.rq.start + t + 1, 0LL), static_cast<long long>(r.rq.len)));
          }
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(lse + 4 * thread), "f"(x) : "memory");
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(limit + 4 * thread), "r"(lim) : "memory");
          if (thread == 0) *least = 0x7fffffff;
          if (!both()) break;
          if (thread < cols) atomicMin(least, lim);
        }
        if (!both()) break;
        const int all = *least;
        for (int j = 0; j < r.tiles; ++j, ++it) {
          if ((it & 1) != e) continue;
          if (!(ok = __all_sync(~0u, wait(S::bDFull + e, (it / 2) & 1)))) break;
          ptx::tc_fence_after();
          const int first = r.first * p.page_size + j * kTileN, key = first + key_row;
          const bool whole = first + kTileN <= min(all, r.first * p.page_size + r.keys);
          float sum = 0.f;
          int x = 0;
          for (; x + 32 <= cols; x += 32) {
            uint32_t u[2][16];
            ptx::tmem_ld16(tD + x, u[0]);
            ptx::tmem_ld16(tD + x + 16, u[1]);
            ptx::tmem_wait_ld();
            sum += sum16(u[0], p.scale_log2, lse + 4 * x, limit + 4 * x, key, whole);
            sum += sum16(u[1], p.scale_log2, lse + 4 * x + 64, limit + 4 * x + 64, key, whole);
          }
          for (; x < cols; x += 16) {  // (columns without a row see no key)
            uint32_t u[16];
            ptx::tmem_ld16(tD + x, u);
            ptx::tmem_wait_ld();
            sum += sum16(u, p.scale_log2, lse + 4 * x, limit + 4 * x, key, whole && x + 16 <= cols);
          }
          ptx::tc_fence_before();
          ptx::mbar_arrive(bar(S::bDEmpty + e));
          if (key_row + j * kTileN >= r.keys) sum = 0.f;
#pragma unroll
          for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
          if ((lane & 15) == 0) pieces[j * 8 + key_row / 16] += sum;
        }
        if (!ok) break;
      }
      if (!ok || !both()) break;
      for (int i = thread; i < r.pages; i += 256) {
        const int page = p.table[r.b * p.table_stride + r.first + i];
        if (page < 0 || page >= p.n_pages) continue;
        const long long out = static_cast<long long>(page) * p.h_kv + r.h;
        float sum = static_cast<long long>(r.first + i) * p.page_size >= r.rq.start ? 0.f : p.mass[out];
        for (int k = i * p.page_size / 16; k < (i + 1) * p.page_size / 16; ++k) sum += pieces[k];
        p.out[out] = sum;
      }
    }
    if (!ok) raise_abort(p, abort_flag);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_many(const MassParams& p, cudaStream_t st) {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      e = cudaFuncSetAttribute(paged_mass_many_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               ManySmem<D>::kBytes);
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  return launch_after(paged_mass_many_kernel<D>, dim3(host::sm_count()), dim3(kManyThreads), ManySmem<D>::kBytes, st, p);
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
  p.status = a.status;
  stall_injection(&p.stall, &p.wait_limit);
  const long long rows = std::min(a.cu_new ? a.window > 0 ? a.window : a.tokens : 1, a.tokens) * static_cast<long long>(p.group);
  if (rows <= kFewRows) {
    p.run_pages = std::max(1, kFewKeys / a.page_size);
    const dim3 block(kWarps * 32);
    auto run = [&](auto kernel, int blocks) { return launch_after(kernel, dim3(blocks * host::sm_count()), block, 0, st, p); };
    if (a.d == 64)
      return rows <= 8 ? run(paged_mass_few_kernel<64, 1>, 3) : run(paged_mass_few_kernel<64, 2>, 2);
    return rows <= 8 ? run(paged_mass_few_kernel<128, 1>, 3) : run(paged_mass_few_kernel<128, 2>, 2);
  }
  p.chunk_tokens = std::min(kCols / p.group, a.cu_new ? a.tokens : 1);
  p.box_rows = maps::box_rows(a.page_size);
  if (!maps::encode_queries(&p.tm_q, a.q, a.q_n, a.q_h, a.d, p.group, a.tokens, a.h_kv, p.chunk_tokens) ||
      !maps::encode_rows(&p.tm_k, a.k_cache, a.ks, a.d, a.page_size, a.h_kv, a.n_pages, p.box_rows))
    return cudaErrorInvalidValue;
  // Runs of 512 to 4096 keys, whichever would end first if every request filled its row of the table: longer ones cost
  // less beside their keys, and leave more blocks idle in the last round (L2 flushed; 2 x 75600 keys, 8 heads, runs of
  // 4096, 2048, 1024, 512: 73, 77, 85, 98 us; 27280 keys, 24 heads: 61, 54, 55, 59, and of 1536, by this rule, 48).
  long long best = LLONG_MAX;
  for (int keys = 512; keys <= kRunTiles * kTileN; keys += 512) {
    const int pages = std::max(1, keys / a.page_size);
    const long long runs = static_cast<long long>(a.batch) * a.h_kv * ((a.max_pages + pages - 1) / pages);
    const long long cost = (runs + host::sm_count() - 1) / host::sm_count() * (pages * a.page_size + kRunCost);
    if (cost <= best) {
      best = cost;
      p.run_pages = pages;
    }
  }
  return a.d == 64 ? launch_many<64>(p, st) : launch_many<128>(p, st);
}

}  // namespace ditattn
