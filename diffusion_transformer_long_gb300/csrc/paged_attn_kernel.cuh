// The paged attention kernel and the join of its parts (paged_attn.cu: the items dealt out over the
// blocks; paged_attn_few.cu: a cluster for each item).
//
// Attention of one new token of each request over its paged keys and values:
//   s_j = scale q . k_j,  m = max s_j,  l = sum exp(s_j - m),  o = sum exp(s_j - m) v_j / l,
//   lse = m + ln l
// for the H_q / H_kv query heads that share a key/value head at once, each key and value read
// once.  2 H_kv D bytes per key feed at most 4 H_q D operations: bound by HBM.
//
// Measured: 16 requests of 30001 to 75600 keys, 40 heads on 8 of 128: 493 us, 7.0 TB/s; 48 of 0 to
// 4608 keys, 24 heads: 207 us, 6.6 TB/s (a copy's rate here is 6.8); one of 27280 keys: 25 us; four
// of 1 to 1024 keys, 2 heads of 64: 5 us.
//
// Work split.  A unit is 64 keys of one item (request, key/value head, block of query heads).  The
// units of the whole batch, counted from the lengths on the device, and a fixed cost for each item
// are dealt out evenly: each block takes one run of consecutive units, whatever request they belong
// to, so that ragged lengths and a single long request fill the GPU alike.  A run that ends inside
// an item leaves fp32 partials (sum, m, l) in the workspace, at most two per block; a second, small
// launch joins them in the order of the blocks (a fixed order: equal calls give equal bits).
//
// Inside a block every warp works alone: it takes every fourth 16-key tile of the run, keeps
// its own ring of stages that its own lane 0 fills by TMA (one 16 x D box of one page for K and
// one for V, 128-byte swizzle), and its own softmax state; the four states are joined through
// shared memory where an item ends.  No block-wide barrier stands between the loads.  Two stages a
// warp, 128 KB of loads in flight an SM, keep HBM busy; a third made the longest case 4 % slower (a
// longer queue only spreads the blocks' ends).
//
// Arithmetic.  Scores S^T = K Q^T on mma.sync m16n8k16 (keys x heads, 8 to 32 heads), so that a
// column is a query head, padding to 8 heads and not to the 16 rows of an A operand, and the
// running output O^T = V^T P^T has the same columns: a thread holds the statistics of the two
// heads whose outputs it holds.  tcgen05 would need 64 or 128 rows for 1 to 32 heads and the
// scores through tensor memory; at 1 to 32 operations per byte the tensor pipe is idle either
// way.  P goes to bf16 in two parts (fp32 output: three), hi + lo (+ lo2), so that its rounding
// (2^-18, fp32: 2^-27) does not show; each tile's product starts from zero and is added in
// fp32, because the tensor core's own accumulation truncates, and over hundreds of tiles that
// would pull the output towards zero.  The running maximum moves only when a tile exceeds it by
// 2^8 (weights up to 256 cost no precision in fp32), and the row sum is compensated, since
// thousands of like terms in turn would lose 2^-24 of the sum at each.
//
// Few short items (one or a few requests, or few selected pages) have a launch of their own: a
// cluster of eight blocks for each item, which needs neither the scan of the lengths nor the
// second launch, since the blocks' sums meet through distributed shared memory.
#pragma once

#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <type_traits>

#include "paged_device.cuh"
#include "paged_launch.h"
#include "sm103_ptx.cuh"

namespace ditattn {
namespace paged {

constexpr int kWarps = 4;
constexpr int kThreadsPaged = kWarps * 32;
constexpr int kTile = 16;                    // keys of a warp's stage
constexpr int kMaxRows = 32;                 // query heads that a block holds
constexpr int kUnitTiles = kWarps;           // tiles of a unit
constexpr int kItemCost = 2;                 // what an item costs beside its units, in units
constexpr int kMaxBlocks = 512;              // largest grid the workspace serves
constexpr int kCluster = 8;                  // blocks that share an item, where each item has a cluster
constexpr float kSlack = 8.f;                // log2 of the largest weight against the running maximum

struct PagedParams {
  CUtensorMap tm_k, tm_v;
  const __nv_bfloat16* q;
  long long q_b, q_h;
  const int* table;
  long long table_stride;
  const int* seq_lens;
  const int* selected;
  int n_selected;
  void* out;
  float* lse;
  float* part_o;    // [blocks][2][R][D]
  float2* part_ml;  // [blocks][2][R]: (maximum in units of log2, sum)
  int4* meta;       // [blocks]: (request, item of it, parts, 0) of the item to join, parts = 0: none
  int batch, h_q, h_kv, group, head_blocks;  // head_blocks: blocks of R query heads in a group
  int page_size, page_tiles, n_pages, max_len;
  float scale_log2;
  int* status;
  long long wait_limit;
  int stall;
};

template <int D>
struct PagedSmem {
  static constexpr int kBox = kTile * D * 2;           // K or V of one tile
  static constexpr int kStages = 64 * 1024 / (kWarps * 2 * kBox);  // 2 (D = 128) or 4
  static constexpr int kRing = kWarps * kStages * 2 * kBox;
  static constexpr int kJoin = kWarps * 8 * D * 4;     // eight heads' sums of each warp
  static constexpr int kBars = kRing + kJoin;          // mbarriers
  static constexpr int kValid = kBars + kWarps * kStages * 8;
  static constexpr int kMl = kValid + kWarps * kStages * 4;
  static constexpr int kScan = kMl + kWarps * kMaxRows * 8;
  static constexpr int kQ = kScan + 64;                // query fragments, where registers have no room
  static constexpr int bytes(int nb) { return kQ + (nb > 2 ? nb * (D / 16) * 32 * 8 : 0); }
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0,
                                            int c1, int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

// One request's item: the 64-key units of its cached (or listed) keys, at least one, so that a
// request without keys still gets its output written.  Its cost adds what its queries, look-ups and
// joining take (2.3 us, about as long as a block's share of HBM needs for 1.6 units), so that a
// block with many short items is not dealt as many keys as one with a few long ones.
struct Item {
  int len, pages, tiles, units;
  __device__ __forceinline__ int cost() const { return units + kItemCost; }
};
__device__ __forceinline__ Item item_of(const PagedParams& p, int b) {
  Item x;
  x.len = min(max(0, p.seq_lens[b]), p.max_len);
  x.pages = pages_of(x.len, p.page_size);
  x.tiles = p.selected ? min(x.pages, p.n_selected) * p.page_tiles : pages_of(x.len, kTile);
  x.units = max(1, (x.tiles + kUnitTiles - 1) / kUnitTiles);
  return x;
}

// Walks a block's run item by item: units [u0, u1) (none, where the run meets only the item's
// extra cost) of item j of request b.
struct Walk {
  int b, j, c0, u0, u1;  // c0: where the run meets the item, in its cost
  long long left;        // of the run's cost, behind this item
  Item it;
  __device__ __forceinline__ void start(const PagedParams& p, int b_, int j_, int c, long long n) {
    b = b_;
    j = j_;
    it = item_of(p, b);
    c0 = c;
    left = n;
    take();
  }
  __device__ __forceinline__ void take() {
    const int n = static_cast<int>(min(static_cast<long long>(it.cost() - c0), left));
    u0 = min(c0, it.units);
    u1 = min(c0 + n, it.units);
    left -= n;
  }
  __device__ __forceinline__ void next(const PagedParams& p) {
    if (++j == p.h_kv * p.head_blocks) {
      j = 0;
      it = item_of(p, ++b);
    }
    c0 = 0;
    take();
  }
  // Tiles of the segment for one warp: first + 4 i < end.
  __device__ __forceinline__ int first(int warp) const { return u0 * kUnitTiles + warp; }
  __device__ __forceinline__ int end() const { return min(u1 * kUnitTiles, it.tiles); }
};

// One warp's loads, running ahead of its arithmetic over the same sequence of tiles.  The pages of
// up to 32 tiles are looked up at once, a tile a lane, one such batch ahead of the one in use.
template <int D>
struct Producer {
  using S = PagedSmem<D>;
  struct Batch {
    int n, head;     // tiles (0: the run is over), key/value head
    int page, spot;  // the lane's tile: page, first row | keys << 16 (0: no key of it counts)
  };
  Walk w;
  int at;  // tiles of w's segment that are in batches
  Batch now, ahead;
  int i;      // the batch's next tile
  int count;  // tiles issued
  __device__ __forceinline__ Batch look_up(const PagedParams& p, int warp, int lane) {
    Batch x;
    x.n = 0;
    while (w.first(warp) + kUnitTiles * at >= w.end()) {
      if (w.left == 0) return x;
      w.next(p);
      at = 0;
    }
    const int first = w.first(warp) + kUnitTiles * at;
    x.n = min(32, (w.end() - first + kUnitTiles - 1) / kUnitTiles);
    x.head = w.j / p.head_blocks;
    x.page = 0;
    x.spot = 0;
    at += x.n;
    const int t = first + kUnitTiles * lane;
    if (lane < x.n) {
      int col = t / p.page_tiles;
      const int row = (t - col * p.page_tiles) * kTile;
      if (p.selected) col = p.selected[(static_cast<long long>(w.b) * p.h_kv + x.head) * p.n_selected + col];
      if (col >= 0 && col < w.it.pages) {
        x.page = p.table[w.b * p.table_stride + col];
        const int keys = min(kTile, w.it.len - col * p.page_size - row);
        if (keys > 0) x.spot = row | keys << 16;
      }
    }
    return x;
  }
  __device__ __forceinline__ void start(const PagedParams& p, const Walk& first, int warp, int lane) {
    w = first;
    at = i = count = 0;
    now = look_up(p, warp, lane);
  }
  // The first tiles, and only then the look-up of the batch behind theirs.
  __device__ __forceinline__ void begin(const PagedParams& p, uint32_t ring, uint32_t bars, int* valid, int warp,
                                        int lane) {
    for (int s = 0; s < S::kStages && i < now.n; ++s) put(p, ring, bars, valid, lane);
    ahead.n = 0;
    if (now.n) ahead = look_up(p, warp, lane);
    while (count < S::kStages && (i < now.n || ahead.n)) issue(p, ring, bars, valid, warp, lane);
  }
  __device__ __forceinline__ void issue(const PagedParams& p, uint32_t ring, uint32_t bars, int* valid, int warp,
                                        int lane) {
    if (i == now.n) {
      if (ahead.n == 0) return;
      now = ahead;
      i = 0;
      ahead = look_up(p, warp, lane);
    }
    put(p, ring, bars, valid, lane);
  }
  __device__ __forceinline__ void put(const PagedParams& p, uint32_t ring, uint32_t bars, int* valid, int lane) {
    const int page = __shfl_sync(~0u, now.page, i);
    int spot = __shfl_sync(~0u, now.spot, i);
    if (page < 0 || page >= p.n_pages) spot = 0;
    ++i;
    const int stage = count % S::kStages;
    ++count;
    if (lane == 0) {
      const uint32_t bar = bars + stage * 8, dst = ring + stage * 2 * S::kBox;
      valid[stage] = spot >> 16;
      if (spot == 0 || p.stall) {  // nothing to load
        if (!p.stall) ptx::mbar_arrive(bar);
      } else {
        ptx::mbar_arrive_expect_tx(bar, 2 * S::kBox);
        tma_load_5d(dst, &p.tm_k, bar, 0, spot & 0xffff, 0, now.head, page);
        tma_load_5d(dst + S::kBox, &p.tm_v, bar, 0, spot & 0xffff, 0, now.head, page);
      }
    }
  }
};

// x / y of non-negative numbers, in 32 bits where they fit (several times cheaper).
__device__ __forceinline__ long long divided(long long x, long long y) {
  return (x | y) >> 32 ? x / y : static_cast<long long>(static_cast<unsigned>(x) / static_cast<unsigned>(y));
}

// kNb: blocks of eight query heads (R = 8 kNb).  kClusters: a cluster for each item instead of a run
// of units for each block.
template <int D, int kNb, typename OT, bool kClusters>
__global__ void __launch_bounds__(kThreadsPaged, 2) paged_attn_kernel(const __grid_constant__ PagedParams p) {
  using S = PagedSmem<D>;
  constexpr int kSteps = D / 16;
  constexpr int kParts = sizeof(OT) == 4 ? 3 : 2;
  constexpr int R = 8 * kNb;
  constexpr bool kQShared = kNb > 2;  // 32 registers of queries for 16 heads fit beside the output's 64
  extern __shared__ __align__(1024) unsigned char smem[];
  float* join = reinterpret_cast<float*>(smem + S::kRing);
  float2* ml = reinterpret_cast<float2*>(smem + S::kMl);
  long long* scan = reinterpret_cast<long long*>(smem + S::kScan);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = ptx::smem_addr(smem) + warp * S::kStages * 2 * S::kBox;
  const uint32_t bars = ptx::smem_addr(smem + S::kBars) + warp * S::kStages * 8;
  int* valid = reinterpret_cast<int*>(smem + S::kValid) + warp * S::kStages;
  const int items = p.h_kv * p.head_blocks;  // of one request
  if (threadIdx.x == 0) {
    ptx::tma_prefetch_desc(&p.tm_k);
    ptx::tma_prefetch_desc(&p.tm_v);
  }
  if (lane == 0) {
    for (int s = 0; s < S::kStages; ++s) ptx::mbar_init(bars + s * 8, 1);
    ptx::fence_mbar_init();
  }
  __syncwarp();
  wait_for_inputs_and_copies();
  const long long c = blockIdx.x;
  long long total = 0, blocks = 0, run0 = 0;  // blocks with a run, and where this one's begins
  long long share = 0, extra = 0;             // runs: share + 1 each for the first `extra`, share for the others
  Walk seg;
  if constexpr (kClusters) {
    // Block r of a cluster takes the r-th eighth of its item.
    const int item = blockIdx.x / kCluster, r = blockIdx.x % kCluster;
    seg.b = item / items;
    seg.j = item - seg.b * items;
    seg.it = item_of(p, seg.b);
    seg.u0 = seg.c0 = static_cast<int>(static_cast<long long>(seg.it.units) * r / kCluster);
    seg.u1 = static_cast<int>(static_cast<long long>(seg.it.units) * (r + 1) / kCluster);
    seg.left = 0;
  } else {
    // The batch's cost, and where this block's run begins: lane l (of up to 32 requests) or thread t
    // (of a chunk of the requests) sums, and the one that holds the run's beginning finds the request.
    const int per = p.batch <= 32 ? 1 : (p.batch + kThreadsPaged - 1) / kThreadsPaged;
    const int who = p.batch <= 32 ? lane : threadIdx.x;
    const int b0 = min(p.batch, who * per), b1 = min(p.batch, b0 + per);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) sum += item_of(p, b).cost();
    sum *= items;
    long long upto = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(~0u, upto, d);
      if (lane >= d) upto += y;
    }
    if (p.batch <= 32) {
      total = __shfl_sync(~0u, upto, 31);
    } else {
      if (lane == 31) scan[warp] = upto;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) upto += scan[w];
        total += scan[w];
      }
    }
    blocks = min(static_cast<long long>(gridDim.x), total);
    if (c >= blocks) {
      if (threadIdx.x == 0) p.meta[c] = make_int4(0, 0, 0, 0);
      return;
    }
    share = divided(total, blocks);
    extra = total - share * blocks;
    run0 = c * share + min(c, extra);
    const long long run = share + (c < extra);
    const bool holds = run0 < upto && run0 >= upto - sum;
    long long at = upto - sum;
    int b = b0;
    if (p.batch <= 32) {
      b = __ffs(__ballot_sync(~0u, holds)) - 1;
      at = __shfl_sync(~0u, at, b);
    } else {
      __syncthreads();
      if (holds) {
        long long n = static_cast<long long>(item_of(p, b).cost()) * items;
        while (at + n <= run0) {
          at += n;
          n = static_cast<long long>(item_of(p, ++b).cost()) * items;
        }
        scan[0] = b;
        scan[1] = at;
      }
      __syncthreads();
      b = static_cast<int>(scan[0]);
      at = scan[1];
    }
    const int cost = item_of(p, b).cost();
    const int j = static_cast<int>(divided(run0 - at, cost));
    seg.start(p, b, j, static_cast<int>(run0 - at - static_cast<long long>(j) * cost), run);
  }
  Producer<D> load;
  load.start(p, seg, warp, lane);
  load.begin(p, ring, bars, valid, warp, lane);

  // ldmatrix addresses of this lane: row and 16-byte chunk of K (A operand, keys x channels) and
  // of V read transposed (channels x keys); a row is 128 bytes per 64 channels, chunk ^ (row & 7).
  const int r8 = lane & 7, mat = lane >> 3;
  const int k_row = r8 + (mat & 1) * 8, k_chunk = mat >> 1;
  const int v_row = r8 + (mat >> 1) * 8, v_chunk = mat & 1;

  bool dead = false;
  int consumed = 0, landed = 0;  // tiles passed; those whose copies have been waited for
  int4 note = make_int4(0, 0, 0, 0);
  long long pos = run0;  // of c0 in the batch's cost
  // A cluster's blocks leave their sums in the ring, whose copies have all landed, and their (m, l) behind.
  float* mine = reinterpret_cast<float*>(smem);  // [R][D]
  float2* mine_ml = reinterpret_cast<float2*>(smem + R * D * 4);
  if constexpr (kClusters) {
    static_assert(R * D * 4 + R * 8 <= S::kRing, "the ring holds a block's sums");
  }
  uint32_t qf[kQShared ? 1 : kNb][kSteps][2];          // query fragments (B operand, channels x heads)
  uint2* q_sm = reinterpret_cast<uint2*>(smem + S::kQ);  // [nb][step][lane]
  auto load_queries = [&](const Walk& w) {
    const int hk = w.j / p.head_blocks, h0 = (w.j - hk * p.head_blocks) * R;
#pragma unroll
    for (int nb = 0; nb < kNb; ++nb) {
      if (kQShared && nb % kWarps != warp) continue;  // shared: each warp fetches its part
      const int h = h0 + nb * 8 + (lane >> 2);
      const uint32_t* q = reinterpret_cast<const uint32_t*>(
          p.q + w.b * p.q_b + static_cast<long long>(hk * p.group + h) * p.q_h + (lane & 3) * 2);
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const uint2 x = h < p.group ? make_uint2(q[k * 8], q[k * 8 + 4]) : make_uint2(0, 0);
        if constexpr (kQShared) {
          q_sm[(nb * kSteps + k) * 32 + lane] = x;
        } else {
          qf[nb][k][0] = x.x;
          qf[nb][k][1] = x.y;
        }
      }
    }
  };
  // The run's next item with units (false: the run is over); `at` follows its place in the batch's cost.
  auto advance = [&](Walk& w, long long& at) {
    do {
      if (w.left == 0) return false;
      at += w.it.cost() - w.c0;
      w.next(p);
    } while (w.u0 == w.u1);
    return true;
  };
  bool more = seg.u0 < seg.u1 || advance(seg, pos);
  if (more) load_queries(seg);
  while (more) {
    if constexpr (kQShared) __syncthreads();
    const int hk = seg.j / p.head_blocks, h0 = (seg.j - hk * p.head_blocks) * R;
    float o[kSteps][kNb][4];
    float m[kNb][2], l[kNb][2], lc[kNb][2];  // lc: the sum's compensation
#pragma unroll
    for (int nb = 0; nb < kNb; ++nb) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[nb][i] = -INFINITY;
        l[nb][i] = lc[nb][i] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < kSteps; ++k) o[k][nb][0] = o[k][nb][1] = o[k][nb][2] = o[k][nb][3] = 0.f;
    }

    for (int t = seg.first(warp); t < seg.end(); t += kUnitTiles) {
      const int stage = consumed % S::kStages;
      if (!dead && !ptx::mbar_wait(bars + stage * 8, (consumed / S::kStages) & 1, p.wait_limit)) dead = true;
      dead = __any_sync(~0u, dead);
      ++consumed;
      if (!dead) landed = consumed;
      const int keys = dead ? 0 : valid[stage];
      if (keys > 0) {
        const uint32_t kb = ring + stage * 2 * S::kBox, vb = kb + S::kBox;
        if (keys < kTile) {
          // rows past the length may hold anything: their weight is 0, and 0 * NaN is not
          const int n = (kTile - keys) * (D / 8);
          for (int x = lane; x < n; x += 32) {
            const int row = keys + x / (D / 8), ch = x % (D / 8);
            const uint32_t a = vb + (ch >> 3) * (kTile * 128) + row * 128 + (ch & 7) * 16;
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
          }
          __syncwarp();
        }
        float s[kNb][4];
#pragma unroll
        for (int nb = 0; nb < kNb; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t a[4];
          const int ch = (k & 3) * 2 + k_chunk;
          ldsm4(kb + (k >> 2) * (kTile * 128) + k_row * 128 + ((ch ^ (k_row & 7)) << 4), a);
#pragma unroll
          for (int nb = 0; nb < kNb; ++nb) {
            if constexpr (kQShared) {
              const uint2 x = q_sm[(nb * kSteps + k) * 32 + lane];
              const uint32_t b[2] = {x.x, x.y};
              mma16816(s[nb], a, b);
            } else {
              mma16816(s[nb], a, qf[nb][k]);
            }
          }
        }
        const bool in0 = (lane >> 2) < keys, in1 = (lane >> 2) + 8 < keys;
        bool moves = false;
#pragma unroll
        for (int nb = 0; nb < kNb; ++nb) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            s[nb][i] = in0 ? s[nb][i] * p.scale_log2 : -INFINITY;
            s[nb][i + 2] = in1 ? s[nb][i + 2] * p.scale_log2 : -INFINITY;
            moves |= fmaxf(s[nb][i], s[nb][i + 2]) > m[nb][i] + kSlack;
          }
        }
        if (__any_sync(~0u, moves)) {
#pragma unroll
          for (int nb = 0; nb < kNb; ++nb) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float x = fmaxf(m[nb][i], fmaxf(s[nb][i], s[nb][i + 2]));
              x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
              x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
              x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
              const float f = x == -INFINITY ? 1.f : ptx::ex2_approx(m[nb][i] - x);
              m[nb][i] = x;
              l[nb][i] *= f;
              lc[nb][i] *= f;
#pragma unroll
              for (int k = 0; k < kSteps; ++k) {
                o[k][nb][i] *= f;
                o[k][nb][i + 2] *= f;
              }
            }
          }
        }
        uint32_t pf[kParts][kNb][2];  // B operand: keys x heads, P in parts
#pragma unroll
        for (int nb = 0; nb < kNb; ++nb) {
          float w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float base = m[nb][i & 1] == -INFINITY ? 0.f : m[nb][i & 1];
            w[i] = ptx::ex2_approx(s[nb][i] - base);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float y = (w[i] + w[i + 2]) - lc[nb][i];
            const float z = l[nb][i] + y;
            lc[nb][i] = (z - l[nb][i]) - y;
            l[nb][i] = z;
          }
#pragma unroll
          for (int part = 0; part < kParts; ++part) {
            const uint32_t a = ptx::pack_bf16x2(w[0], w[1]), b = ptx::pack_bf16x2(w[2], w[3]);
            pf[part][nb][0] = transposed(a);
            pf[part][nb][1] = transposed(b);
            w[0] -= ptx::bf16lo(a);
            w[1] -= ptx::bf16hi(a);
            w[2] -= ptx::bf16lo(b);
            w[3] -= ptx::bf16hi(b);
          }
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t a[4];
          const int ch = (k & 3) * 2 + v_chunk;
          ldsm4_trans(vb + (k >> 2) * (kTile * 128) + v_row * 128 + ((ch ^ (v_row & 7)) << 4), a);
#pragma unroll
          for (int nb = 0; nb < kNb; ++nb) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int part = kParts - 1; part >= 0; --part) mma16816(d, a, pf[part][nb]);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[k][nb][i] += d[i];
          }
        }
        if (keys < kTile) ptx::fence_proxy_async_smem();  // the zeroed rows, before the next copy
      }
      __syncwarp();
      if (!dead) load.issue(p, ring, bars, valid, warp, lane);
    }

    // The next item's queries are on their way while this one's states are joined.
    Walk next = seg;
    long long next_pos = pos;
    more = advance(next, next_pos);
    if (more && !kQShared) load_queries(next);

    // ---- the four warps' states of this segment, joined: the output, or a part of it
    const bool whole = !kClusters && seg.u0 == 0 && seg.u1 == seg.it.units;
    const int slot = seg.u0 > 0 ? 0 : 1;
#pragma unroll
    for (int nb = 0; nb < kNb; ++nb) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = l[nb][i] - lc[nb][i];
        x += __shfl_xor_sync(~0u, x, 4);
        x += __shfl_xor_sync(~0u, x, 8);
        x += __shfl_xor_sync(~0u, x, 16);
        if (lane < 4) ml[warp * kMaxRows + nb * 8 + lane * 2 + i] = make_float2(m[nb][i], x);
        float* dst = join + (warp * 8 + (lane & 3) * 2 + i) * D;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const int d = k * 16 + (lane >> 2);
          dst[d ^ ((lane & 3) << 3)] = o[k][nb][i];
          dst[(d + 8) ^ ((lane & 3) << 3)] = o[k][nb][i + 2];
        }
      }
      __syncthreads();
      {
        constexpr int kCols = 8 * D / kThreadsPaged;  // channels of a thread: 8 (D = 128) or 4
        const int head = threadIdx.x / (D / kCols), d0 = threadIdx.x % (D / kCols) * kCols;
        const int h = h0 + nb * 8 + head;
        float M = -INFINITY, L = 0.f, f[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * kMaxRows + nb * 8 + head].x);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 x = ml[w * kMaxRows + nb * 8 + head];
          f[w] = M == -INFINITY ? 0.f : ptx::ex2_approx(x.x - M);
          L = fmaf(f[w], x.y, L);
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const long long row = static_cast<long long>(seg.b) * p.h_q + hk * p.group + h;
        const long long part = (c * 2 + slot) * R + nb * 8 + head;
#pragma unroll
        for (int i = 0; i < kCols; i += 4) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float4 y = *reinterpret_cast<const float4*>(join + (w * 8 + head) * D + ((d0 + i) ^ ((head >> 1) << 3)));
            x.x = fmaf(f[w], y.x, x.x);
            x.y = fmaf(f[w], y.y, x.y);
            x.z = fmaf(f[w], y.z, x.z);
            x.w = fmaf(f[w], y.w, x.w);
          }
          if constexpr (kClusters) {
            *reinterpret_cast<float4*>(mine + (nb * 8 + head) * D + d0 + i) = x;
          } else if (!whole) {
            *reinterpret_cast<float4*>(p.part_o + part * D + d0 + i) = x;
          } else if (h < p.group) {
            if (L == 0.f) x = make_float4(0.f, 0.f, 0.f, 0.f);  // (sums of weights 0 and values that are not finite)
            OT* dst = static_cast<OT*>(p.out) + row * D + d0 + i;
            if constexpr (sizeof(OT) == 4)
              *reinterpret_cast<float4*>(dst) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
            else
              *reinterpret_cast<uint2*>(dst) =
                  make_uint2(ptx::pack_bf16x2(x.x * inv, x.y * inv), ptx::pack_bf16x2(x.z * inv, x.w * inv));
          }
        }
        if (d0 == 0) {
          if (kClusters) mine_ml[nb * 8 + head] = make_float2(M, L);
          else if (!whole) p.part_ml[part] = make_float2(M, L);
          else if (p.lse && h < p.group) p.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
        }
      }
      __syncthreads();
    }
    if (!kClusters && !whole && slot == 1) {
      // the item goes on in later blocks: up to the one that holds its last unit
      const long long last = pos - seg.c0 + seg.it.units - 1;
      const long long longer = extra * (share + 1);
      const long long owner = last < longer ? divided(last, share + 1) : extra + divided(last - longer, share);
      note = make_int4(seg.b, seg.j, static_cast<int>(owner - c) + 1, 0);
    }
    if (more && kQShared) load_queries(next);
    seg = next;
    pos = next_pos;
  }
  if constexpr (kClusters) {
    // Every block's sums against their common maximum; block r joins the heads r, r + 8, ..  A maximum of
    // -inf does not mean that there is nothing to join: the fmaxf of scores that are all NaN leaves it there, and
    // the sums are NaN.  A block without units, whose sums were never written, has the sum -1.
    if (seg.u0 == seg.u1 && threadIdx.x < R) mine_ml[threadIdx.x] = make_float2(-INFINITY, -1.f);
    const auto cluster = cooperative_groups::this_cluster();
    cluster.sync();
    const int hk = seg.j / p.head_blocks, h0 = (seg.j - hk * p.head_blocks) * R;
    constexpr int kAtOnce = kThreadsPaged / D;  // heads: 1 (D = 128) or 2
    const int d = threadIdx.x % D;
    for (int head = blockIdx.x % kCluster + threadIdx.x / D * kCluster; head < R && h0 + head < p.group;
         head += kAtOnce * kCluster) {
      float2 y[kCluster];
      float x[kCluster], M = -INFINITY, L = 0.f, sum = 0.f;
#pragma unroll
      for (int r = 0; r < kCluster; ++r) {
        y[r] = cluster.map_shared_rank(mine_ml, r)[head];
        x[r] = cluster.map_shared_rank(mine, r)[head * D + d];
        M = fmaxf(M, y[r].x);
      }
      const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int r = 0; r < kCluster; ++r) {
        if (y[r].y < 0.f) continue;
        const float f = ptx::ex2_approx(y[r].x - base);
        L = fmaf(f, y[r].y, L);
        sum = fmaf(f, x[r], sum);
      }
      const long long row = static_cast<long long>(seg.b) * p.h_q + hk * p.group + h0 + head;
      static_cast<OT*>(p.out)[row * D + d] = static_cast<OT>(L == 0.f ? 0.f : sum / L);
      if (p.lse && d == 0) p.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    }
    cluster.sync();  // no block's sums go before all have been read
  } else if (threadIdx.x == 0) {
    p.meta[c] = note;
  }
  if (dead) {
    if (lane == 0) {
      atomicMax(p.status, 1);
      // leave only when the copies still in flight have landed (or this wait has run out too)
      for (; landed < load.count && !p.stall; ++landed)
        ptx::mbar_wait(bars + landed % S::kStages * 8, (landed / S::kStages) & 1, p.wait_limit);
    }
  }
}

// Joins the parts of the item that begins in block blockIdx.x and ends in a later one: part 0 is
// that block's second, the others are the first of the blocks behind it.  One block of threads
// per item and query head, a thread per channel quad and a quarter (D = 64: an eighth) of the parts.
template <int D, int kNb, typename OT>
__global__ void __launch_bounds__(128) paged_join_kernel(const __grid_constant__ PagedParams p) {
  constexpr int R = 8 * kNb, kQuads = D / 4, kSlices = 128 / kQuads;
  __shared__ float4 acc_sm[kSlices][kQuads];
  __shared__ float2 ml_sm[kSlices];
  wait_for_inputs();
  const int4 note = p.meta[blockIdx.x];
  const int n = note.z;
  if (n == 0) return;
  const int hk = note.y / p.head_blocks, head = blockIdx.y;
  const int h = (note.y - hk * p.head_blocks) * R + head;
  if (h >= p.group) return;
  auto at = [&](int i) { return (static_cast<long long>(blockIdx.x + i) * 2 + (i == 0)) * R + head; };
  // each slice runs through its parts once, against its own running maximum; then the slices meet
  const int quad = threadIdx.x % kQuads, slice = threadIdx.x / kQuads;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, L = 0.f;
  auto add = [&](float m, float l, const float4& y) {
    // a part with the maximum -inf weighs nothing, but NaN sums (all its scores were NaN) have to show
    const float top = fmaxf(M, m), base = top == -INFINITY ? 0.f : top;
    const float f = ptx::ex2_approx(M - base), w = ptx::ex2_approx(m - base);
    M = top;
    L = fmaf(w, l, L * f);
    acc.x = fmaf(w, y.x, acc.x * f);
    acc.y = fmaf(w, y.y, acc.y * f);
    acc.z = fmaf(w, y.z, acc.z * f);
    acc.w = fmaf(w, y.w, acc.w * f);
  };
  constexpr int kAhead = 8;
  for (int i0 = slice; i0 < n; i0 += kSlices * kAhead) {
    float2 x[kAhead];
    float4 y[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + k * kSlices;
      if (i < n) {
        x[k] = p.part_ml[at(i)];
        y[k] = *reinterpret_cast<const float4*>(p.part_o + at(i) * D + quad * 4);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i0 + k * kSlices < n) add(x[k].x, x[k].y, y[k]);
  }
  acc_sm[slice][quad] = acc;
  if (quad == 0) ml_sm[slice] = make_float2(M, L);
  __syncthreads();
  if (slice != 0) return;
  for (int s = 1; s < min(n, kSlices); ++s) add(ml_sm[s].x, ml_sm[s].y, acc_sm[s][quad]);
  const float inv = L == 0.f ? 0.f : 1.f / L;
  if (L == 0.f) acc = make_float4(0.f, 0.f, 0.f, 0.f);  // (sums of weights 0 and values that are not finite)
  const long long row = static_cast<long long>(note.x) * p.h_q + hk * p.group + h;
  OT* dst = static_cast<OT*>(p.out) + row * D + quad * 4;
  if constexpr (sizeof(OT) == 4)
    *reinterpret_cast<float4*>(dst) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  else
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(ptx::pack_bf16x2(acc.x * inv, acc.y * inv), ptx::pack_bf16x2(acc.z * inv, acc.w * inv));
  if (p.lse && quad == 0) p.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// Sets a kernel's shared-memory limit, once for each device.
template <int D, int kNb, typename OT, bool kClusters>
cudaError_t prepare_kernel() {
  static std::mutex mu;
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(paged_attn_kernel<D, kNb, OT, kClusters>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             PagedSmem<D>::bytes(kNb));
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  return cudaSuccess;
}

// f(D, kNb, OT()) for the given sizes, the first two as integral constants.
template <typename F>
cudaError_t for_sizes(int d, int rows, bool f32, F f) {
  auto with_type = [&](auto D, auto nb) {
    return f32 ? f(D, nb, float()) : f(D, nb, __nv_bfloat16());
  };
  auto with_rows = [&](auto D) {
    switch (rows) {
      case 8: return with_type(D, std::integral_constant<int, 1>());
      case 16: return with_type(D, std::integral_constant<int, 2>());
      case 24: return with_type(D, std::integral_constant<int, 3>());
      default: return with_type(D, std::integral_constant<int, 4>());
    }
  };
  return d == 64 ? with_rows(std::integral_constant<int, 64>()) : with_rows(std::integral_constant<int, 128>());
}

// The launch with a cluster for each of `items` items (paged_attn_few.cu).
cudaError_t launch_few(const PagedParams& p, int d, int rows, bool f32, int items, cudaStream_t st);

}  // namespace paged
}  // namespace ditattn
