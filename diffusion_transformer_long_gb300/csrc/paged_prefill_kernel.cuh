// Attention of a step's new tokens over a paged key/value cache, and the join of its parts.
//
// Query token i of request b, at position p = start_b + i, with key/value head h of its group of
// G = H_q / H_kv query heads:
//   s_j = scale q . k_j over the cached keys j < seq_lens[b] (causal: j <= p too),
//   o = sum_j softmax_j(s_j) v_j,  lse = ln sum_j exp(s_j)
//
// An item is (request, key/value head, block of tokens): two Q tiles of 128 rows, row r of a tile being
// token r / G, head r % G of the group, so that a group's heads share one pass over the keys whatever G is
// and a few tokens still fill a tile.  One TMA box of (64 channels, G heads, 128 / G tokens) a tile and
// channel block lays the rows out that way.  The pipeline is that of the dense kernel (attn_kernel.cuh:
// scores and products on tcgen05 with both accumulators in tensor memory, the softmax's online maximum
// raised only when it falls behind by 2^8, weights rounded to bf16 and normalised by the sum of the rounded
// ones, the lse from the unrounded sum), with four differences:
//
// - Keys and values come page by page: the producer warp's lanes look a batch of table entries up (one
//   batch ahead), and each copies its own run of at most 128 rows of one page (the largest power of two
//   that divides the page size) to its place in the 128-byte-swizzled tile.  An entry outside the pool
//   becomes a copy from past the pool's end, which reads as zeros, and a bit in the tile's mask.
// - Each row has its own last key, and each Q tile its own last tile, so that a tile that no row of one Q
//   tile sees is not multiplied for it.  Values behind the request's last key are zeroed in shared memory.
//   Values that some rows of a tile must not see are looked through for infinities and NaN, which a weight
//   of 0 would not hide: they are taken out and given to the rows that see them at the end.
// - Work is dealt out by cost (an item's keys, and a fixed cost beside them): whole items in waves over the
//   blocks while there are many, and the rest in runs of key tiles, whatever they belong to, such that all
//   blocks' costs end up alike: causal items are of very different lengths, and a few tokens on a long
//   cache are few items.  A run that ends inside an item leaves fp32 parts in the workspace, at most two a
//   block, joined in the blocks' order by a second launch: equal calls give equal bits.  Where the table has no
//   room for long items they stay whole and there is no second launch.
// - One warp works the segments of the block's run out, from the lengths on the device, into a ring that the
//   other roles read: they agree by construction and hold none of the arithmetic in registers.
//
// Steps of few tokens a request (at most 64 rows on average) take items of one Q tile of 64 rows: items follow each other
// through the two halves of the block's resources in turn, behind five key and value tiles instead of three (256
// requests of 4 tokens on 100-4096 keys, 24 heads on 8: 479 -> 385 us; 8192 of 2 tokens on 16-1100: 6.9 -> 5.0 ms).
//
// Bound by the tensor pipe and the softmax's chain for chunks of tokens, by HBM for a few tokens a request.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "attn_kernel.cuh"
#include "paged_device.cuh"
#include "paged_launch.h"
#include "sm103_ptx.cuh"

namespace ditattn {
namespace prefill {

constexpr int kSegs = 4;               // segments in the ring
constexpr int kSegWords = 16;
constexpr int kMaskRing = 16;          // key tiles whose masks are held (the producer runs at most 8 ahead)
constexpr int kHeldWords = 16;         // per segment: 3 tiles x 128 keys, then a flag of each epilogue warp
constexpr int kItemCost = 1024;         // what an item costs beside its keys, in keys
constexpr int kMinRun = 512;           // a block's smallest run, in keys
constexpr int kItemRows = 2 * kBlockM;
constexpr int kSplitCost = 2000;       // what parts and their join cost a block, in keys (about 24 us)
constexpr int kWholeWaves = 6;         // waves up to which whole items are tried
constexpr int kWalkCost = 64;          // of a block's share, in keys, that there is for each request where loads are added up
constexpr int kMaxGrid = 256;          // largest grid
constexpr long long kHeadBytes = 192LL << 20;  // of a request's keys and values, above which its items go head by head
constexpr int kScheduleWarp = kPvWarp + 1;
constexpr int kConsumers = 3 + 8 + 4;  // of a segment: producer, two issuers, softmax and epilogue warps

// How a cache's rows reach a tile.  A tile of D = 128 holds two blocks of 64 channels, 128 bytes a row.  A copy brings
// a run of rows of one block, and the blocks are 16 KB apart; or (fused) both blocks of the run, as a 5-D box (64
// channels, 8 rows, channel blocks, groups of 8 rows, ..): groups of 8 rows follow each other, the blocks in turn in
// each.  That takes one of the four dimensions row-in-group, group, head, page out of the map, which the strides allow
// where pages are whole numbers of heads apart (by_head), or of groups of rows.
// (The layout is a template's: an issuer that works descriptors out between the products starves the tensor pipe,
// 1640 -> 1360 TFLOP/s on 54560 keys in pages of 128.)
struct KvPlace {
  int by_head;  // fused: page * apart + head is the last coordinate, else page * apart + group the last but one
  int apart;
};
template <int D, bool kFused>
struct KvTile {
  static_assert(D == 128 || !kFused, "one channel block needs no fusing");
  static constexpr uint32_t kGroup = kFused ? 2048 : 1024;                // bytes from one group of 8 rows to the next
  static constexpr uint32_t kBlock = kFused ? 1024 : kBlockM * 128;  // from one channel block to the next
};

struct PrefillParams {
  CUtensorMap tm_q;        // (D, head of the group, token, key/value head)
  CUtensorMap tm_k, tm_v;  // maps::encode_rows, or, where kFused, paged_prefill.cu: encode_fused
  const __nv_bfloat16* v_cache;
  Strides vs;
  const int* table;
  long long table_stride;
  const int* seq_lens;
  const int* cu_new;
  const int* start_lens;  // or null: a request's new tokens are its last
  void* out;
  int out_align32;
  float* lse;       // may be null
  float* part_o;    // [blocks][2][256][D]
  float* part_lse;  // [blocks][2][256], base 2
  int4* meta;       // [blocks]: (first row of the item's tokens, tokens, key/value head, parts; 0: nothing to join)
  int batch, tokens, h_q, h_kv, group;
  int tile_tokens, item_tokens;  // of a Q tile, 128 / group, and of an item
  int page_size, n_pages, max_len;
  int box_rows;   // rows of one copy
  KvPlace kv[2];  // of K and V, fused
  int div_group;  // 2^16 / group, rounded up: r / group for r < 128 is r * div_group >> 16
  int causal;
  int key_bytes;  // of one key and value, all heads
  int split;  // 0: items stay whole
  float scale_log2;
  int* status;
  long long wait_limit;
  int stall;
};

// One block's shared memory.  `one`: items of at most 64 rows of one Q tile (the products' other rows are whatever lies
// behind them, and nobody looks at theirs), which take everything that two Q tiles have (places for Q and weights, tensor
// memory, a softmax warpgroup) in turn, so that an item's end and the next one's start overlap.  What half the rows
// leave holds two more key and value tiles (of D = 64: ten in all).
template <int kD, bool one>
struct Smem {
  static constexpr bool kOne = one;
  static constexpr int D = kD;
  static constexpr int kTiles = kOne ? 1 : 2;  // Q tiles of an item
  static constexpr int kStages = kOne ? 640 / D : 3;
  static constexpr uint32_t kRegion = kBlockM * 128;         // one channel block of a tile
  static constexpr uint32_t kTile = kBlockM * D * 2;         // Q, K or V
  static constexpr int kRows = kOne ? 64 : kBlockM;          // rows of an item's Q tile
  static constexpr uint32_t kPRegion = kRows * 128;          // 64 keys of the weights
  static constexpr uint32_t kPTile = 2 * kPRegion;
  static constexpr int kQTurns = kOne ? 2 : 1;
  static constexpr uint32_t kQRegion = kRows * 128;          // one channel block of Q
  static constexpr uint32_t kQTile = kQRegion * (D / 64);
  static constexpr uint32_t kQ = 0, kP = kQ + 2 * kQTile, kKV = kP + 2 * kPTile;
  static constexpr uint32_t kBars = kKV + kStages * kTile;
  // barrier indices; t: Q tile of an item, or turn
  static constexpr int bQFull = 0;                   // + turn: an item's Q tiles have landed
  static constexpr int bQEmpty = bQFull + kQTurns;   // + turn: its last S product is done
  static constexpr int bKFull = bQEmpty + kQTurns;   // + slot: a K tile has landed
  static constexpr int bVFull = bKFull + kStages;    // + slot: a V tile has landed
  static constexpr int bKVEmpty = bVFull + kStages;  // + slot: the slot's tile was consumed
  static constexpr int bSFull = bKVEmpty + kStages;  // + t: S_t computed
  static constexpr int bSEmpty = bSFull + 2;         // + t: S_t read into registers (kRows)
  static constexpr int bPLo = bSEmpty + 2;           // + t: keys 0-63 of P_t written (kRows)
  static constexpr int bPFull = bPLo + 2;            // + t: keys 64-127 of P_t written (kRows)
  static constexpr int bPVDone = bPFull + 2;         // + t: O_t += P_t V done
  static constexpr int bOEmpty = bPVDone + 2;        // + t: O_t read by the epilogue (128)
  static constexpr int bEpiReady = bOEmpty + 2;      // + t: normaliser of an item written (kRows)
  static constexpr int bEpiTaken = bEpiReady + 2;    // + t: normaliser read (128)
  static constexpr int bDrainS = bEpiTaken + 2;      // abort drain, S issuer
  static constexpr int bDrainPV = bDrainS + 1;       // abort drain, PV issuer
  static constexpr int bSegFull = bDrainPV + 1;      // + slot of the ring of segments
  static constexpr int bSegEmpty = bSegFull + kSegs;
  static constexpr int bVEdge = bSegEmpty + kSegs;  // a value tile that some row must not see whole has landed
  static constexpr int bVFixed = bVEdge + 1;        // ... and is ready for the product (128)
  static constexpr int kNumBars = bVFixed + 1;
  static constexpr uint32_t kTmemSlot = kBars + kNumBars * 8;
  static constexpr uint32_t kAbort = kTmemSlot + 4;
  static constexpr uint32_t kMasks = kAbort + 4;
  static constexpr uint32_t kSeg = (kMasks + kMaskRing * 4 + 15) & ~15u;
  static constexpr uint32_t kHeld = kSeg + kSegs * kSegWords * 4;
  static constexpr uint32_t kInvLp = kHeld + kSegs * kHeldWords * 4;
  static constexpr uint32_t kUsed = kInvLp + 2 * kBlockM * 4;
  static constexpr uint32_t kBytes = kUsed + 1024;
  static_assert(kBytes <= 232448, "shared memory budget");
};

// One request of the step, from the lengths on the device.
struct Request {
  int row0, n;      // first row of its new tokens, how many
  int len;          // cached keys
  long long start;  // position of the first new token, within [-2^30, len] (a step has at most 2^30 tokens)
  __device__ __forceinline__ void load(const PrefillParams& p, int b) {
    row0 = min(max(p.cu_new[b], 0), p.tokens);
    n = max(0, min(max(p.cu_new[b + 1], 0), p.tokens) - row0);
    len = min(max(p.seq_lens[b], 0), p.max_len);
    start = p.start_lens ? max(min(p.start_lens[b], len), -(1 << 30)) : static_cast<long long>(len) - n;
  }
  __device__ __forceinline__ int items(const PrefillParams& p) const {
    return (n + p.item_tokens - 1) / p.item_tokens;
  }
  // Keys that the first `upto` tokens see at most.
  __device__ __forceinline__ int seen(const PrefillParams& p, long long upto) const {
    if (!p.causal) return len;
    return static_cast<int>(min(max(start + upto, 0LL), static_cast<long long>(len)));
  }
  __device__ __forceinline__ int item_keys(const PrefillParams& p, int i) const {
    return seen(p, min(static_cast<long long>(n), static_cast<long long>(i + 1) * p.item_tokens));
  }
  // Cost of the first i items of one head: i kItemCost + sum of item_keys.  All but the request's last
  // item end at start + (u + 1) tb, clipped to [0, len].
  __device__ __forceinline__ long long cost(const PrefillParams& p, int i) const {
    long long sum = static_cast<long long>(i) * kItemCost;
    if (!p.causal) return sum + static_cast<long long>(i) * len;
    if (i > 0 && i == items(p)) sum += item_keys(p, --i);
    const unsigned tb = p.item_tokens;
    const long long lo = start < 0 ? min(static_cast<unsigned>(i), static_cast<unsigned>(-start) / tb) : 0;
    long long hi = len > start ? (static_cast<unsigned>(len - start) + tb - 1) / tb - 1 : 0;  // items that end before len
    hi = min(max(hi, lo), static_cast<long long>(i));
    const long long m = hi - lo;
    sum += m * start + static_cast<long long>(tb) * (m * (lo + hi + 1) / 2);
    return sum + (i - hi) * len;
  }
  // Whether the request's items count head by head, or block of tokens by block of tokens.
  __device__ __forceinline__ bool by_head(const PrefillParams& p) const {
    return static_cast<long long>(len) * p.key_bytes > kHeadBytes;
  }
  // Item w of the request (it has fewer than 2^31): block i of head h.
  __device__ __forceinline__ void item(const PrefillParams& p, long long w, int& i, int& h) const {
    const unsigned n = by_head(p) ? items(p) : p.h_kv, q = static_cast<unsigned>(w) / n, r = static_cast<unsigned>(w) - q * n;
    i = by_head(p) ? r : q;
    h = by_head(p) ? q : r;
  }
};

struct Segment {
  int b, h;        // request (below 0: no more), key/value head
  int row0, ntok;  // first row of the item's tokens, how many
  int pos0;        // position of the first, at most len
  int len;
  int k0, e0, e1;  // key tiles [k0, e_t) of Q tile t
  int kind;        // 0: the whole item, 1: a later part (slot 0), 2: its first part (slot 1)
  __device__ __forceinline__ int end(int t) const { return t ? e1 : e0; }
  __device__ __forceinline__ int last() const { return max(e0, e1); }
  __device__ __forceinline__ bool present(const PrefillParams& p, int t) const {
    return t == 0 || ntok > p.tile_tokens;
  }
  // Keys that row r of Q tile t sees.  Rows without a token see what the tile's last token does.
  __device__ __forceinline__ int limit(const PrefillParams& p, int t, int r) const {
    if (!p.causal) return len;
    const int tok = min(t * p.tile_tokens + ((r * p.div_group) >> 16), min(ntok, (t + 1) * p.tile_tokens) - 1);
    return static_cast<int>(min(max(static_cast<long long>(pos0) + tok + 1, 0LL), static_cast<long long>(len)));
  }
  // Keys that every row sees.
  __device__ __forceinline__ int seen_by_all(const PrefillParams& p) const { return limit(p, 0, 0); }
  // The segment's key tiles from this one on (counted from k0) hold keys that some row does not see, or the
  // request's last key.
  __device__ __forceinline__ int edge(const PrefillParams& p) const {
    return max(0, min(last(), seen_by_all(p) / kBlockN) - k0);
  }
  __device__ __forceinline__ bool has_token(const PrefillParams& p, int t, int r, int& tok) const {
    const int i = (r * p.div_group) >> 16;
    tok = t * p.tile_tokens + i;
    return i < p.tile_tokens && tok < ntok;
  }
};

using detail::k_item;  // K/V ring items of a segment in consumption order, as in the dense kernel
using detail::v_item;

// The dense kernel's bounded wait and abort, by shared address (a generic pointer costs the softmax two registers).
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
__device__ __forceinline__ void raise_abort(const PrefillParams& p, uint32_t abort_flag) {
  asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(abort_flag), "r"(1) : "memory");
  atomicOr(p.status, kStatusTimeout);
}

// Shared-memory matrix descriptors, as the dense kernel's: the high word holds the stride byte offset (from one
// group of 8 rows to the next), the version and the 128-byte swizzle, the low word the address and the leading
// byte offset.
__device__ constexpr uint32_t desc_hi(uint32_t group) { return (group >> 4) | (1u << 14) | (2u << 29); }
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return (addr >> 4) | ((lbo >> 4) << 16); }
__device__ __forceinline__ uint64_t desc(uint32_t hi, uint32_t lo) {
  return (static_cast<uint64_t>(hi) << 32) | static_cast<uint64_t>(lo);
}

template <int N>
__device__ __forceinline__ uint32_t pick(const uint32_t (&a)[N], int slot) {
  uint32_t r = a[0];
#pragma unroll
  for (int s = 1; s < N; ++s)
    if (slot == s) r = a[s];
  return r;
}

// The ring of segments as a role sees it.
template <typename S>
struct Segments {
  uint32_t sbase;
  int n = 0;  // taken so far
  __device__ __forceinline__ explicit Segments(uint32_t s) : sbase(s) {}
  __device__ __forceinline__ uint32_t bar(int i) const { return sbase + S::kBars + 8u * i; }
  __device__ __forceinline__ uint32_t slot() const { return sbase + S::kSeg + (n % kSegs) * kSegWords * 4; }
  __device__ __forceinline__ uint32_t held() const { return sbase + S::kHeld + (n % kSegs) * kHeldWords * 4; }
  __device__ __forceinline__ bool wait(const PrefillParams& p) const {
    return wait_or_abort(bar(S::bSegFull + n % kSegs), (n / kSegs) & 1, sbase + S::kAbort, p.wait_limit);
  }
  __device__ __forceinline__ Segment read() const {
    int w[12];
#pragma unroll
    for (int i = 0; i < 3; ++i)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                   : "r"(slot() + 16 * i)
                   : "memory");
    return {w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7], w[8], w[9]};
  }
  // One lane of the role's warp: the segment's words are no longer needed.
  __device__ __forceinline__ void release() const { ptx::mbar_arrive(bar(S::bSegEmpty + n % kSegs)); }
};

// The block's segments (one warp).  The blocks of a wave work on neighbouring items, side by side through the same
// keys (with a run of items to each block, 152 places of all heads' keys were read at once: 27280 keys, 24 heads,
// 25 % of the reads hit L2).  A request's items count block of tokens by block of tokens, all heads of each, so that a
// wave's are of like lengths (one prompt of 4608 tokens, 24 heads on 8: 174 us; head by head 196), but
// head by head where all heads' keys and values are too many for L2 (27280 tokens, 24 heads, 335 MB: 3.21 ms; by
// blocks of tokens 3.37; of 112 MB, 3.53 and 3.38).
// Waves of whole items go over the blocks, to and fro, for as long as no block has more than its share of the cost;
// what is left is dealt out so that all blocks' costs end up alike.  Where that would gain less than the parts cost, all
// items stay whole (one prompt of 4608 tokens, 24 heads on 8, L2 cold: 138 us; in parts 158).
// The code runs once, and what it costs is fetching it: loops are rolled, divisions of 32 bits where they fit.
template <typename S>
__device__ __forceinline__ void scheduler(const PrefillParams& p, uint32_t sbase, int lane) {
  const int c = blockIdx.x, grid = gridDim.x;
  Request rq;
  long long total = 0, items = 0;
  int least = 0x7fffffff, most = -1;  // keys of the shortest and the longest item
  for (int b = lane; b < p.batch; b += 32) {
    rq.load(p, b);
    const int nb = rq.items(p);
    total += rq.cost(p, nb);
    items += nb;
    if (nb > 0) {  // (item_keys does not fall with the item)
      least = min(least, rq.item_keys(p, 0));
      most = max(most, rq.item_keys(p, nb - 1));
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    total += __shfl_xor_sync(~0u, total, o);
    items += __shfl_xor_sync(~0u, items, o);
  }
  total *= p.h_kv;
  items *= p.h_kv;
  least = __reduce_min_sync(~0u, least);
  most = __reduce_max_sync(~0u, most);
  const bool even = least == most;
  const long long share = total / grid;
  // Waves that are safe without looking at the blocks' loads.
  long long waves = p.split ? items / grid : (items + grid - 1) / grid;
  // (Adding waves' costs up walks over the requests, 0.2 us each: 256 of 4 tokens, 8 heads on 2, 195 us with it and 134
  // without; 24 heads on 8, 392 and 433.)
  const bool look = p.split && !even && share >= static_cast<long long>(p.batch) * kWalkCost;
  if (p.split && !even) waves = look ? min(waves, min(2LL, share / (most + kItemCost))) : 0;

  int4 meta = make_int4(0, 0, 0, 0);
  int n = 0;  // segments written
  bool ok = true;
  auto emit = [&](const Segment& s) {
    const int slot = n % kSegs;
    if (n >= kSegs) {
      if (lane == 0)
        ok = wait_or_abort(sbase + S::kBars + 8u * (S::bSegEmpty + slot), (n / kSegs - 1) & 1, sbase + S::kAbort, p.wait_limit);
      ok = __shfl_sync(~0u, ok, 0) != 0;
      if (!ok) return;
    }
    if (lane == 0) {
      const uint32_t at = sbase + S::kSeg + slot * kSegWords * 4;
      const int w[12] = {s.b, s.h, s.row0, s.ntok, s.pos0, s.len, s.k0, s.e0, s.e1, s.kind, 0, 0};
#pragma unroll
      for (int i = 0; i < 3; ++i)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + 16 * i), "r"(w[4 * i]), "r"(w[4 * i + 1]),
                     "r"(w[4 * i + 2]), "r"(w[4 * i + 3])
                     : "memory");
      ptx::mbar_arrive(sbase + S::kBars + 8u * (S::bSegFull + slot));
    }
    ++n;
  };
  // Key tiles [a, e) of item i of request b, for head h.
  auto emit_item = [&](int b, int i, int h, int a, int e, int ntiles) {
    Segment s;
    s.b = b;
    s.h = h;
    const int t0 = i * p.item_tokens;
    s.row0 = rq.row0 + t0;
    s.ntok = min(rq.n - t0, p.item_tokens);
    s.len = rq.len;
    s.pos0 = static_cast<int>(max(min(rq.start + t0, static_cast<long long>(rq.len)), -(1LL << 30)));
    s.k0 = a;
    const int f0 = (rq.seen(p, t0 + min(s.ntok, p.tile_tokens)) + kBlockN - 1) / kBlockN;
    s.e0 = max(a, min(f0, e));
    s.e1 = s.ntok > p.tile_tokens ? e : a;
    s.kind = a == 0 && e == ntiles ? 0 : a == 0 ? 2 : 1;
    emit(s);
  };
  // The first request, from b on, up to which `value` (of a request, in rq) adds up to more than x - base; base becomes
  // the sum before it.  b = batch: there is none.
  auto seek = [&](int& b, long long& base, long long x, auto value) {
    for (; b < p.batch; b += 32) {
      long long mine = 0;
      if (b + lane < p.batch) {
        rq.load(p, b + lane);
        mine = value();
      }
      long long upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += y;
      }
      const unsigned past = __ballot_sync(~0u, base + upto > x);
      if (past) {
        const int l = __ffs(past) - 1;
        base += __shfl_sync(~0u, upto - mine, l);
        b += l;
        rq.load(p, b);
        return;
      }
      base += __shfl_sync(~0u, upto, 31);
    }
  };

  int wave_b = 0;
  long long wave_base = 0, wave_have = 0;  // items before request wave_b, and its own
  // Each lane holds the loads of `own` blocks in a row, then their shares of the rest, then where their runs end.
  constexpr int kOwn = kMaxGrid / 32;
  const int own = (grid + 31) / 32;
  long long end[kOwn], settled[kOwn];
  Request load_rq;
  int load_b = 0;
  long long load_base = 0, load_have = 0;  // (a lane's own, as wave_b ..)
  int cost[kOwn];
  // The costs of wave k.  0: no block's load passes its share with them, 1: none by more than the parts cost, 2: one does.
  auto wave_costs = [&](long long k) {
    int over = 0;
#pragma unroll 1
    for (int i = 0; i < own; ++i) {
      // In the order of the items: of block lane own + i, or on the way back of lane own + own - 1 - i.
      const int q = k & 1 ? own - 1 - i : i, x = lane * own + q;
      cost[q] = 0;
      if (x >= grid) continue;
      const long long w = k * grid + (k & 1 ? grid - 1 - x : x);
      if (w >= items) continue;
      while (w >= load_base + load_have) {
        load_base += load_have;
        load_rq.load(p, ++load_b);
        load_have = static_cast<long long>(load_rq.items(p)) * p.h_kv;
      }
      int block, h;
      load_rq.item(p, w - load_base, block, h);
      cost[q] = load_rq.item_keys(p, block) + kItemCost;
      const long long load = end[q] + cost[q];
      over = max(over, (load > share) + (load > share + kSplitCost));
    }
    return static_cast<int>(__reduce_max_sync(~0u, static_cast<unsigned>(over)));
  };
  const long long full = items / grid, all_waves = (items + grid - 1) / grid;
  // Waves up to the blocks' shares, each as soon as it is known to be within them.  Of few waves, whole items all the
  // same where that leaves no block further behind than the parts cost.
  const bool whole = p.split && all_waves <= kWholeWaves && share + kSplitCost >= most + kItemCost;
  if (whole && even && all_waves * (most + kItemCost) <= share + kSplitCost) waves = all_waves;
  const long long sure = waves;  // (within both)
  bool one_by_one = sure > 0, adding = look && sure < all_waves && (whole || one_by_one);
  long long k = 0, added = 0, before = 0;  // waves that are out, and in the loads; cost of what the waves took
#pragma unroll 1
  for (int q = 0; q < kOwn; ++q) end[q] = settled[q] = 0;
  if (adding) {
    load_rq.load(p, 0);
    load_have = static_cast<long long>(load_rq.items(p)) * p.h_kv;
  }
  for (;;) {
    for (; ok && k < waves; ++k) {
      const long long w = k * grid + (k & 1 ? grid - 1 - c : c);
      if (w >= items) continue;
      if (w >= wave_base + wave_have)
        seek(wave_b, wave_base, w, [&] { return static_cast<long long>(rq.items(p)) * p.h_kv; });
      else
        rq.load(p, wave_b);
      wave_have = static_cast<long long>(rq.items(p)) * p.h_kv;
      int i, h;
      rq.item(p, w - wave_base, i, h);
      const int ntiles = (rq.item_keys(p, i) + kBlockN - 1) / kBlockN;
      emit_item(wave_b, i, h, 0, ntiles, ntiles);
    }
    if (!ok || !adding) break;
#pragma unroll 1
    for (bool out = false; adding && !out;) {
      int over = added < all_waves ? wave_costs(added) : 0;
      if (added < sure) over = 0;
      if (one_by_one && (over > 0 || added >= full)) {
        one_by_one = false;
        adding = whole;
#pragma unroll 1
        for (int q = 0; q < own; ++q) settled[q] = end[q];
        if (!adding) break;
      }
      if (added == all_waves) waves = all_waves;
      if (over == 2 || added == all_waves) {
        adding = false;
        break;
      }
#pragma unroll 1
      for (int q = 0; q < own; ++q) end[q] += cost[q];
      ++added;
      if (one_by_one && added > waves) {
        waves = added;
        out = true;
      }
    }
  }

  if (ok && p.split && waves * grid < items) {
    if (even) {
      before = total / items * (waves * grid);
    } else if (waves > 0) {
#pragma unroll 1
      for (int q = 0; q < own; ++q) before += end[q] = settled[q];
#pragma unroll
      for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(~0u, before, o);
    }
    if (even || waves == 0 || total - before < static_cast<long long>(grid) * kMinRun) {
      const long long blocks = min(static_cast<long long>(grid), max(1LL, (total - before) / kMinRun));
#pragma unroll 1
      for (int q = 0; q < own; ++q) end[q] = lane * own + q < blocks ? 1 : 0;
    } else {
#pragma unroll 1
      for (int q = 0; q < own; ++q) {
        const long long rest = share - end[q];
        end[q] = lane * own + q < grid && rest > 0 ? rest : 0;
      }
    }
    long long mine = 0;
#pragma unroll 1
    for (int q = 0; q < own; ++q) mine = end[q] += mine;
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += y;
    }
    const long long all = __shfl_sync(~0u, upto, 31);
    const double unit = static_cast<double>(total - before) / static_cast<double>(max(1LL, all));
#pragma unroll 1
    for (int q = 0; q < own; ++q) {
      const long long x = upto - mine + end[q];  // of `all` (none: the first block's)
      end[q] = x == all ? total : before + static_cast<long long>(static_cast<double>(x) * unit);
    }
    // This block's run: [run0, run1).
    long long run0 = before, run1 = before;
    {
      long long x0 = 0, x1 = 0;
#pragma unroll 1
      for (int q = 0; q < own; ++q) {
        if (q == (c + own - 1) % own) x0 = end[q];
        if (q == c % own) x1 = end[q];
      }
      x0 = __shfl_sync(~0u, x0, ((c + own - 1) / own - 1) & 31);
      run1 = __shfl_sync(~0u, x1, c / own);
      if (c > 0) run0 = x0;
    }
    if (ok && run0 < total) {
      int b = 0;
      long long base = 0;
      seek(b, base, run0, [&] { return rq.cost(p, rq.items(p)) * p.h_kv; });
      int nb = rq.items(p);
      // Head h, item i, and how far into its cost.
      int h = 0, i;
      long long x0 = run0 - base;
      {
        // By blocks of tokens, all heads' items i count before any head's i + 1.
        const long long per_head = rq.cost(p, nb), many = rq.by_head(p) ? 1 : p.h_kv;
        if (rq.by_head(p)) {
          h = static_cast<int>(x0 / per_head);
          x0 -= h * per_head;
        }
        int lo = 0, hi = nb - 1;
        while (lo < hi) {
          const int mid = lo + (hi - lo + 1) / 2;
          if (rq.cost(p, mid) * many <= x0) lo = mid; else hi = mid - 1;
        }
        i = lo;
        x0 -= rq.cost(p, i) * many;
        if (!rq.by_head(p)) {
          const long long each = static_cast<long long>(rq.item_keys(p, i)) + kItemCost;
          h = static_cast<int>(x0 / each);
          x0 -= h * each;
        }
      }
      long long at = run0;  // x0's place in the whole
      while (ok) {
        const int keys = rq.item_keys(p, i);
        const long long cost = static_cast<long long>(keys) + kItemCost, take = min(cost - x0, run1 - at);
        const int ntiles = (keys + kBlockN - 1) / kBlockN;
        auto cut = [&](long long x) { return x >= keys ? ntiles : static_cast<int>((x + kBlockN - 1) / kBlockN); };
        const int a = cut(x0), e = cut(x0 + take);
        // A run that meets an item begun before has a part of it, if an empty one, unless its tiles are all done.
        if (a < e || (ntiles == 0 && x0 == 0 && take > 0) || (x0 > 0 && a < ntiles)) {
          if (a == 0 && e < ntiles) {
            // The item's last part is in the first block whose run ends behind the item's last tile's start.
            const long long x = at - x0 + static_cast<long long>(ntiles - 1) * kBlockN;
            int last = 0;
#pragma unroll 1
            for (int q = 0; q < own; ++q) last += lane * own + q < grid && end[q] <= x;
            last = __reduce_add_sync(~0u, last);
            const int t0 = i * p.item_tokens;
            meta = make_int4(rq.row0 + t0, min(rq.n - t0, p.item_tokens), h, last - c + 1);
          }
          emit_item(b, i, h, a, e, ntiles);
        }
        at += take;
        if (at >= run1) break;
        x0 = 0;
        bool over;
        if (rq.by_head(p)) {
          over = ++i == nb;
          if (over) {
            i = 0;
            over = ++h == p.h_kv;
          }
        } else {
          over = ++h == p.h_kv;
          if (over) {
            h = 0;
            over = ++i == nb;
          }
        }
        if (over) {
          i = h = 0;
          ++b;
          long long none = 0;
          seek(b, none, 0, [&] { return static_cast<long long>(rq.n); });  // the next with new tokens
          if (b >= p.batch) break;  // (not reached: the run would have ended)
          nb = rq.items(p);
        }
      }
    }
  }
  if (ok) {
    Segment s{};
    s.b = -1;
    emit(s);
  }
  if (p.split && lane == 0) p.meta[c] = meta;
  if (!ok) raise_abort(p, sbase + S::kAbort);
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

// Copies: Q of each segment, then its key and value tiles (one warp; each lane its own rows of a tile).
template <typename S, bool kFused>
__device__ __forceinline__ void producer(const PrefillParams& p, uint32_t sbase, int lane) {
  constexpr int D = S::D, kStages = S::kStages;
  constexpr int kRegions = D / 64;
  auto bar = [&](int i) { return sbase + S::kBars + 8u * i; };
  // Lane 0 waits for all.
  auto wait = [&](int b, uint32_t parity) {
    bool done = true;
    if (lane == 0) done = wait_or_abort(bar(b), parity, sbase + S::kAbort, p.wait_limit);
    return __shfl_sync(~0u, done, 0) != 0;
  };
  const int boxes = kBlockN / p.box_rows;  // of a tile: 1, 2, 4 or 8
  const int per_batch = 32 / boxes;        // tiles looked up at once
  const int box = lane % boxes;            // the lane's box of a tile
  // The lane copies its box, or channel block lane / boxes of it where those are copied apart.
  const int copy_block = kFused ? 0 : lane / boxes;
  const uint32_t copy_dst = sbase + S::kKV + box * (p.box_rows / 8) * KvTile<D, kFused>::kGroup +
                            copy_block * KvTile<D, kFused>::kBlock;
  const uint32_t q_bytes = static_cast<uint32_t>(p.group * p.tile_tokens) * 128 * kRegions;

  uint32_t kpar = 0, vpar = 0;  // bit s: parity of the next K_FULL[s] / V_FULL[s] phase
  int last_bar[kStages];        // barrier and parity of the newest copy into each slot
  uint32_t last_par[kStages];
#pragma unroll
  for (int s = 0; s < kStages; ++s) {
    last_bar[s] = -1;
    last_par[s] = 0;
  }
  uint32_t qpar = 0, q_loaded = 0;  // bit t: parity of turn t's next Q load, whether there was one
  int it = 0, tiles = 0;            // ring index, key tiles so far
  bool ok = true;
  Segments<S> segs(sbase);
  for (;; ++segs.n) {
    if (!(ok = __all_sync(~0u, segs.wait(p)))) break;
    const Segment sg = segs.read();
    __syncwarp();
    if (lane == 0) segs.release();
    if (sg.b < 0) break;
    const int kend = sg.last();
    if (kend == sg.k0) continue;  // no keys
    // A Q tile is free once its segment's last S MMAs have completed.
    const int turn = S::kOne ? segs.n & 1 : 0;
    if (!(ok = wait(S::bQEmpty + turn, ((qpar >> turn) & 1) ^ 1))) break;
    if (lane == 0) {
      ptx::mbar_arrive_expect_tx(bar(S::bQFull + turn), q_bytes * ((sg.e0 > sg.k0) + (sg.e1 > sg.k0)));
#pragma unroll
      for (int t = 0; t < S::kTiles; ++t)
        if (sg.end(t) > sg.k0)
#pragma unroll
          for (int r = 0; r < kRegions; ++r)
            ptx::tma_load_4d(sbase + S::kQ + (t + turn) * S::kQTile + r * S::kQRegion, &p.tm_q, bar(S::bQFull + turn), r * 64, 0,
                             sg.row0 + t * p.tile_tokens, sg.h);
    }
    qpar ^= 1u << turn;
    q_loaded |= 1u << turn;
    if (p.stall) return;  // test only: the consumers' first K wait will expire

    const int pages = pages_of(sg.len, p.page_size);
    const int* const row = p.table + sg.b * p.table_stride;
    // The lane's box of tile j0 + lane / boxes: page (-1: none, -2: behind the keys), first row in it.
    auto look_up = [&](int j0, int& page, int& first) {
      const unsigned key = static_cast<unsigned>(j0 + lane / boxes) * kBlockN + box * p.box_rows;
      const int col = static_cast<int>(key / static_cast<unsigned>(p.page_size));
      first = static_cast<int>(key - static_cast<unsigned>(col) * p.page_size);
      page = -2;
      if (j0 + lane / boxes < kend && col < pages) {
        page = row[col];
        if (page < 0 || page >= p.n_pages) page = -1;
      }
    };
    int page_a, first_a, page_b, first_b;  // the batch in use and the one ahead
    int base = sg.k0;
    look_up(base, page_a, first_a);
    look_up(base + per_batch, page_b, first_b);
    int kpage = -2, kfirst = 0, vpage = -2, vfirst = 0;  // of the lane's box in the newest key tile, and in the one before
    auto take = [&](int j) {
      if (j - base == per_batch) {
        base = j;
        page_a = page_b;
        first_a = first_b;
        look_up(base + per_batch, page_b, first_b);
      }
      const int from = (j - base) * boxes + box;
      vpage = kpage;
      vfirst = kfirst;
      kpage = __shfl_sync(~0u, page_a, from);
      kfirst = __shfl_sync(~0u, first_a, from);
    };
    // The slot's turn comes late (three slots, two tiles in use), so that all but the copies themselves
    // stands before the wait for it.  (The copies may complete before the bytes are expected: the phase
    // still waits for lane 0's arrival.)
    auto load = [&](bool is_v, int page, int first) {
      const int s = it % kStages;
      const int fb = (is_v ? S::bVFull : S::bKFull) + s;
      const uint32_t par = ((is_v ? vpar : kpar) >> s) & 1;
      if (is_v) vpar ^= 1u << s; else kpar ^= 1u << s;
      if (!is_v) {
        // A bit for every 16 keys: without a page.
        const unsigned none = __ballot_sync(~0u, page == -1) & ((1u << boxes) - 1);
        unsigned mask = 0;
        if (none)
          for (int q = 0; q < 8; ++q)
            if ((none >> (q * boxes / 8)) & 1) mask |= 1u << q;
        if (lane == 0)
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(sbase + S::kMasks + 4 * (tiles % kMaskRing)), "r"(mask)
                       : "memory");
        ++tiles;
      }
      const CUtensorMap* const tm = is_v ? &p.tm_v : &p.tm_k;
      const KvPlace kv = p.kv[is_v];
      const uint32_t dst = copy_dst + s * S::kTile;
      if (page < 0) page = p.n_pages;  // (past the pool: zeros)
      int c2 = sg.h, c3 = page;
      if constexpr (kFused) {
        c2 = first / 8 + (kv.by_head ? 0 : page * kv.apart);
        c3 = sg.h + (kv.by_head ? page * kv.apart : 0);
      }
      if (!wait(S::bKVEmpty + s, ((it / kStages) & 1) ^ 1)) return false;
      if (lane == 0) ptx::mbar_arrive_expect_tx(bar(fb), S::kTile);
      if constexpr (kFused) {
        if (lane < boxes) tma_load_5d(dst, tm, bar(fb), 0, 0, 0, c2, c3);
      } else if (lane < boxes * kRegions) {
        ptx::tma_load_4d(dst, tm, bar(fb), copy_block * 64, first, c2, c3);
      }
#pragma unroll
      for (int q = 0; q < kStages; ++q)
        if (q == s) {
          last_bar[q] = fb;
          last_par[q] = par;
        }
      ++it;
      return true;
    };
    take(sg.k0);
    if (!(ok = load(false, kpage, kfirst))) break;
    for (int j = sg.k0; j < kend; ++j) {
      if (j + 1 < kend) {
        take(j + 1);
        if (!(ok = load(false, kpage, kfirst))) break;
        ok = load(true, vpage, vfirst);
      } else {
        ok = load(true, kpage, kfirst);
      }
      if (!ok) break;
    }
    if (!ok) break;
  }
  if (!ok) {
    if (lane == 0) raise_abort(p, sbase + S::kAbort);
    // Let every copy this warp started land before the block can exit.
#pragma unroll
    for (int turn = 0; turn < S::kQTurns; ++turn)
      if ((q_loaded >> turn) & 1) ptx::mbar_wait(bar(S::bQFull + turn), ((qpar >> turn) & 1) ^ 1, p.wait_limit);
#pragma unroll
    for (int s = 0; s < kStages; ++s)
      if (last_bar[s] >= 0) ptx::mbar_wait(bar(last_bar[s]), last_par[s], p.wait_limit);
  }
}

// S_t = Q_t K^T (one thread).
template <typename S, bool kFused>
__device__ __forceinline__ void s_issuer(const PrefillParams& p, uint32_t sbase, uint32_t tmem) {
  constexpr int D = S::D, kStages = S::kStages;
  auto bar = [&](int i) { return sbase + S::kBars + 8u * i; };
  constexpr uint32_t kIdesc = ptx::idesc_bf16_f32(kBlockM, kBlockN, false, false);
  constexpr uint32_t qhi = desc_hi(1024), khi = desc_hi(KvTile<D, kFused>::kGroup);
  constexpr uint32_t kblock = KvTile<D, kFused>::kBlock >> 4;
  uint32_t ks[kStages];
#pragma unroll
  for (int s = 0; s < kStages; ++s) ks[s] = desc_lo(sbase + S::kKV + s * S::kTile, 16);
  const uint32_t qs[2] = {desc_lo(sbase + S::kQ, 16), desc_lo(sbase + S::kQ + S::kQTile, 16)};
  // Both K-major: a step of 16 channels advances 32 bytes inside a channel block, then goes to the next.
  auto issue = [&](int t, int slot) {
    const uint32_t kb = pick(ks, slot), qa = t ? qs[1] : qs[0];
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint32_t step = (k % 4) * 2;
      ptx::mma_bf16_ss(tmem + t * kBlockN, desc(qhi, qa + (k / 4) * (S::kQRegion >> 4) + step),
                       desc(khi, kb + (k / 4) * kblock + step), kIdesc, k > 0 ? 1u : 0u);
    }
  };
  auto wait = [&](int b, uint32_t parity) { return wait_or_abort(bar(b), parity, sbase + S::kAbort, p.wait_limit); };

  uint32_t kpar = 0, gpar = 0, qpar = 0;  // bit t: parity of the S tiles issued, of the Q loads taken
  int ring0 = 0;
  bool ok = true;
  Segments<S> segs(sbase);
  for (; ok; ++segs.n) {
    if (!(ok = segs.wait(p))) break;
    const Segment sg = segs.read();
    segs.release();
    if (sg.b < 0) break;
    const int nt = sg.last() - sg.k0;
    if (nt == 0) continue;
    const int turn = S::kOne ? segs.n & 1 : 0;
    if (!(ok = wait(S::bQFull + turn, (qpar >> turn) & 1))) break;
    qpar ^= 1u << turn;
    for (int j = 0; j < nt; ++j) {
      const int sK = (ring0 + k_item(j)) % kStages;
      ok = wait(S::bKFull + sK, (kpar >> sK) & 1);
      kpar ^= 1u << sK;
      if (!ok) break;
#pragma unroll
      for (int t = 0; t < S::kTiles; ++t) {
        if (!ok || sg.k0 + j >= sg.end(t)) continue;
        // S is overwritten: its softmax must have loaded the last one (nothing to wait for the first time).
        const int at = S::kOne ? turn : t;
        if (!(ok = wait(S::bSEmpty + at, ((gpar >> at) & 1) ^ 1))) continue;
        ptx::tc_fence_after();
        issue(at, sK);
        ptx::mma_commit(bar(S::bSFull + at));
        gpar ^= 1u << at;
      }
      if (!ok) break;
      ptx::mma_commit(bar(S::bKVEmpty + sK));
    }
    if (ok) ptx::mma_commit(bar(S::bQEmpty + turn));
    ring0 += 2 * nt;
  }
  if (!ok) {
    raise_abort(p, sbase + S::kAbort);
    ptx::mma_commit(bar(S::bDrainS));
    ptx::mbar_wait(bar(S::bDrainS), 0, p.wait_limit);
  }
}

// A bit in each half of w whose bf16 is infinite or NaN: bits 15 and 31.
__device__ __forceinline__ uint32_t non_finite(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// Row `row` of a value tile, before the products: zeros if it is not one of the first `valid` (a weight of 0 does not
// hide what a page holds behind the request's last key), and else, where `look`, without its infinities and NaN;
// true: it had some.  (The epilogue's threads, a row each; whole rows are gone through, in an order that spreads the
// banks, so the swizzle does not matter.)
template <int D, bool kFused>
__device__ __forceinline__ bool fix_row(uint32_t tile, int row, int valid, bool look) {
  const uint32_t at = tile + (row / 8) * KvTile<D, kFused>::kGroup + (row % 8) * 128;
  uint32_t bad = 0;
#pragma unroll 1
  for (int ch = 0; ch < D / 8; ++ch) {
    const uint32_t piece = at + (ch / 8) * KvTile<D, kFused>::kBlock + ((ch + row) & 7) * 16;
    if (row >= valid) {
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(piece), "r"(0) : "memory");
    } else if (look) {
      uint32_t w[4];
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "r"(piece)
                   : "memory");
      uint32_t here = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t f = non_finite(w[i]);
        here |= f;
        w[i] &= ~(((f >> 15) & 1) * 0xffffu | (f >> 31) * 0xffff0000u);
      }
      if (here)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(piece), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                     : "memory");
      bad |= here;
    }
  }
  return bad != 0;
}

// O_t += P_t V (one thread: what lanes wait for one another costs here, each product waits for).
template <typename S, bool kFused>
__device__ __forceinline__ void pv_issuer(const PrefillParams& p, uint32_t sbase, uint32_t tmem) {
  constexpr int D = S::D, kStages = S::kStages;
  auto bar = [&](int i) { return sbase + S::kBars + 8u * i; };
  constexpr uint32_t kIdesc = ptx::idesc_bf16_f32(kBlockM, D, false, true);
  constexpr uint32_t phi = desc_hi(1024), vhi = desc_hi(KvTile<D, kFused>::kGroup);
  constexpr uint32_t vgroups = KvTile<D, kFused>::kGroup >> 3;
  uint32_t vs[kStages];
#pragma unroll
  for (int s = 0; s < kStages; ++s) vs[s] = desc_lo(sbase + S::kKV + s * S::kTile, KvTile<D, kFused>::kBlock);
  const uint32_t ps[2] = {desc_lo(sbase + S::kP, 16), desc_lo(sbase + S::kP + S::kPTile, 16)};
  // P K-major; V with the channels contiguous, 16 keys (two groups of rows) a step.
  auto issue = [&](int t, int slot, bool acc, int half) {
    const uint32_t vb = pick(vs, slot), pa = t ? ps[1] : ps[0];
#pragma unroll
    for (int k = half * 4; k < half * 4 + 4; ++k)
      ptx::mma_bf16_ss(tmem + 2 * kBlockN + t * D, desc(phi, pa + (k / 4) * (S::kPRegion >> 4) + (k % 4) * 2),
                       desc(vhi, vb + k * vgroups), kIdesc, (acc || k > 0) ? 1u : 0u);
  };
  auto wait = [&](int b, uint32_t parity) { return wait_or_abort(bar(b), parity, sbase + S::kAbort, p.wait_limit); };

  uint32_t vpar = 0, fixed = 0;
  uint32_t gpar = 0;  // bit t: parity of the PV tiles issued
  uint32_t used = 3;  // bit t: parity of O_EMPTY for the last segment that wrote O_t
  int ring0 = 0;
  bool ok = true;
  Segments<S> segs(sbase);
  for (; ok; ++segs.n) {
    if (!(ok = segs.wait(p))) break;
    int nt0, nt1, edge;
    {
      const Segment sg = segs.read();
      if (sg.b < 0) break;
      nt0 = sg.e0 - sg.k0;
      nt1 = sg.e1 - sg.k0;
      edge = sg.edge(p);
    }
    segs.release();
    const int nt = max(nt0, nt1), turn = segs.n & 1;
    for (int j = 0; j < nt; ++j) {
      const int sV = (ring0 + v_item(j, nt)) % kStages;
      ok = wait(S::bVFull + sV, (vpar >> sV) & 1);
      vpar ^= 1u << sV;
      if (!ok) break;
      if (j >= edge) {
        ptx::mbar_arrive(bar(S::bVEdge));
        if (!(ok = wait(S::bVFixed, fixed))) break;
        fixed ^= 1;
      }
#pragma unroll
      for (int t = 0; t < S::kTiles; ++t) {
        if (!ok || j >= (t ? nt1 : nt0)) continue;
        const int at = S::kOne ? turn : t;
        const uint32_t parity = (gpar >> at) & 1;
        if (!(ok = wait(S::bPLo + at, parity))) continue;
        // The first PV of a segment overwrites O_t: the last one's epilogue must have read it.
        if (j == 0) {
          if (!(ok = wait(S::bOEmpty + at, (used >> at) & 1))) continue;  // (nothing to wait for the first time)
          used ^= 1u << at;
        }
        ptx::tc_fence_after();
        issue(at, sV, j > 0, 0);
        if (!(ok = wait(S::bPFull + at, parity))) continue;
        ptx::tc_fence_after();
        issue(at, sV, j > 0, 1);
        ptx::mma_commit(bar(S::bPVDone + at));
        gpar ^= 1u << at;
      }
      if (!ok) break;
      ptx::mma_commit(bar(S::bKVEmpty + sV));
    }
    ring0 += 2 * nt;
  }
  if (!ok) {
    raise_abort(p, sbase + S::kAbort);
    ptx::mma_commit(bar(S::bDrainPV));
    ptx::mbar_wait(bar(S::bDrainPV), 0, p.wait_limit);
  }
}

// Softmax of Q tile t, or of every other item (four warps, a row a thread).
template <typename S>
__device__ __forceinline__ void softmax_wg(const PrefillParams& p, uint32_t sbase, uint32_t tmem, int t, int warp,
                                           int lane) {
  constexpr int D = S::D;
  auto bar = [&](int i) { return sbase + S::kBars + 8u * i; };
  const int quarter = warp & 3;
  const int r = quarter * 32 + lane;  // row in the Q tile == TMEM lane
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t tS = tmem + t * kBlockN + lane_off;
  const uint32_t tO = tmem + 2 * kBlockN + t * D + lane_off;
  const uint32_t sP = sbase + S::kP + t * S::kPTile;
  const uint32_t sw = static_cast<uint32_t>(r & 7);
  const float c = p.scale_log2;
  const int tile = S::kOne ? 0 : t;  // of the item
  auto wait = [&](int b, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_or_abort(bar(b), parity, sbase + S::kAbort, p.wait_limit));
  };

  int g = 0;      // tiles processed by this warpgroup
  int tiles = 0;  // key tiles of the block so far, for their masks
  uint32_t taken = 1;  // parity of EPI_TAKEN for the last segment
  bool ok = true;
  Segments<S> segs(sbase);
  for (; ok; ++segs.n) {
    if (!(ok = __all_sync(~0u, segs.wait(p)))) break;
    int nt, left;  // the Q tile's key tiles; the row's keys from the first of them on
    {
      const Segment sg = segs.read();
      if (sg.b < 0) break;
      if (S::kOne ? (segs.n & 1) != t || r >= S::kRows : !sg.present(p, t)) {
        tiles += sg.last() - sg.k0;
        __syncwarp();
        if (lane == 0) segs.release();
        continue;
      }
      nt = sg.end(tile) - sg.k0;
      left = sg.limit(p, tile, r) - sg.k0 * kBlockN;
    }
    float m = -INFINITY;  // running max of scale*log2e*s (possibly stale by < 2^8)
    float l = 0.f;        // running sum of 2^(c*s - m), for the LSE
    float lp = 0.f;       // running sum of the bf16-rounded P the PV GEMM sees, for O
    bool first = true;
    uint32_t none = 0;  // the tile's 16-key pieces without a page
    // One tile, whose scores have been waited for.  `masked`: some row does not see it whole.
    auto work = [&](auto masked) {
      float s[kBlockN];
      float cmax[kBlockN / 32];
#pragma unroll
      for (int cc = 0; cc < kBlockN / 32; ++cc) {
        uint32_t u[32];
        ptx::tmem_ld32_max(tS + cc * 32, u, cmax[cc]);
#pragma unroll
        for (int i = 0; i < 32; ++i) s[cc * 32 + i] = __uint_as_float(u[i]);
      }
      ptx::tmem_wait_ld();
      ptx::tc_fence_before();
      ptx::mbar_arrive(bar(S::bSEmpty + t));

      float mx = ptx::fmax3(cmax[0], cmax[1], fmaxf(cmax[2], cmax[3]));
      if constexpr (decltype(masked)::value) {
        // Keys that the row does not see are masked to -inf, so their P is exactly 0, and the max is
        // taken over the others only.
#pragma unroll
        for (int i = 0; i < kBlockN; ++i)
          if (i >= left) s[i] = -INFINITY;
        if (none != 0) {
#pragma unroll
          for (int i = 0; i < kBlockN; ++i)
            if ((none >> (i / 16)) & 1) s[i] = -INFINITY;
        }
        float a[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          a[q] = ptx::fmax3(s[16 * q], s[16 * q + 1], s[16 * q + 2]);
#pragma unroll
          for (int i = 3; i < 15; i += 2) a[q] = ptx::fmax3(a[q], s[16 * q + i], s[16 * q + i + 1]);
          a[q] = fmaxf(a[q], s[16 * q + 15]);
        }
        mx = ptx::fmax3(ptx::fmax3(a[0], a[1], a[2]), ptx::fmax3(a[3], a[4], a[5]), fmaxf(a[6], a[7]));
      }
      const float m_tile = mx * c;
      const bool raise = m_tile > m + kRescaleLog2;
      float alpha = 1.f;
      if (raise) {
        alpha = ptx::ex2_approx(m - m_tile);  // 0 where m = -inf
        m = m_tile;
      }
      l *= alpha;
      lp *= alpha;
      bool pv_prev_done = (g == 0);
      if (!first && __any_sync(0xffffffffu, raise)) {
        if (!(ok = wait(S::bPVDone + t, (g - 1) & 1))) return;
        pv_prev_done = true;
        ptx::tc_fence_after();
#pragma unroll 1
        for (int cc = 0; cc < D / 16; ++cc) {
          uint32_t u[16];
          ptx::tmem_ld16(tO + cc * 16, u);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * alpha);
          ptx::tmem_st16(tO + cc * 16, u);
        }
        ptx::tmem_wait_st();
      }

      // P = 2^(c*s - m); a row that has seen nothing yet keeps m = -inf, and takes 0 in its place.
      const float mm = m == -INFINITY ? 0.f : m;
      const uint64_t c2 = ptx::f2pack(c, c);
      const uint64_t nm2 = ptx::f2pack(-mm, -mm);
      uint64_t acc_l[4];
      float acc_lp[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) acc_l[q] = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) acc_lp[q] = 0.f;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int i = half * 64; i < half * 64 + 64; i += 2) {
          float x0, x1;
          ptx::f2unpack(ptx::ffma2(ptx::f2pack(s[i], s[i + 1]), c2, nm2), x0, x1);
          s[i] = ptx::ex2_approx(x0);
          s[i + 1] = ptx::ex2_approx(x1);
        }
        // The P_t buffer is free once the last PV has read it.
        if (half == 0 && !pv_prev_done && !(ok = wait(S::bPVDone + t, (g - 1) & 1))) return;
#pragma unroll
        for (int ch = half * 8; ch < half * 8 + 8; ++ch) {
          uint32_t wv[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float p0 = s[8 * ch + 2 * q], p1 = s[8 * ch + 2 * q + 1];
            wv[q] = ptx::pack_bf16x2(p0, p1);
            acc_l[q] = ptx::fadd2(acc_l[q], ptx::f2pack(p0, p1));
            detail::add_bf16x2(acc_lp[2 * q], acc_lp[2 * q + 1], wv[q]);
          }
          const uint32_t addr = sP + half * S::kPRegion + r * 128 + ((static_cast<uint32_t>(ch % 8) ^ sw) << 4);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(wv[0]), "r"(wv[1]), "r"(wv[2]),
                       "r"(wv[3])
                       : "memory");
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(half == 0 ? S::bPLo + t : S::bPFull + t));
      }
      const uint64_t sl = ptx::fadd2(ptx::fadd2(acc_l[0], acc_l[1]), ptx::fadd2(acc_l[2], acc_l[3]));
      float a0, a1;
      ptx::f2unpack(sl, a0, a1);
      l += a0 + a1;
      lp += ((acc_lp[0] + acc_lp[1]) + (acc_lp[2] + acc_lp[3])) + ((acc_lp[4] + acc_lp[5]) + (acc_lp[6] + acc_lp[7]));
      --nt;
      ++g;
      ++tiles;
      left -= kBlockN;
      first = false;
    };
    // The next tile's scores; whether some row does not see it whole.
    auto next = [&](bool& mask) {
      if (!(ok = wait(S::bSFull + t, g & 1))) return false;
      ptx::tc_fence_after();
      asm volatile("ld.shared.b32 %0, [%1];"
                   : "=r"(none)
                   : "r"(sbase + S::kMasks + 4 * (tiles % kMaskRing))
                   : "memory");
      mask = __any_sync(0xffffffffu, left < kBlockN || none);
      return true;
    };
    // Two loops, so that the common tile's instructions stand together: with the masked tile's in their midst the
    // warps waited for instructions, by up to a tenth of the time.
    while (ok && nt > 0) {
      bool mask = false;
      while (nt > 0 && next(mask) && !mask) {
        work(std::integral_constant<bool, false>{});
        if (!ok) break;
      }
      if (ok && mask) work(std::integral_constant<bool, true>{});
    }
    if (!ok) break;

    // 1 / sum to the epilogue (0: no key scored above -inf), the LSE to where it goes.
    const Segment sg = segs.read();
    tiles += sg.last() - sg.end(tile);
    const float lse2 = m + log2f(l);
    if (!(ok = wait(S::bEpiTaken + t, taken))) break;  // (the first time there is nothing to wait for)
    taken ^= 1;
    reinterpret_cast<float*>(__cvta_shared_to_generic(sbase + S::kInvLp))[t * kBlockM + r] = lp == 0.f ? 0.f : 1.f / lp;
    ptx::mbar_arrive(bar(S::bEpiReady + t));
    int tok;
    if (sg.has_token(p, tile, r, tok)) {
      const int head = r - ((r * p.div_group) >> 16) * p.group;
      if (sg.kind)
        p.part_lse[(static_cast<int>(blockIdx.x) * 2 + sg.kind - 1) * kItemRows + tile * kBlockM + r] = lse2;
      else if (p.lse)
        p.lse[(sg.row0 + tok) * p.h_q + sg.h * p.group + head] = lse2 * 0.69314718055994530942f;
    }
    __syncwarp();
    if (lane == 0) segs.release();
  }
  if (!ok) raise_abort(p, sbase + S::kAbort);
}

// What the PV products left out: the infinities and NaN among the values that some rows of the item do not
// see, added to the stored output `dst` (D channels) of a row that sees `limit` keys.
template <int D, typename T>
__device__ __forceinline__ void give_back(const PrefillParams& p, const Segment& sg, uint32_t held, int limit, T* dst) {
  const int tile0 = sg.seen_by_all(p) / kBlockN;
  #pragma unroll 1
  for (int w = 0; w < 12; ++w) {
    uint32_t rows;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(rows) : "r"(held + 4 * w) : "memory");
    for (; rows; rows &= rows - 1) {
      const int key = (tile0 + w / 4) * kBlockN + (w % 4) * 32 + __ffs(rows) - 1;
      if (key >= limit) continue;
      const int page = p.table[sg.b * p.table_stride + key / p.page_size];
      if (page < 0 || page >= p.n_pages) continue;
      const __nv_bfloat16* v = p.v_cache + page * p.vs.b_ + sg.h * p.vs.h_ + (key % p.page_size) * p.vs.n_;
#pragma unroll 1
      for (int i = 0; i < D; ++i) {
        const float f = __bfloat162float(v[i]);
        if (isfinite(f)) continue;
        if constexpr (sizeof(T) == 4)
          dst[i] += f;
        else
          dst[i] = __float2bfloat16(__bfloat162float(dst[i]) + f);
      }
    }
  }
}

// O_t out of tensor memory, normalised, to the output or to the block's parts (four warps).  The stores are
// the dense kernel's: fp32 rows through two butterfly stages (8 rows x 128 bytes a store), bf16 rows as they are.
template <typename S, bool kOutF32, bool kFused>
__device__ __forceinline__ void epilogue_wg(const PrefillParams& p, uint32_t sbase, uint32_t tmem, int warp, int lane) {
  constexpr int D = S::D, kStages = S::kStages;
  auto bar = [&](int i) { return sbase + S::kBars + 8u * i; };
  const int quarter = warp & 3;
  const int r = quarter * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const float* hand = reinterpret_cast<const float*>(__cvta_shared_to_generic(sbase + S::kInvLp));
  const int r_lo = lane & 7, cgrp = lane >> 3;  // fp32 store layout after the transpose
  auto wait = [&](int b, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_or_abort(bar(b), parity, sbase + S::kAbort, p.wait_limit));
  };

  uint32_t spar = 0, gpar = 0;  // bit t: parity of O_t's segments, of their key tiles
  int ring0 = 0;         // ring index of the segment's first tile
  uint32_t fixed = 0;    // parity of V_EDGE and V_FIXED
  bool ok = true;
  Segments<S> segs(sbase);
  for (; ok; ++segs.n) {
    if (!(ok = __all_sync(~0u, segs.wait(p)))) break;
    const Segment sg = segs.read();
    if (sg.b < 0) break;
    // Between segments' outputs these warps are idle: the value tiles at the request's end, or that some rows must
    // not see, pass through their hands.
    uint32_t held = 0;  // whether something was taken out of a tile
    {
      const int n = sg.last() - sg.k0, seen = sg.seen_by_all(p);
      if (n > sg.edge(p)) {
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(segs.held() + 4 * (12 + quarter)), "r"(0) : "memory");
        if (lane < 3)
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(segs.held() + 4 * (4 * lane + quarter)), "r"(0) : "memory");
        __syncwarp();
      }
      for (int j = sg.edge(p); j < n; ++j) {
        // (The PV issuer tells when it has landed: of V_FULL's phases these warps see few, and by its parity
        // they could not tell which.)
        if (!(ok = wait(S::bVEdge, fixed))) break;
        const int s = (ring0 + v_item(j, n)) % kStages;
        const int key0 = (sg.k0 + j) * kBlockN, valid = min(sg.len - key0, kBlockN);
        const unsigned rows =
            __ballot_sync(~0u, fix_row<D, kFused>(sbase + S::kKV + s * S::kTile, r, valid, key0 + valid > seen));
        if (rows && lane == 0) {
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(segs.held() + 4 * (4 * (key0 / kBlockN - seen / kBlockN) + quarter)),
                       "r"(rows)
                       : "memory");
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(segs.held() + 4 * (12 + quarter)), "r"(1) : "memory");
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(bar(S::bVFixed));
        if (!(ok = wait(S::bVFixed, fixed))) break;  // (for the other warps' flags)
        fixed ^= 1;
      }
      if (!ok) break;
      if (n > sg.edge(p)) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t flag;
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(flag) : "r"(segs.held() + 4 * (12 + q)) : "memory");
          held |= flag;
        }
      }
      ring0 = (ring0 + 2 * n) % kStages;
    }
#pragma unroll 1
    for (int t = 0; t < S::kTiles; ++t) {
      if (!sg.present(p, t)) continue;
      const int nt = sg.end(t) - sg.k0, from = S::kOne ? segs.n & 1 : t;
      if (!(ok = wait(S::bEpiReady + from, (spar >> from) & 1))) break;
      spar ^= 1u << from;
      gpar ^= static_cast<uint32_t>(nt & 1) << from;
      const float inv_l = hand[from * kBlockM + r];
      ptx::mbar_arrive(bar(S::bEpiTaken + from));
      const bool none = inv_l == 0.f;  // the row has no key above -inf: its output is 0 whatever O_t holds
      if (nt > 0 && !(ok = wait(S::bPVDone + from, ((gpar >> from) & 1) ^ 1))) break;
      ptx::tc_fence_after();
      const uint32_t tO = tmem + 2 * kBlockN + from * D + lane_off;
      auto release_if = [&](bool last) {
        if (last && nt > 0) {  // O_t has been read: the PV issuer may start the next segment's
          ptx::tc_fence_before();
          ptx::mbar_arrive(bar(S::bOEmpty + from));
        }
      };
      // Row x of the tile (tokens and heads in turn) to its row in the output or the parts, or below 0.
      auto place = [&](int x) {
        int tok;
        if (!sg.has_token(p, t, x, tok)) return -1;
        if (sg.kind) return (static_cast<int>(blockIdx.x) * 2 + sg.kind - 1) * kItemRows + t * kBlockM + x;
        const int head = x - ((x * p.div_group) >> 16) * p.group;
        return (sg.row0 + tok) * p.h_q + sg.h * p.group + head;  // (tokens * h_q < 2^31)
      };
      if (kOutF32 || sg.kind) {
        float* const base = sg.kind ? p.part_o : static_cast<float*>(p.out);
        const bool align32 = sg.kind || p.out_align32;
        int at[4];
#pragma unroll
        for (int rr = 0; rr < 4; ++rr) at[rr] = place(quarter * 32 + rr * 8 + r_lo);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t x[32];
          ptx::tmem_ld32(tO + c * 32, x);
          ptx::tmem_wait_ld();
          release_if(c == D / 32 - 1);
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = none ? 0u : __float_as_uint(__uint_as_float(x[i]) * inv_l);
          detail::swap_lane_reg_bit<4, 4>(x, lane);
          detail::swap_lane_reg_bit<3, 3>(x, lane);
          // x[8*rr + i] = (row 32*quarter + 8*rr + r_lo, column 32*c + 8*cgrp + i)
#pragma unroll
          for (int rr = 0; rr < 4; ++rr)
            if (at[rr] >= 0)
              detail::st_global_32B(base + static_cast<size_t>(at[rr]) * D + c * 32 + cgrp * 8, align32, &x[rr * 8]);
        }
        if (held) {
          __syncwarp();
          const int mine = place(r);
          if (mine >= 0 && !none)
            give_back<D>(p, sg, segs.held(), sg.limit(p, t, r), base + static_cast<size_t>(mine) * D);
        }
      } else if constexpr (!kOutF32) {
        const int mine = place(r);
        __nv_bfloat16* const dst = static_cast<__nv_bfloat16*>(p.out) + static_cast<long long>(mine) * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t a[32];
          ptx::tmem_ld32(tO + c * 32, a);
          ptx::tmem_wait_ld();
          release_if(c == D / 32 - 1);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            a[i] = none ? 0u
                        : ptx::pack_bf16x2(__uint_as_float(a[2 * i]) * inv_l, __uint_as_float(a[2 * i + 1]) * inv_l);
          if (mine >= 0) {
            detail::st_global_32B(dst + c * 32, p.out_align32, &a[0]);
            detail::st_global_32B(dst + c * 32 + 16, p.out_align32, &a[8]);
          }
        }
        if (held && mine >= 0 && !none) give_back<D>(p, sg, segs.held(), sg.limit(p, t, r), dst);
      }
    }
    if (!ok) break;
    __syncwarp();
    if (lane == 0) segs.release();
  }
  if (!ok) raise_abort(p, sbase + S::kAbort);
}

template <int kD, bool kOne, bool kOutF32, bool kFused>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ PrefillParams p) {
  using S = Smem<kD, kOne>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = ptx::smem_addr(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    auto bar = [&](int i) { return sbase + S::kBars + 8u * i; };
    for (int s = 0; s < S::kQTurns; ++s) {
      ptx::mbar_init(bar(S::bQFull + s), 1);
      ptx::mbar_init(bar(S::bQEmpty + s), 1);
    }
    for (int s = 0; s < S::kStages; ++s) {
      ptx::mbar_init(bar(S::bKFull + s), 1);
      ptx::mbar_init(bar(S::bVFull + s), 1);
      ptx::mbar_init(bar(S::bKVEmpty + s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(bar(S::bSFull + t), 1);
      ptx::mbar_init(bar(S::bSEmpty + t), S::kRows);
      ptx::mbar_init(bar(S::bPFull + t), S::kRows);
      ptx::mbar_init(bar(S::bPLo + t), S::kRows);
      ptx::mbar_init(bar(S::bPVDone + t), 1);
      ptx::mbar_init(bar(S::bOEmpty + t), kBlockM);
      ptx::mbar_init(bar(S::bEpiReady + t), S::kRows);
      ptx::mbar_init(bar(S::bEpiTaken + t), kBlockM);
    }
    for (int s = 0; s < kSegs; ++s) {
      ptx::mbar_init(bar(S::bSegFull + s), 1);
      ptx::mbar_init(bar(S::bSegEmpty + s), kConsumers);
    }
    ptx::mbar_init(bar(S::bVEdge), 1);
    ptx::mbar_init(bar(S::bVFixed), kBlockM);
    ptx::mbar_init(bar(S::bDrainS), 1);
    ptx::mbar_init(bar(S::bDrainPV), 1);
    *reinterpret_cast<volatile int*>(smem + S::kAbort) = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    ptx::tma_prefetch_desc(&p.tm_q);
    ptx::tma_prefetch_desc(&p.tm_k);
    ptx::tma_prefetch_desc(&p.tm_v);
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(sbase + S::kTmemSlot, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + S::kTmemSlot);
  wait_for_inputs_and_copies();

  using Regs = RegSplit<false>;
  // (The order of the code counts: with the softmax's first, or the scheduler behind the issuers, 27280 tokens take 2 %
  // longer, 4608 on 27280 keys up to 5.)
  if (warp >= kLoadWarp && warp < kEpiWarp0) {
    ptx::setmaxnreg_dec<Regs::kIssue>();
    if (warp == kScheduleWarp) {
      scheduler<S>(p, sbase, lane);
    } else if (warp == kLoadWarp) {
      producer<S, kFused>(p, sbase, lane);
    } else if (warp == kMmaWarp) {
      if (lane == 0) s_issuer<S, kFused>(p, sbase, tmem);
    } else if (warp == kPvWarp) {
      if (lane == 0) pv_issuer<S, kFused>(p, sbase, tmem);
    }
    __syncwarp();
  } else if (warp < kLoadWarp) {
    ptx::setmaxnreg_inc<Regs::kSoftmax>();
    softmax_wg<S>(p, sbase, tmem, warp >> 2, warp, lane);
  } else if (warp >= kEpiWarp0) {
    ptx::setmaxnreg_dec<Regs::kEpilogue>();
    epilogue_wg<S, kOutF32, kFused>(p, sbase, tmem, warp, lane);
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

constexpr int kJoinRows = 8;  // rows (warps) of a join block

// The items that more than one block worked on: a row's parts, each normalised with its lse, in the order of
// the blocks, weighted by 2^(lse - max).
template <int D, bool kOutF32>
__global__ void __launch_bounds__(kJoinRows * 32) join_kernel(const __grid_constant__ PrefillParams p) {
  wait_for_inputs();
  const int4 m = p.meta[blockIdx.x];
  if (m.w == 0) return;
  const int lane = threadIdx.x & 31, row = blockIdx.y * kJoinRows + (threadIdx.x >> 5);
  const int t = row / kBlockM, r = row % kBlockM;
  const int i = (r * p.div_group) >> 16, tok = t * p.tile_tokens + i;
  if (i >= p.tile_tokens || tok >= m.y) return;
  // Part 0 is the first block's slot 1, part n the n-th next block's slot 0.
  auto part = [&](int n) { return (static_cast<size_t>(blockIdx.x + n) * 2 + (n == 0)) * kItemRows + row; };
  constexpr int kV = D / 32;
  float top = -INFINITY;
  for (int n = lane; n < m.w; n += 32) top = fmaxf(top, p.part_lse[part(n)]);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if (top == -INFINITY) top = 0.f;  // (no part has a key, or all are NaN, which their weights show)
  float acc[kV] = {}, sum = 0.f;
  for (int n0 = 0; n0 < m.w; n0 += 32) {
    const int mine = n0 + lane;
    // Below 0: the part has no key above -inf for this row, and counts for nothing.  (A weight that rounds to
    // 0 still shows what is not finite.)
    float w = mine < m.w ? p.part_lse[part(mine)] : -INFINITY;
    w = w == -INFINITY ? -1.f : exp2f(w - top);
    const int end = min(32, m.w - n0);
#pragma unroll 4
    for (int n = 0; n < end; ++n) {
      const float wn = __shfl_sync(~0u, w, n);
      const float* o = p.part_o + part(n0 + n) * D + lane * kV;
      float x[kV];
#pragma unroll
      for (int q = 0; q < kV; ++q) x[q] = o[q];
      if (wn < 0.f) continue;
      sum += wn;
#pragma unroll
      for (int q = 0; q < kV; ++q) acc[q] = fmaf(wn, x[q], acc[q]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const size_t at = static_cast<size_t>(m.x + tok) * p.h_q + m.z * p.group + (r - i * p.group);
  if (p.lse && lane == 0) p.lse[at] = (top + log2f(sum)) * 0.69314718055994530942f;
  if constexpr (kOutF32) {
    float* dst = static_cast<float*>(p.out) + at * D + lane * kV;
#pragma unroll
    for (int q = 0; q < kV; ++q) dst[q] = acc[q] * inv;
  } else {
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + at * D + lane * kV);
#pragma unroll
    for (int q = 0; q < kV; q += 2) dst[q / 2] = ptx::pack_bf16x2(acc[q] * inv, acc[q + 1] * inv);
  }
}

}  // namespace prefill
}  // namespace ditattn
