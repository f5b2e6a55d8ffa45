// Host side of the attention of new tokens over a paged cache: tensor maps, the workspace, the launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "attn_host.cuh"
#include "paged_maps.cuh"
#include "paged_prefill_kernel.cuh"

namespace ditattn {

using namespace prefill;

namespace {

// Requests with room for at most this many keys keep their items whole: one launch and no workspace.
constexpr long long kWholeKeys = 1024;
// SM clocks that a key tile of an item may take, some five times what it does (2.0 us): with the limit of a single step's
// wait alone, items of more than 10^8 keys ran out of it.
constexpr long long kTileClocks = 20000;
// Items are of one Q tile of 64 rows where the step's rows (tokens x heads of a group) fill at most 1 / kOneShare of a
// whole tile a request (16 tokens, 24 heads on 8, 64 requests of 100-4096 keys: 128 us, of two tiles 145; 30 tokens, more than
// one such item a request: 194 and 154).
constexpr long long kOneShare = 2;

// A paged cache's map of fused copies of `rows` rows (see KvTile); false: the strides do not allow one.
bool encode_fused(CUtensorMap* m, KvPlace* kv, const void* base, const Strides& s, int d, int page_size, int heads,
                  int n_pages, int rows) {
  constexpr long long kMost = 1LL << 31;  // coordinates, and steps between them, are 32-bit numbers
  const int groups = page_size / 8;
  if (d != 128) return false;
  long long apart = s.b_ / s.h_;
  if (s.b_ % s.h_ == 0 && apart >= heads && apart * n_pages + heads < kMost) {
    *kv = {1, static_cast<int>(apart)};
    if (maps::encode<5>(m, base, {64, 8, d / 64, groups, (n_pages - 1) * apart + heads}, {s.n_, 64, 8 * s.n_, s.h_},
                  {64, 8, d / 64, rows / 8, 1}))
      return true;
  }
  apart = s.b_ / (8 * s.n_);
  if (s.b_ % (8 * s.n_) != 0 || apart < groups || apart * n_pages + groups >= kMost) return false;
  *kv = {0, static_cast<int>(apart)};
  return maps::encode<5>(m, base, {64, 8, d / 64, (n_pages - 1) * apart + groups, heads}, {s.n_, 64, 8 * s.n_, s.h_},
                   {64, 8, d / 64, rows / 8, 1});
}

// Sets the shared-memory opt-in once per device and instantiation.
template <int D, bool kOne, bool kF32, bool kFused>
cudaError_t prepare() {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!done[dev]) {
    e = cudaFuncSetAttribute(prefill_kernel<D, kOne, kF32, kFused>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D, kOne>::kBytes);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  return cudaSuccess;
}

template <int D, bool kOne, bool kF32, bool kFused>
cudaError_t launch(const PrefillParams& p, int blocks, cudaStream_t st) {
  cudaError_t e = prepare<D, kOne, kF32, kFused>();
  if (e != cudaSuccess) return e;
  e = launch_after(prefill_kernel<D, kOne, kF32, kFused>, dim3(blocks), dim3(kThreads), Smem<D, kOne>::kBytes, st, p);
  if (e != cudaSuccess || !p.split) return e;
  const int rows = std::min(p.tokens, p.item_tokens) <= p.tile_tokens ? std::min(p.tokens, p.tile_tokens) * p.group : kItemRows;
  return launch_after(join_kernel<D, kF32>, dim3(blocks, (rows + kJoinRows - 1) / kJoinRows), dim3(kJoinRows * 32), 0,
                      st, p);
}

int grid_blocks() {
  const int blocks = std::min(kMaxGrid, host::sm_count());
  return grid_limit() > 0 ? std::min(blocks, grid_limit()) : blocks;
}

// Rows of the parts that the workspace holds: two items a block.
size_t part_rows() { return static_cast<size_t>(std::min(kMaxGrid, host::sm_count())) * 2 * kItemRows; }

}  // namespace

size_t paged_prefill_workspace(int d, long long keys) {
  if (keys <= kWholeKeys) return 0;
  return part_rows() * (d + 1) * 4 + kMaxGrid * sizeof(int4);
}

cudaError_t launch_paged_prefill(const PrefillLaunch& a, cudaStream_t st) {
  PrefillParams p;
  p.group = a.h_q / a.h_kv;
  const bool one = static_cast<long long>(a.tokens) * p.group * kOneShare <= static_cast<long long>(a.batch) * kBlockM &&
                   p.group <= Smem<64, true>::kRows;
  p.tile_tokens = (one ? Smem<64, true>::kRows : kBlockM) / p.group;
  p.item_tokens = (one ? 1 : 2) * p.tile_tokens;
  p.box_rows = maps::box_rows(a.page_size);
  if (!maps::encode_queries(&p.tm_q, a.q, a.q_n, a.q_h, a.d, p.group, a.tokens, a.h_kv, p.tile_tokens))
    return cudaErrorInvalidValue;
  // Copies of 16 rows are fused in pages of long requests: the copies' number bounds them (54560 keys, one head: 970
  // and 1197 us; 4 x 9024, 24 heads on 8: 387 and 415).  For short ones a fused copy's longer way counts (16 x 2512: 309
  // and 296; 8 x 5024: 463 and 465), and of larger runs there are few enough (runs of 128: 1032 and 927 us).
  const bool fused = p.box_rows == 16 && static_cast<long long>(a.max_pages) * a.page_size > 5120 &&
      encode_fused(&p.tm_k, &p.kv[0], a.k_cache, a.ks, a.d, a.page_size, a.h_kv, a.n_pages, p.box_rows) &&
      encode_fused(&p.tm_v, &p.kv[1], a.v_cache, a.vs, a.d, a.page_size, a.h_kv, a.n_pages, p.box_rows);
  if (!fused && (!maps::encode_rows(&p.tm_k, a.k_cache, a.ks, a.d, a.page_size, a.h_kv, a.n_pages, p.box_rows) ||
                 !maps::encode_rows(&p.tm_v, a.v_cache, a.vs, a.d, a.page_size, a.h_kv, a.n_pages, p.box_rows)))
    return cudaErrorInvalidValue;
  p.v_cache = static_cast<const __nv_bfloat16*>(a.v_cache);
  p.vs = a.vs;
  p.table = a.table;
  p.table_stride = a.table_stride;
  p.seq_lens = a.seq_lens;
  p.cu_new = a.cu_new;
  p.start_lens = a.start_lens;
  p.out = a.out;
  p.out_align32 = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
  p.lse = a.lse;
  p.batch = a.batch;
  p.tokens = a.tokens;
  p.h_q = a.h_q;
  p.h_kv = a.h_kv;
  p.page_size = a.page_size;
  p.n_pages = a.n_pages;
  p.max_len = a.max_pages * a.page_size;
  p.div_group = (65536 + p.group - 1) / p.group;
  p.causal = a.causal;
  p.key_bytes = static_cast<int>(std::min<long long>(4LL * a.h_kv * a.d, 1 << 30));
  p.split = p.max_len > kWholeKeys;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.status = a.status;
  stall_injection(&p.stall, &p.wait_limit);
  // Some waits last a whole item: the epilogue's for its sums, the idle softmax's for the next, the ring's for a place.
  p.wait_limit += static_cast<long long>(p.max_len / kBlockN) * kTileClocks;
  p.part_o = static_cast<float*>(a.workspace);
  p.part_lse = p.part_o + part_rows() * a.d;
  p.meta = reinterpret_cast<int4*>(p.part_lse + part_rows());
  const int blocks = grid_blocks();
  auto run = [&](auto d, auto fused_copies) {
    constexpr int D = decltype(d)::value;
    constexpr bool kFused = decltype(fused_copies)::value;
    if (one) return a.out_f32 ? launch<D, true, true, kFused>(p, blocks, st) : launch<D, true, false, kFused>(p, blocks, st);
    return a.out_f32 ? launch<D, false, true, kFused>(p, blocks, st) : launch<D, false, false, kFused>(p, blocks, st);
  };
  if (a.d == 64) return run(std::integral_constant<int, 64>{}, std::false_type{});
  return fused ? run(std::integral_constant<int, 128>{}, std::true_type{})
               : run(std::integral_constant<int, 128>{}, std::false_type{});
}

}  // namespace ditattn
