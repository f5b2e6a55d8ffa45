// Host side of the paged attention: tensor maps, the choice of the launch, and the launch whose items
// are dealt out over the blocks.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "attn_host.cuh"
#include "paged_attn_kernel.cuh"

namespace ditattn {

using namespace paged;

namespace {

// 5-D map (64 channels, row, channel block, head, page) of a paged cache: boxes of 16 rows x D.
bool encode_cache(CUtensorMap* m, const void* base, const Strides& s, int d, int page_size, int heads, int n_pages) {
  const cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(page_size), static_cast<cuuint64_t>(d / 64),
                              static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(n_pages)};
  const cuuint64_t strides[4] = {static_cast<cuuint64_t>(s.n_) * 2, 128, static_cast<cuuint64_t>(s.h_) * 2,
                                 static_cast<cuuint64_t>(s.b_) * 2};
  const cuuint32_t box[5] = {64, kTile, static_cast<cuuint32_t>(d / 64), 1, 1};
  const cuuint32_t elem[5] = {1, 1, 1, 1, 1};
  EncodeTiledFn fn = tensor_map_encoder();
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, elem,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query heads that share one pass over the keys: the group's, in eights, up to 32.
int row_block(int group) { return std::min((group + 7) / 8 * 8, kMaxRows); }

// Few short items get a cluster of blocks each: against the runs, 8 items of 1024 keys 4.9 and 7.4 us, of
// 4096 keys 8.5 and 9.2, of 8192 keys 14.2 and 12.0.  So does one request whose heads' clusters fill
// most of the GPU (24 heads, 32768 keys: 63.0 and 65.8 us); several may be of very different lengths.
bool few_items(int batch, int h_q, int h_kv, long long keys) {
  const int group = h_q / h_kv, R = row_block(group);
  const long long blocks = static_cast<long long>(batch) * h_kv * ((group + R - 1) / R) * kCluster;
  const int slots = 2 * host::sm_count();  // two blocks fit an SM (registers, 82 to 92 KB of shared memory)
  return grid_limit() == 0 && blocks <= slots && (keys <= 4096 || (batch == 1 && 5 * blocks >= 3 * slots));
}

}  // namespace

// Partials of two segments of each block: fp32 sums, (maximum, sum) pairs, and the join's notes.
// Clusters need none.
size_t paged_attn_workspace(int batch, int h_q, int h_kv, int d, long long keys) {
  if (few_items(batch, h_q, h_kv, keys)) return 0;
  const size_t rows = static_cast<size_t>(kMaxBlocks) * 2 * row_block(h_q / h_kv);
  return rows * d * 4 + rows * 8 + kMaxBlocks * 16;
}

cudaError_t launch_paged_attn(const PagedAttnLaunch& a, cudaStream_t st) {
  PagedParams p;
  if (!encode_cache(&p.tm_k, a.k_cache, a.ks, a.d, a.page_size, a.h_kv, a.n_pages) ||
      !encode_cache(&p.tm_v, a.v_cache, a.vs, a.d, a.page_size, a.h_kv, a.n_pages))
    return cudaErrorInvalidValue;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.q_b = a.q_b;
  p.q_h = a.q_h;
  p.table = a.table;
  p.table_stride = a.table_stride;
  p.seq_lens = a.seq_lens;
  p.selected = a.selected;
  p.n_selected = a.n_selected;
  p.out = a.out;
  p.lse = a.lse;
  p.batch = a.batch;
  p.h_q = a.h_q;
  p.h_kv = a.h_kv;
  p.group = a.h_q / a.h_kv;
  const int R = row_block(p.group);
  p.head_blocks = (p.group + R - 1) / R;
  p.page_size = a.page_size;
  p.page_tiles = a.page_size / kTile;
  p.n_pages = a.n_pages;
  p.max_len = a.max_pages * a.page_size;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.status = a.status;
  stall_injection(&p.stall, &p.wait_limit);
  const size_t rows = static_cast<size_t>(kMaxBlocks) * 2 * R;
  p.part_o = static_cast<float*>(a.workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + rows * a.d);
  p.meta = reinterpret_cast<int4*>(p.part_ml + rows);
  if (few_items(a.batch, a.h_q, a.h_kv, static_cast<long long>(a.selected ? a.n_selected : a.max_pages) * a.page_size))
    return launch_few(p, a.d, R, a.out_f32, a.batch * a.h_kv * p.head_blocks, st);
  int blocks = std::min(kMaxBlocks, 2 * host::sm_count());
  if (grid_limit() > 0) blocks = std::min(blocks, grid_limit());
  return for_sizes(a.d, R, a.out_f32, [&](auto D, auto nb, auto zero) {
    using OT = decltype(zero);
    cudaError_t e = prepare_kernel<D(), nb(), OT, false>();
    if (e != cudaSuccess) return e;
    e = launch_after(paged_attn_kernel<D(), nb(), OT, false>, dim3(blocks), dim3(kThreadsPaged),
                     PagedSmem<D()>::bytes(nb()), st, p);
    if (e != cudaSuccess) return e;
    return launch_after(paged_join_kernel<D(), nb(), OT>, dim3(blocks, std::min(p.group, R)), dim3(128), 0, st, p);
  });
}

}  // namespace ditattn
