// Host side of the attention of new tokens over a paged cache: tensor maps, the workspace, the launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "attn_host.cuh"
#include "paged_prefill_kernel.cuh"

namespace ditattn {

using namespace prefill;

namespace {

// Requests with room for at most this many keys keep their items whole: one launch and no workspace.
constexpr long long kWholeKeys = 1024;

bool encode(CUtensorMap* m, const void* base, const cuuint64_t (&dims)[4], const long long (&strides)[3],
            int box1, int box2) {
  EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t st[3];
  for (int i = 0; i < 3; ++i) st[i] = static_cast<cuuint64_t>(strides[i]) * 2;
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box1), static_cast<cuuint32_t>(box2), 1};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, st, box, elem,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// (D, row, head, page) of a paged cache: boxes of `rows` rows x 64 channels.
bool encode_cache(CUtensorMap* m, const void* base, const Strides& s, int d, int page_size, int heads, int n_pages,
                  int rows) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(page_size),
                              static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(n_pages)};
  return encode(m, base, dims, {s.n_, s.h_, s.b_}, rows, 1);
}

// Sets the shared-memory opt-in once per device and instantiation.
template <int D, bool kF32>
cudaError_t prepare() {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!done[dev]) {
    e = cudaFuncSetAttribute(prefill_kernel<D, kF32>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  return cudaSuccess;
}

template <int D, bool kF32>
cudaError_t launch(const PrefillParams& p, int blocks, cudaStream_t st) {
  cudaError_t e = prepare<D, kF32>();
  if (e != cudaSuccess) return e;
  e = launch_after(prefill_kernel<D, kF32>, dim3(blocks), dim3(kThreads), Smem<D>::kBytes, st, p);
  if (e != cudaSuccess || !p.split) return e;
  const int rows = p.tokens <= p.tile_tokens ? p.tokens * p.group : kItemRows;
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
  p.tile_tokens = kBlockM / p.group;
  p.box_rows = 16;
  while (p.box_rows < kBlockN && a.page_size % (2 * p.box_rows) == 0) p.box_rows *= 2;
  const cuuint64_t qdims[4] = {static_cast<cuuint64_t>(a.d), static_cast<cuuint64_t>(p.group),
                               static_cast<cuuint64_t>(a.tokens), static_cast<cuuint64_t>(a.h_kv)};
  if (!encode(&p.tm_q, a.q, qdims, {a.q_h, a.q_n, a.q_h * p.group}, p.group, p.tile_tokens) ||
      !encode_cache(&p.tm_k, a.k_cache, a.ks, a.d, a.page_size, a.h_kv, a.n_pages, p.box_rows) ||
      !encode_cache(&p.tm_v, a.v_cache, a.vs, a.d, a.page_size, a.h_kv, a.n_pages, p.box_rows))
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
  p.split = p.max_len > kWholeKeys;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.status = a.status;
  stall_injection(&p.stall, &p.wait_limit);
  p.part_o = static_cast<float*>(a.workspace);
  p.part_lse = p.part_o + part_rows() * a.d;
  p.meta = reinterpret_cast<int4*>(p.part_lse + part_rows());
  const int blocks = grid_blocks();
  if (a.d == 64) return a.out_f32 ? launch<64, true>(p, blocks, st) : launch<64, false>(p, blocks, st);
  return a.out_f32 ? launch<128, true>(p, blocks, st) : launch<128, false>(p, blocks, st);
}

}  // namespace ditattn
