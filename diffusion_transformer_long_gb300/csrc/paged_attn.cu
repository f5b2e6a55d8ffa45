// Attention of one new token of each request over its paged keys and values:
//   s_j = scale q . k_j,  m = max s_j,  l = sum exp(s_j - m),  o = sum exp(s_j - m) v_j / l,
//   lse = m + ln l.
//
// One block per (request, query head); the warps take the keys in turn, a lane holds D / 32
// channels of the running output, and the warps' states are joined at the end.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "paged_launch.h"
#include "sm103_ptx.cuh"

namespace ditattn {
namespace {

constexpr int kWarps = 4;

struct PagedParams {
  PagedAttnLaunch a;
};

template <int D, typename OT>
__global__ void __launch_bounds__(kWarps * 32) paged_attn_simple(const PagedParams p) {
  constexpr int kC = D / 32;  // channels of a lane
  __shared__ float sm_o[kWarps][D], sm_m[kWarps], sm_l[kWarps];
  const PagedAttnLaunch& a = p.a;
  const int b = blockIdx.x / a.h_q, h = blockIdx.x % a.h_q, hk = h / (a.h_q / a.h_kv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = a.page_size;
  const int len = min(max(0, a.seq_lens[b]), a.max_pages * P);
  const int pages = pages_of(len, P);
  const int entries = a.selected ? min(pages, a.n_selected) : pages;
  const int* sel = a.selected ? a.selected + (static_cast<long long>(b) * a.h_kv + hk) * a.n_selected : nullptr;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + b * a.q_b + h * a.q_h;
  float qr[kC], o[kC], m = -INFINITY;
  double l = 0.0;  // thousands of like terms in turn: 32 bits would lose 2^-24 of the sum at each
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    qr[i] = __bfloat162float(q[lane + 32 * i]);
    o[i] = 0.f;
  }
  for (int e = 0; e < entries; ++e) {
    const int i = sel ? sel[e] : e;
    if (i < 0 || i >= pages) continue;
    const int page = a.table[b * a.table_stride + i];
    if (page < 0 || page >= a.n_pages) continue;
    const int rows = min(P, len - i * P);
    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k_cache) + page * a.ks.b_ + hk * a.ks.h_;
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v_cache) + page * a.vs.b_ + hk * a.vs.h_;
    for (int r = warp; r < rows; r += kWarps) {
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < kC; ++c) s = fmaf(qr[c], __bfloat162float(k[r * a.ks.n_ + lane + 32 * c]), s);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
      s *= a.scale;
      const float mn = fmaxf(m, s);
      const float base = mn == -INFINITY ? 0.f : mn;
      const float f = expf(m - base), w = expf(s - base);
      m = mn;
      l = l * f + w;
#pragma unroll
      for (int c = 0; c < kC; ++c) o[c] = fmaf(w, __bfloat162float(v[r * a.vs.n_ + lane + 32 * c]), o[c] * f);
    }
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = static_cast<float>(l);
  }
#pragma unroll
  for (int c = 0; c < kC; ++c) sm_o[warp][lane + 32 * c] = o[c];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w]);
  const float base = M == -INFINITY ? 0.f : M;
  for (int w = 0; w < kWarps; ++w) L += sm_l[w] * expf(sm_m[w] - base);
  for (int d = threadIdx.x; d < D; d += kWarps * 32) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += sm_o[w][d] * expf(sm_m[w] - base);
    static_cast<OT*>(a.out)[(static_cast<long long>(b) * a.h_q + h) * D + d] = static_cast<OT>(L == 0.f ? 0.f : x / L);
  }
  if (a.lse && threadIdx.x == 0) a.lse[static_cast<long long>(b) * a.h_q + h] = base + logf(L);
}

}  // namespace

size_t paged_attn_workspace(int, int, int d) { return 512 * 2 * 16 * (static_cast<size_t>(d) + 2) * 4; }

cudaError_t launch_paged_attn(const PagedAttnLaunch& a, cudaStream_t st) {
  PagedParams p{a};
  const unsigned grid = static_cast<unsigned>(a.batch) * a.h_q;
  if (a.d == 64) {
    if (a.out_f32) paged_attn_simple<64, float><<<grid, kWarps * 32, 0, st>>>(p);
    else paged_attn_simple<64, __nv_bfloat16><<<grid, kWarps * 32, 0, st>>>(p);
  } else {
    if (a.out_f32) paged_attn_simple<128, float><<<grid, kWarps * 32, 0, st>>>(p);
    else paged_attn_simple<128, __nv_bfloat16><<<grid, kWarps * 32, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace ditattn
