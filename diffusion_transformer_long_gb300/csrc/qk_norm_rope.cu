// Norms of queries and keys for each head, with rotary positions, in one pass.
//
//   r = 1 / sqrt(mean_d x_d^2 + eps),  z_d = w_d r x_d
//   pair i of the first 2 n channels, (2 i, 2 i + 1) or (i, i + n), at angle t_i = pos_a(i) f_i:
//     y_first = s (z_first cos t_i - z_second sin t_i),  y_second = s (z_first sin t_i + z_second cos t_i)
// Each value is read and written once: bound by HBM (75600 tokens, 40 + 40 heads of 128, token-major to
// head-major: 505 us, 6.1 TB/s; half-and-half pairs in place of interleaved ones 487 us, 6.4; a copy's rate is 6.8).
//
// A lane holds two 16-byte pieces of a head, of 8 channels each, so that a warp takes four heads of 128 or eight of 64 at
// a step (queries, then keys), and a pair's channels are in one lane: neighbours in a piece, or the pieces i and
// i + n / 8.  Every warp walks over tokens by itself, the loads of kIters steps ahead of its arithmetic (the next
// token's first ones before its angles), and no barrier holds it up: with a block's warps on one token and its angles
// shared behind a barrier, 75600 tokens took 1370 us; with one piece a lane and the other of a pair by a shuffle,
// 600 us, bound by the instructions.  It works the token's cosines and sines out into shared memory, and folds them with
// the weights into two factors a channel, y = r (A x + B x'), with x' the pair's other channel.  Where there are few
// tokens several warps take one, a part of its heads each.
//
// The angle is exact whatever the position: a position is a whole number, so that f_i in turns need only be
// known modulo 1, and as a 64-bit fraction its product with the position wraps by itself.  The phase is then off by
// at most |pos| (2^-64 + |f_i| 2^-95) turns, and rounded to 32 bits once.  (In 32-bit floats position 75600 is off by 0.004 of a
// radian.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attn_host.cuh"
#include "paged_device.cuh"
#include "paged_launch.h"
#include "sm103_ptx.cuh"

namespace ditattn {
namespace {

constexpr int kIters = 4;   // steps of a warp whose loads are in flight at once
constexpr int kWarps = 8;   // of a block
constexpr int kBlocks = 2;  // of an SM

struct Side {
  const __nv_bfloat16* in;
  __nv_bfloat16* out;
  Strides is, os;
  const void* weight;  // null: 1
  int heads;
};

struct RopeParams {
  Side side[2];  // queries, keys
  int weight_f32, norm;
  float eps;
  const int* positions;  // [axes][..]: positions[b pos_b + a pos_axis + n], or null
  long long pos_b, pos_axis;
  const int* cu_new;  // packed requests: position start_lens[r] + n - cu_new[r]
  const int* start_lens;
  int requests;
  const float* freqs;
  int pairs;           // 0: no rotation
  int axis_end[4];     // pairs up to the end of each axis
  float rot_scale;
  int batch, n;        // tokens of each batch
  int parts;           // warps of a token
};

// f in turns, modulo 1, as a 64-bit fraction: |f| = m 2^e with m of 24 bits, and 1 / (2 pi) as a fraction of 96
// bits.  Cut off, not rounded: below the exact fraction by less than 2^-64 + |f| 2^-95.
// (For finite f.)
__device__ __forceinline__ uint64_t turns(float f) {
  constexpr unsigned __int128 kInverse2Pi =
      (static_cast<unsigned __int128>(0x28be60dbULL) << 64) | 0x9391054a7f09d5f4ULL;
  const uint32_t bits = __float_as_uint(f);
  const int exponent = (bits >> 23) & 255;
  const uint32_t m = (bits & 0x7fffffu) | (exponent ? 0x800000u : 0u);
  const unsigned __int128 x = kInverse2Pi * m;         // m / (2 pi) 2^96
  const int shift = 32 - (max(exponent, 1) - 150);     // to a multiple of 2^-64, times 2^e
  const uint64_t t = shift >= 128 ? 0 : shift >= 0 ? static_cast<uint64_t>(x >> shift)
                                                   : shift > -64 ? static_cast<uint64_t>(x) << -shift : 0;
  return bits >> 31 ? 0 - t : t;
}

// The request that holds packed token n, or below 0: the last whose first token is at or before it.  (One warp.)
__device__ __forceinline__ int request_of(const RopeParams& p, int n, int lane) {
  int lo = 0, count = p.requests;  // among [lo, lo + count)
  while (count > 0) {
    const int step = (count + 31) / 32;
    const int at = lo + lane * step;
    const bool before = lane * step < count && p.cu_new[at] <= n;
    const unsigned some = __ballot_sync(~0u, before);
    if (some == 0) return -1;
    const int last = 31 - __clz(some);
    lo += last * step;
    if (step == 1) break;
    count = min(step, count - last * step);
  }
  return n < p.cu_new[lo + 1] ? lo : -1;
}

// kWhole: all channels turn.
template <int D, bool kInterleaved, bool kWhole>
__global__ void __launch_bounds__(kWarps * 32, kBlocks) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kLanes = D / 16, kHeads = 32 / kLanes;  // lanes of a head, heads of a warp's step
  __shared__ uint64_t step_turns[64];                   // the pairs' turns a position
  __shared__ float size[64];                            // their scale (NaN where the frequency is not finite)
  __shared__ float2 turn[kWarps][64];                   // (cos, sin) of the pairs at each warp's token, scaled
  __shared__ float weights[2][D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int l = lane % kLanes, sub = lane / kLanes;
  const int turning = p.pairs / 8;  // pieces of first channels
  // The lane's pieces: the two of its pairs (not interleaved), or any two.
  const int piece0 = kInterleaved || l < turning ? l : 2 * l;
  const int piece1 = kInterleaved ? l + kLanes : l < turning ? l + turning : 2 * l + 1;
  const bool rotated[2] = {piece0 < 2 * turning, piece1 < 2 * turning};
  const int heads = p.side[0].heads + p.side[1].heads, steps = (heads + kHeads - 1) / kHeads;
  const unsigned units = static_cast<unsigned>(p.batch) * p.n * p.parts, stride = gridDim.x * kWarps;
  unsigned unit = blockIdx.x * kWarps + warp;
  int b, n, part;  // of the unit
  auto split = [&](unsigned u) {
    const unsigned token = p.parts == 1 ? u : u / p.parts;
    part = static_cast<int>(u - token * p.parts);
    b = p.batch == 1 ? 0 : static_cast<int>(token / p.n);
    n = static_cast<int>(token - static_cast<unsigned>(b) * p.n);
  };
  // The lane's walk over its heads at the token (all queries' before the keys'), for loads or for stores.
  struct Walk {
    int head;       // of both
    int side;
    char* at;       // the head's first channel
    int64_t apart;  // bytes to the next head
  };
  auto place = [&](Walk& w, bool out) {
    w.side = w.head >= p.side[0].heads;
    const Side& s = p.side[w.side];
    const Strides& st = out ? s.os : s.is;
    const int h = w.head - (w.side ? p.side[0].heads : 0);
    w.at = reinterpret_cast<char*>(out ? s.out : const_cast<__nv_bfloat16*>(s.in)) + 2 * (b * st.b_ + n * st.n_ + h * st.h_);
    w.apart = 2 * p.parts * kHeads * st.h_;
  };
  auto advance = [&](Walk& w, bool out) {
    w.head += p.parts * kHeads;
    w.at += w.apart;
    if (w.side == 0 && w.head >= p.side[0].heads && w.head < heads) place(w, out);
  };
  Walk ld = {}, sd = {};
  uint4 x[kIters][2];
  auto load = [&](uint4 (&y)[2]) {
    if (ld.head < heads) {
      y[0] = load_once(ld.at + 16 * piece0);
      y[1] = load_once(ld.at + 16 * piece1);
      advance(ld, false);
    }
  };
  auto load_first = [&]() {
    ld.head = part * kHeads + sub;
    if (ld.head < heads) place(ld, false);
#pragma unroll
    for (int i = 0; i < kIters; ++i) load(x[i]);
  };
  // Lane a: the token's position on axis a; packed: each lane's is that of the one axis.
  auto position = [&](bool& live) -> long long {
    live = true;
    if (p.pairs == 0) return 0;
    if (!p.cu_new) {
      const bool has = lane == 0 || (lane < 4 && p.axis_end[lane - 1] < p.pairs);
      return has ? p.positions[b * p.pos_b + lane * p.pos_axis + n] : 0;
    }
    const int r = request_of(p, n, lane);
    live = r >= 0;
    return live ? static_cast<long long>(p.start_lens[r]) + n - p.cu_new[r] : 0;
  };

  wait_for_inputs();
  bool live = false;
  long long at = 0;
  if (unit < units) {
    split(unit);
    load_first();
    at = position(live);
  }
  if (threadIdx.x < p.pairs) {
    const float f = p.freqs[threadIdx.x];
    step_turns[threadIdx.x] = turns(f);
    size[threadIdx.x] = isfinite(f) ? p.rot_scale : __int_as_float(0x7fffffff);
  }
  for (int i = threadIdx.x; i < 2 * D; i += kWarps * 32) {
    const Side& s = p.side[i / D];
    const int d = i % D;
    weights[i / D][d] = !s.weight ? 1.f
                        : p.weight_f32 ? static_cast<const float*>(s.weight)[d]
                                       : __bfloat162float(static_cast<const __nv_bfloat16*>(s.weight)[d]);
  }
  __syncthreads();

  while (unit < units) {
    if (live) {
      for (int i = lane; i - lane < p.pairs; i += 32) {
        int axis = 0;
#pragma unroll
        for (int a = 0; a < 3; ++a) axis += i >= p.axis_end[a];
        const long long mine = __shfl_sync(~0u, at, p.cu_new ? 0 : axis & 3);
        if (i < p.pairs) {
          const uint64_t phase = static_cast<uint64_t>(mine) * step_turns[i] + 0x80000000u;
          float c, s;
          sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 0x1p-31f, &s, &c);
          turn[warp][i] = make_float2(c * size[i], s * size[i]);
        }
      }
      __syncwarp();
      float fa[2][8], fb[2][8];
      int now = -1;  // whose factors the lane has
      sd.head = part * kHeads + sub;
      if (sd.head < heads) place(sd, true);
      int step = part;
      while (step < steps) {
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
          if (step >= steps) break;
          if (__any_sync(~0u, sd.side != now)) {
            now = sd.side;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int c0 = 8 * (h ? piece1 : piece0);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                fa[h][j] = weights[now][c0 + j];
                fb[h][j] = 0.f;
                if (rotated[h]) {
                  const float2 t = turn[warp][kInterleaved ? (c0 + j) / 2 : 8 * piece0 + j];
                  fa[h][j] *= t.x;
                  const float other = weights[now][kInterleaved ? (c0 + j) ^ 1 : 8 * (h ? piece0 : piece1) + j];
                  fb[h][j] = other * ((kInterleaved ? j & 1 : h) ? t.y : -t.y);
                }
              }
            }
          }
          float v[2][8];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t w[4] = {x[i][h].x, x[i][h].y, x[i][h].z, x[i][h].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[h][2 * j] = ptx::bf16lo(w[j]);
              v[h][2 * j + 1] = ptx::bf16hi(w[j]);
            }
          }
          load(x[i]);
          float r = 1.f;
          if (p.norm) {
            float sum = 0.f, more = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              sum = fmaf(v[0][j], v[0][j], sum);
              more = fmaf(v[1][j], v[1][j], more);
            }
            sum += more;
#pragma unroll
            for (int o = kLanes / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
            r = rsqrtf(sum * (1.f / D) + p.eps);
          }
          uint4 z[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              float y[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float o = fb[h][j + e] * (kInterleaved ? v[h][j + 1 - e] : v[1 - h][j + e]);
                if constexpr (!kWhole) o = rotated[h] ? o : 0.f;  // (0 times what is not finite)
                y[e] = fmaf(fa[h][j + e], v[h][j + e], o) * r;
              }
              w[j / 2] = ptx::pack_bf16x2(y[0], y[1]);
            }
            z[h] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (sd.head < heads) {
            *reinterpret_cast<uint4*>(sd.at + 16 * piece0) = z[0];
            *reinterpret_cast<uint4*>(sd.at + 16 * piece1) = z[1];
            advance(sd, true);
          }
          step += p.parts;
        }
      }
      __syncwarp();
    }
    unit += stride;
    if (unit >= units) break;
    split(unit);
    load_first();
    at = position(live);
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeLaunch& a, cudaStream_t st) {
  RopeParams p;
  for (int i = 0; i < 2; ++i)
    p.side[i] = {static_cast<const __nv_bfloat16*>(a.in[i]), static_cast<__nv_bfloat16*>(a.out[i]), a.is[i], a.os[i],
                 a.weight[i], a.heads[i]};
  p.weight_f32 = a.weight_f32;
  p.norm = a.norm;
  p.eps = a.eps;
  p.positions = a.positions;
  p.pos_b = a.pos_b;
  p.pos_axis = a.pos_axis;
  p.cu_new = a.cu_new;
  p.start_lens = a.start_lens;
  p.requests = a.requests;
  p.freqs = a.freqs;
  p.pairs = a.pairs;
  for (int i = 0, sum = 0; i < 4; ++i) p.axis_end[i] = sum += i < a.axes ? a.axis_pairs[i] : 0;
  p.rot_scale = a.rot_scale;
  p.batch = a.batch;
  p.n = a.n;
  const int heads = 512 / a.d;  // of a warp's step
  const int steps = (a.heads[0] + a.heads[1] + heads - 1) / heads;
  const long long tokens = static_cast<long long>(a.batch) * a.n;
  // A warp a token, or, of fewer tokens than the GPU's warps, several.  (Of a few tokens a warp, splitting them too so
  // that the last round is shorter costs more angles than it saves: 4608 tokens, 24 + 24 heads, 29 and 34 us.)
  const long long warps = static_cast<long long>(host::sm_count()) * kBlocks * kWarps;
  p.parts = static_cast<int>(std::min<long long>(steps, std::max(1LL, warps / tokens)));
  const long long blocks = std::min(warps, tokens * p.parts + kWarps - 1) / kWarps;
  const dim3 grid(static_cast<unsigned>(blocks)), block(32 * kWarps);
  auto run = [&](auto kernel) { return launch_after(kernel, grid, block, 0, st, p); };
  const bool whole = 2 * p.pairs == a.d;
  if (a.d == 64) {
    if (a.interleaved) return whole ? run(qk_norm_rope_kernel<64, true, true>) : run(qk_norm_rope_kernel<64, true, false>);
    return whole ? run(qk_norm_rope_kernel<64, false, true>) : run(qk_norm_rope_kernel<64, false, false>);
  }
  if (a.interleaved) return whole ? run(qk_norm_rope_kernel<128, true, true>) : run(qk_norm_rope_kernel<128, true, false>);
  return whole ? run(qk_norm_rope_kernel<128, false, true>) : run(qk_norm_rope_kernel<128, false, false>);
}

}  // namespace ditattn
