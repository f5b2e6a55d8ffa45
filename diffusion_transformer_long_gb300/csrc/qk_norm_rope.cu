// Norms of queries and keys for each head, with rotary positions, in one pass.
//
//   r = 1 / sqrt(mean_d x_d^2 + eps),  z_d = w_d r x_d
//   pair i of the first 2 n channels, (2 i, 2 i + 1) or (i, i + n), at angle t_i = pos_a(i) f_i:
//     y_first = s (z_first cos t_i - z_second sin t_i),  y_second = s (z_first sin t_i + z_second cos t_i)
// Each value is read and written once: bound by HBM (75600 tokens, 40 + 40 heads of 128, token-major to
// head-major: %s us, %s TB/s; one token of each of 64 requests, 24 + 8 heads: %s us in a graph).
//
// A lane holds 8 neighbouring channels of a head, 16 bytes, so that a warp takes two heads of 128 or four of 64 at
// a step.  Every warp walks over tokens by itself, with kIters steps' loads in flight (the next token's first ones
// before its angles), and no barrier holds it up: with a block's warps on one token and its angles shared behind
// a barrier, 75600 tokens took 1370 us.  It works the token's cosines and sines out into shared memory, and folds them
// with the weights into two factors a channel, y = r (A x + B x'), with x' the pair's other channel: the lane's own, or
// that of the lane n / 8 away.  Where there are few tokens several warps take one, a part of its heads each.
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

namespace ditattn {
namespace {

constexpr int kIters = 4;   // steps of a warp whose loads are in flight at once
constexpr int kWarps = 8;   // of a block
constexpr int kBlocks = 4;  // of an SM

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

template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kWarps * 32, kBlocks) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;  // lanes of a head, heads of a warp's step
  __shared__ uint64_t step_turns[64];                  // the pairs' turns a position
  __shared__ float size[64];                           // their scale (NaN where the frequency is not finite)
  __shared__ float2 turn[kWarps][64];                  // (cos, sin) of the pairs at each warp's token, scaled
  __shared__ float weights[2][D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int chan = lane % kLanes * 8, sub = lane / kLanes;
  const bool rotated = chan < 2 * p.pairs;
  const bool second = !kInterleaved && chan >= p.pairs;  // the lane's channels are the pairs' second ones
  const int from = !rotated || kInterleaved ? lane : second ? lane - p.pairs / 8 : lane + p.pairs / 8;
  // Steps: kHeads query heads, or key heads, at a time.
  const int q_steps = (p.side[0].heads + kHeads - 1) / kHeads;
  const int steps = q_steps + (p.side[1].heads + kHeads - 1) / kHeads;
  const unsigned units = static_cast<unsigned>(p.batch) * p.n * p.parts, stride = gridDim.x * kWarps;
  unsigned unit = blockIdx.x * kWarps + warp;
  int b, n, part;  // of the unit
  auto split = [&](unsigned u) {
    const unsigned token = p.parts == 1 ? u : u / p.parts;
    part = static_cast<int>(u - token * p.parts);
    b = p.batch == 1 ? 0 : static_cast<int>(token / p.n);
    n = static_cast<int>(token - static_cast<unsigned>(b) * p.n);
  };
  uint4 x[kIters];
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int step = base + i * p.parts, side = step >= q_steps;
      const Side& s = p.side[side];
      const int head = (step - (side ? q_steps : 0)) * kHeads + sub;
      x[i] = make_uint4(0, 0, 0, 0);
      if (step < steps && head < s.heads) x[i] = load_once(s.in + b * s.is.b_ + head * s.is.h_ + n * s.is.n_ + chan);
    }
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
    load(part);
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
      float fa[8], fb[8];
      int now = -1;  // whose factors they are
      for (int base = part; base < steps; base += kIters * p.parts) {
        if (base != part) load(base);
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
          const int step = base + i * p.parts, side = step >= q_steps;
          if (step >= steps) break;
          const Side& s = p.side[side];
          const int head = (step - (side ? q_steps : 0)) * kHeads + sub;
          if (side != now) {
            now = side;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int c = chan + j;
              fa[j] = weights[side][c];
              fb[j] = 0.f;
              if (rotated) {
                const int pair = kInterleaved ? c / 2 : second ? c - p.pairs : c;
                const int other = kInterleaved ? c ^ 1 : second ? c - p.pairs : c + p.pairs;
                const float2 t = turn[warp][pair];
                fa[j] *= t.x;
                fb[j] = weights[side][other] * ((kInterleaved ? c & 1 : second) ? t.y : -t.y);
              }
            }
          }
          const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          float v[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
          }
          float r = 1.f;
          if (p.norm) {
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(v[j], v[j], sum);
#pragma unroll
            for (int o = kLanes / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
            r = rsqrtf(sum * (1.f / D) + p.eps);
          }
          uint32_t z[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float o0 = v[2 * j + 1], o1 = v[2 * j];  // the pairs' other channels
            if (!kInterleaved && p.pairs) {
              const uint32_t o = __shfl_sync(~0u, w[j], from);
              o0 = __uint_as_float(o << 16);
              o1 = __uint_as_float(o & 0xffff0000u);
            }
            // (0 times what is not finite: channels that are not turned take no other)
            const float y0 = fmaf(fa[2 * j], v[2 * j], rotated ? fb[2 * j] * o0 : 0.f) * r;
            const float y1 = fmaf(fa[2 * j + 1], v[2 * j + 1], rotated ? fb[2 * j + 1] * o1 : 0.f) * r;
            const __nv_bfloat162 h = __floats2bfloat162_rn(y0, y1);
            z[j] = *reinterpret_cast<const uint32_t*>(&h);
          }
          if (head < s.heads)
            *reinterpret_cast<uint4*>(s.out + b * s.os.b_ + head * s.os.h_ + n * s.os.n_ + chan) =
                make_uint4(z[0], z[1], z[2], z[3]);
        }
      }
      __syncwarp();
    }
    unit += stride;
    if (unit >= units) break;
    split(unit);
    load(part);
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
  const int heads = 256 / a.d;  // of a warp's step
  const int steps = (a.heads[0] + heads - 1) / heads + (a.heads[1] + heads - 1) / heads;
  const long long tokens = static_cast<long long>(a.batch) * a.n;
  // A warp a token, or, of fewer tokens than the GPU's warps, several.
  const long long warps = static_cast<long long>(host::sm_count()) * kBlocks * kWarps;
  p.parts = static_cast<int>(std::min<long long>(steps, std::max(1LL, warps / tokens)));
  const long long blocks = std::min(warps, tokens * p.parts + kWarps - 1) / kWarps;
  const dim3 grid(static_cast<unsigned>(blocks)), block(32 * kWarps);
  if (a.d == 64)
    return a.interleaved ? launch_after(qk_norm_rope_kernel<64, true>, grid, block, 0, st, p)
                         : launch_after(qk_norm_rope_kernel<64, false>, grid, block, 0, st, p);
  return a.interleaved ? launch_after(qk_norm_rope_kernel<128, true>, grid, block, 0, st, p)
                       : launch_after(qk_norm_rope_kernel<128, false>, grid, block, 0, st, p);
}

}  // namespace ditattn
