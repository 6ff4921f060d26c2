// la_block_norm_bwd.cuh -- what the backward passes of the norms around a block share.
//
// With n = (x - mean) r, r = 1 / sqrt(mean square + eps), and the gradient g of
// n, a row's gradient is
//
//     dx = r (g - mean(g) - n mean(g n))          (RMS norm: without the means of x and g)
//
// so a row needs two sums that do not wait for one another (of x^2 and of g x;
// layer norm: of x first, then those about the mean, and of g).  A team of threads
// takes a row and keeps it in registers, so every input is read once; it walks
// over many rows, with the next row's loads in flight, and keeps its columns' share
// of the weights' gradients in registers.  Those shares are added in a fixed
// order: over a block's teams, then over the blocks by a second kernel.
#pragma once

#include "../../include/la_gb300.h"
#include "la_act.cuh"
#include "la_internal.h"

namespace la {

constexpr int kNormTeamThreads = 256;  // threads per block of teams inside a warp

// Sums of K values over groups of W neighbouring lanes, in every lane: the values are halved
// among the lanes first, so that K sums take little more shuffles than one.
template <int K, int W> __device__ __forceinline__ void lane_sums(float (&v)[K]) {
  const int lane = threadIdx.x % 32;
  constexpr unsigned all = 0xffffffffu;
  if constexpr (K == 1 || W < 4) {
#pragma unroll
    for (int off = W / 2; off > 0; off >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(all, v[k], off);
  } else if constexpr (K == 2) {
    const bool up = lane & (W / 2);
    float s = (up ? v[1] : v[0]) + __shfl_xor_sync(all, up ? v[0] : v[1], W / 2);
#pragma unroll
    for (int off = W / 4; off > 0; off >>= 1) s += __shfl_xor_sync(all, s, off);
    v[0] = __shfl_sync(all, s, 0, W);
    v[1] = __shfl_sync(all, s, W / 2, W);
  } else {
    static_assert(K == 3 || K == 4, "up to four sums");
    const bool up = lane & (W / 2), odd = lane & (W / 4);
    const float v3 = K == 4 ? v[K - 1] : 0.f;
    const float a = (up ? v[2] : v[0]) + __shfl_xor_sync(all, up ? v[0] : v[2], W / 2);
    const float b = (up ? v3 : v[1]) + __shfl_xor_sync(all, up ? v[1] : v3, W / 2);
    float s = (odd ? b : a) + __shfl_xor_sync(all, odd ? a : b, W / 4);
#pragma unroll
    for (int off = W / 8; off > 0; off >>= 1) s += __shfl_xor_sync(all, s, off);
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = __shfl_sync(all, s, k * (W / 4), W);
  }
}

// Sums of K values over the team: LANES neighbouring lanes, or the block (LANES =
// 0).  `red` holds two sets, used in turn, so that one barrier is enough.
template <int LANES, int K>
__device__ __forceinline__ void team_sums(float (&v)[K], float (*red)[4][32], int &turn) {
  lane_sums<K, LANES ? LANES : 32>(v);
  if constexpr (LANES == 0) {
    static_assert(K <= 4, "red holds four sums");
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) red[turn][k][warp] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lane < warps ? red[turn][k][lane] : 0.f;
    lane_sums<K, 32>(v);
    turn ^= 1;
  }
}

// V values as cells: pairs of fp32 in a register pair each, one instruction for both (V = 1:
// single values).
template <int V> struct Cells {
  using C = typename CellOf<V>::type;
  static constexpr int H = V > 1 ? V / 2 : 1;
  __device__ static __forceinline__ void pack(const float *f, C *c) {
#pragma unroll
    for (int i = 0; i < H; ++i) {
      if constexpr (V == 1) c[i] = f[i];
      else c[i] = pack2(f[2 * i], f[2 * i + 1]);
    }
  }
  __device__ static __forceinline__ void unpack(const C *c, float *f) {
#pragma unroll
    for (int i = 0; i < H; ++i) {
      if constexpr (V == 1) f[i] = c[i];
      else unpack2(c[i], f[2 * i], f[2 * i + 1]);
    }
  }
};

// V fp32 parameters at p + c, `other` where there are none or the place is past d.
template <int V>
__device__ __forceinline__ void params_or(const float *p, int c, int d, float other, float *f) {
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = c < d ? other : 0.f;
  if (!p || c >= d) return;
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 u = __ldg(reinterpret_cast<const float4 *>(p + c + i));
      f[i] = u.x, f[i + 1] = u.y, f[i + 2] = u.z, f[i + 3] = u.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = __ldg(p + c + i);
  }
}

// A block's share of a weight's gradient: the teams' shares acc[I * V] added
// and written to dst[0 .. d).  `sum` is shared memory of 8 x 32 V I floats.
template <int V, int LANES, int I>
__device__ __forceinline__ void block_share(float *acc, float *dst, int d, float *sum) {
  const int lane = threadIdx.x % 32;
  if constexpr (LANES == 0) {
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * V;
      if (c < d) store_vec<float, V % 4 ? 1 : 4>(dst + c, acc + i * V);
      if constexpr (V == 8)
        if (c < d) store_vec<float, 4>(dst + c + 4, acc + i * V + 4);
    }
  } else {
    constexpr int W = LANES * V * I;  // columns
#pragma unroll
    for (int off = LANES; off < 32; off <<= 1)
#pragma unroll
      for (int j = 0; j < I * V; ++j) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], off);
    __syncthreads();
    if (lane < LANES) {
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e)
          sum[threadIdx.x / 32 * W + (lane + i * LANES) * V + e] = acc[i * V + e];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += kNormTeamThreads) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kNormTeamThreads / 32; ++w) s += sum[w * W + c];
      dst[c] = s;
    }
  }
}

// The second step of the weights' gradients: out[k][c] = sum over `parts` rows of
// part[k * parts + i][c], for up to four gradients in one launch.
struct WeightSums {
  const float *part;
  int parts, width;
  float *out[4];
};
cudaError_t launch_weight_sums(const WeightSums &w, int count, cudaStream_t stream);

// Blocks (for each of `heads`) for rows that would fill `wanted` blocks: `per_sm` to an SM, one to
// kNormMostBlocks.
constexpr int kNormMostBlocks = 4;
inline unsigned norm_bwd_blocks(long long wanted, int per_sm, int heads) {
  per_sm = per_sm < 1 ? 1 : per_sm > kNormMostBlocks ? kNormMostBlocks : per_sm;
  const long long fill = (152ll * per_sm + heads - 1) / heads;
  return (unsigned)(wanted < fill ? wanted : fill);
}

template <int N> struct IntC { static constexpr int value = N; };

// Calls f(IntC<LANES>, IntC<I>, IntC<most threads>, threads) with the team for rows of width
// d in vectors of V elements: 4 to 32 lanes with one vector each, a warp with more, then
// a block.
template <int V, typename F>
cudaError_t with_bwd_team(int d, F f) {
  const int vecs = (d + V - 1) / V;
  if constexpr (V > 1) {
    if (vecs <= 4) return f(IntC<4>{}, IntC<1>{}, IntC<kNormTeamThreads>{}, 4);
    if (vecs <= 8) return f(IntC<8>{}, IntC<1>{}, IntC<kNormTeamThreads>{}, 8);
    if (vecs <= 16) return f(IntC<16>{}, IntC<1>{}, IntC<kNormTeamThreads>{}, 16);
    if (vecs <= 32) return f(IntC<32>{}, IntC<1>{}, IntC<kNormTeamThreads>{}, 32);
    if (vecs <= 64) return f(IntC<32>{}, IntC<2>{}, IntC<kNormTeamThreads>{}, 32);
  } else {
    if (vecs <= 128) return f(IntC<32>{}, IntC<4>{}, IntC<kNormTeamThreads>{}, 32);
  }
  constexpr int I = V == 8 ? 1 : V == 4 ? 2 : 8;
  auto threads = [&](int per) { return ((vecs + per - 1) / per + 31) / 32 * 32; };
  if (threads(I) <= 512) return f(IntC<0>{}, IntC<I>{}, IntC<512>{}, threads(I));
  // The fewer threads a block may have, the more registers each: 2000 x 5001 fp32 with rows of up
  // to 512 threads 187 us, compiled for 1024 378; 2000 x 8192 fp32 77, 176; 1111 x 9543 bf16 with
  // up to 768 191, 202.
  if (threads(2 * I) <= 512) return f(IntC<0>{}, IntC<2 * I>{}, IntC<512>{}, threads(2 * I));
  if (threads(2 * I) <= 768) return f(IntC<0>{}, IntC<2 * I>{}, IntC<768>{}, threads(2 * I));
  return f(IntC<0>{}, IntC<2 * I>{}, IntC<1024>{}, threads(2 * I));
}

}  // namespace la
