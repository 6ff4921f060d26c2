// la_causal_conv.cu -- causal depthwise convolution over time with its rolling
// state, for whole sequences and single tokens.
//
//     y[t] = act(bias + sum_{w < W} weight[w] x[t - W + 1 + w])
//
// Per element 2W flops and an activation for one load and one store: a stream
// over x and y.  A thread owns one vector of channels and a run of tokens,
// which it walks in batches of BATCH: the loads of a batch are all in flight
// while the batch before it is computed, and the W - 1 previous inputs stay in
// registers.  Only the rows in front of a run are read twice.  The threads of
// a block lie side by side in channels first, then in time.  A block's weights
// are transposed in shared memory: read directly, a warp's 16-byte loads of
// [D, W] would touch 32 lines each.
#include <cstdint>

#include "../../include/la_gb300.h"
#include "la_act.cuh"
#include "la_internal.h"

namespace la {
namespace {

constexpr int kThreads = 256;
// Tokens per batch, and the bytes a thread loads of each.  4 x 4096 x 4096 bf16
// (x a slice of rows twice as wide): 8 bytes in batches of 8, 55 us; 16 bytes
// in batches of 4 or 8, 55 and 61; 8 bytes in batches of 4, 62.  The batches in
// flight are held in registers: 114 a thread, two blocks per SM.
constexpr int kBatch = 8, kVecBytes = 8;

// 1 << lane_bits threads lie side by side in channels; runs of `batches` batches.
template <typename T, int W, int VEC, int BATCH, int ACT>
__global__ void __launch_bounds__(kThreads)
causal_conv_kernel(const ConvArgs a, int lane_bits, int runs, int batches) {
  using R = Raw<T, VEC>;
  using Cell = typename CellOf<VEC>::type;
  constexpr int H = VEC > 1 ? VEC / 2 : 1;  // pairs of channels, or the one channel
  extern __shared__ float4 shared4[];
  float *wt = reinterpret_cast<float *>(shared4);  // [W][wide], then the bias
  const int lanes = 1 << lane_bits, wide = lanes * VEC;
  const int nv = a.D / VEC, tiles = (nv + lanes - 1) >> lane_bits;
  const int tile = blockIdx.x % tiles;
  const int c0 = tile * wide, nc = min(wide, a.D - c0);
  const int cl = threadIdx.x & (lanes - 1);
  const long long run = (long long)(blockIdx.x / tiles) * (kThreads >> lane_bits) +
                        (threadIdx.x >> lane_bits);
  const bool live = run < (long long)a.B * runs && (tile << lane_bits) + cl < nv;
  const int c = c0 + cl * VEC;
  const long long b = live ? div_index(run, runs) : 0;
  const int r = live ? (int)(run - b * runs) : 0;
  const int len = a.lengths ? min(max(a.lengths[b], 0), a.L) : a.L;
  const int t0 = r * batches * BATCH, n = live ? min(batches * BATCH, len - t0) : 0;
  const T *xb = static_cast<const T *>(a.x) + b * a.L * a.x_stride + c;
  // Not through the read-only path: the final state may lie over it.
  const T *s0 = a.state0 ? static_cast<const T *>(a.state0) + b * (W - 1) * a.D + c : nullptr;
  auto row = [&](int t) {  // input t of the sequence, t >= -(W - 1)
    R v{};
    if (t >= 0) v = load_raw<T, VEC>(xb + t * a.x_stride);
    else if (s0) v = load_raw<T, VEC>(s0 + (long long)(t + W - 1) * a.D);
    return v;
  };
  R in[BATCH], before[W - 1];
  const T *next = xb + t0 * a.x_stride;  // the next row to load
  auto fetch = [&](int left) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (i < left) in[i] = load_raw<T, VEC>(next + i * a.x_stride);
    next += BATCH * a.x_stride;
  };
  if (n > 0) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k) before[k] = row(t0 - (W - 1) + k);
    fetch(n);
  }
  // (after the first loads have left)
  for (int i = threadIdx.x; i < nc * W; i += kThreads)
    wt[i % W * wide + i / W] = a.weight[(long long)c0 * W + i];
  for (int i = threadIdx.x; i < nc; i += kThreads)
    wt[W * wide + i] = a.bias ? a.bias[c0 + i] : 0.f;

  // The thread of the first run writes the final state, after it has read the
  // initial one: row j is input len - (W - 1) + j, never one that an earlier
  // row has overwritten.
  if (live && r == 0 && a.state_final) {
    T *sf = static_cast<T *>(a.state_final) + b * (W - 1) * a.D + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      store_raw<T, VEC>(sf + (long long)j * a.D, row(len - (W - 1) + j));
  }
  __syncthreads();
  if (n <= 0) return;

  Cell w[W + 1][H], win[W - 1 + BATCH][H];
#pragma unroll
  for (int k = 0; k <= W; ++k) {
    const float *from = wt + k * wide + cl * VEC;
    if constexpr (VEC == 1) {
      w[k][0] = from[0];
    } else if constexpr (VEC == 2) {
      const float2 f = *reinterpret_cast<const float2 *>(from);
      w[k][0] = pack2(f.x, f.y);
    } else {
#pragma unroll
      for (int i = 0; i < H; i += 2) {
        const float4 f = *reinterpret_cast<const float4 *>(from + 2 * i);
        w[k][i] = pack2(f.x, f.y), w[k][i + 1] = pack2(f.z, f.w);
      }
    }
  }
  auto bring = [&](const R &raw, int k) {
    float f[VEC];
    raw.unpack(f);
#pragma unroll
    for (int i = 0; i < H; ++i) {
      if constexpr (VEC == 1) win[k][i] = f[i];
      else win[k][i] = pack2(f[2 * i], f[2 * i + 1]);
    }
  };
#pragma unroll
  for (int k = 0; k < W - 1; ++k) bring(before[k], k);
  T *yr = static_cast<T *>(a.y) + (b * a.L + t0) * a.y_stride + c;
  for (int done = 0; done < n; done += BATCH) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) bring(in[i], W - 1 + i);
    if (done + BATCH < n) fetch(n - done - BATCH);
#pragma unroll
    for (int t = 0; t < BATCH; ++t) {
      if (done + t >= n) break;
      float f[VEC];
#pragma unroll
      for (int i = 0; i < H; ++i) {
        Cell o = w[W][i];
#pragma unroll
        for (int k = 0; k < W; ++k) o = fma2(w[k][i], win[t + k][i], o);
        o = activate2(ACT, o);
        if constexpr (VEC == 1) f[i] = o;
        else unpack2(o, f[2 * i], f[2 * i + 1]);
      }
      store_vec<T, VEC>(yr, f);
      yr += a.y_stride;
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
#pragma unroll
      for (int i = 0; i < H; ++i) win[k][i] = win[BATCH + k][i];
  }
}


template <typename T, int W, int VEC, int BATCH>
cudaError_t launch_run(const ConvArgs &a) {
  const int nv = a.D / VEC;
  int lane_bits = 5;
  while (lane_bits > 0 && 1 << (lane_bits - 1) >= nv) --lane_bits;
  // Runs as long as they leave the GPU full (some 150,000 threads at a time):
  // each reads W - 1 rows twice and starts with nothing in flight.  The case
  // above: runs of 16, 32, 64, 128 tokens in 69, 58, 58, 55 us.  The limit of
  // 100e3 threads against 50e3, 200e3 and 400e3, W = 4, in us:
  //   1 x 4096 x 4096 bf16   17.8, 16.7, 20.7, 25.2    fp32  28.2, 27.8, 25.6, 26.0
  //   16 x 512 x 1024 bf16   12.9, 11.5, 15.1, 15.0    fp32  17.1, 16.8, 16.5, 17.7
  //   4 x 4096 x 4096 bf16   53.2, 52.8, 55.8, 56.0    fp32  97.0, 96.7, 88.7, 86.6
  int batches = 1;
  auto threads = [&](int m) { return (double)a.B * nv * ((a.L + m * BATCH - 1) / (m * BATCH)); };
  while (batches < 32 && threads(2 * batches) >= 100e3) batches *= 2;
  const int run = batches * BATCH;
  const int runs = a.L > 0 ? (a.L + run - 1) / run : 1;  // L = 0 still passes the state on
  const int tiles = (nv + (1 << lane_bits) - 1) >> lane_bits, per = kThreads >> lane_bits;
  const long long blocks = ((long long)a.B * runs + per - 1) / per * tiles;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  const size_t smem = ((size_t)(W + 1) * VEC << lane_bits) * sizeof(float);
  auto *kernel = a.act == LA_ACT_SILU ? causal_conv_kernel<T, W, VEC, BATCH, LA_ACT_SILU>
                                      : causal_conv_kernel<T, W, VEC, BATCH, LA_ACT_NONE>;
  kernel<<<(unsigned)blocks, kThreads, smem, a.stream>>>(a, lane_bits, runs, batches);
  return cudaGetLastError();
}

template <typename T, int W>
cudaError_t launch_w(const ConvArgs &a) {
  // The widest vectors, up to 8 bytes, that every row's alignment allows (4 x
  // 4096 x 4096 bf16 52 us; 4098 wide in pairs 54, element by element 73; 4097
  // wide 74).  One token's call is a launch, pairs or not.
  auto rows_fit = [&](int v) {
    auto fits = [&](const void *p) {
      return reinterpret_cast<uintptr_t>(p) % (v * sizeof(T)) == 0;
    };
    return a.D % v == 0 && a.x_stride % v == 0 && a.y_stride % v == 0 && fits(a.x) &&
           fits(a.y) && fits(a.state0) && fits(a.state_final);
  };
  constexpr int V = kVecBytes / (int)sizeof(T);
  if (a.L <= 1) return rows_fit(V) ? launch_run<T, W, V, 1>(a) : launch_run<T, W, 1, 1>(a);
  if (rows_fit(V)) return launch_run<T, W, V, kBatch>(a);
  if constexpr (V > 2) {
    if (rows_fit(2)) return launch_run<T, W, 2, kBatch>(a);
  }
  return launch_run<T, W, 1, kBatch>(a);
}

template <typename T>
cudaError_t launch_t(const ConvArgs &a) {
  switch (a.width) {
    case 2: return launch_w<T, 2>(a);
    case 3: return launch_w<T, 3>(a);
    case 4: return launch_w<T, 4>(a);
    case 5: return launch_w<T, 5>(a);
    case 6: return launch_w<T, 6>(a);
    case 7: return launch_w<T, 7>(a);
    case 8: return launch_w<T, 8>(a);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_causal_conv(const ConvArgs &a) {
  return a.dtype == LA_F32 ? launch_t<float>(a) : launch_t<__nv_bfloat16>(a);
}

}  // namespace la
