// la_causal_conv.cu -- causal depthwise convolution over time with its rolling
// state, for whole sequences and single tokens.
//
//     y[t] = act(bias + sum_{w < W} weight[w] x[t - W + 1 + w])
//
// Per element 2W flops and an activation for one load and one store: a stream
// over x and y.  A thread owns one vector of channels and a run of tokens; the
// W - 1 previous inputs stay in registers as it walks the run, so x is read
// once but for the W - 1 rows in front of each run.
#include <cstdint>

#include "../../include/la_gb300.h"
#include "la_act.cuh"
#include "la_internal.h"

namespace la {
namespace {

constexpr int kThreads = 128;

template <typename T, int W, int VEC>
__global__ void __launch_bounds__(kThreads)
causal_conv_kernel(const T *__restrict__ x, long long x_stride, int B, int L, int D, int run,
                   int runs, const float *__restrict__ weight, const float *__restrict__ bias,
                   int act, const int *__restrict__ lengths, const T *state0, T *__restrict__ y,
                   long long y_stride, T *state_final) {
  const int nv = D / VEC;
  const long long idx = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (idx >= (long long)B * runs * nv) return;
  const int c = (int)(idx % nv) * VEC;
  const int r = (int)(idx / nv % runs);
  const long long b = idx / nv / runs;
  const int len = lengths ? min(max(lengths[b], 0), L) : L;
  const int t0 = r * run, t1 = min(t0 + run, len);
  const T *xb = x + b * L * x_stride + c;
  const T *s0 = state0 ? state0 + b * (W - 1) * D + c : nullptr;

  float win[W][VEC];  // win[w] = x[t - W + 1 + w]; win[W - 1] is filled at token t
#pragma unroll
  for (int w = 0; w < W - 1; ++w) {
    const int t = t0 - (W - 1) + w;
    if (t >= 0 && t0 < t1) {
      load_vec<T, VEC>(xb + t * x_stride, win[w]);
    } else if (t < 0 && s0) {
      load_vec<T, VEC>(s0 + (long long)(t + W - 1) * D, win[w]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) win[w][i] = 0.f;
    }
  }
  // The thread of the first run writes the final state, after it has read the
  // initial one (which may be the same buffer): row j is input len + j of
  // state0 followed by x, never one that an earlier row has overwritten.
  if (r == 0 && state_final) {
    T *sf = state_final + b * (W - 1) * D + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int m = len + j;
      float f[VEC];
      if (m >= W - 1) {
        load_vec<T, VEC>(xb + (long long)(m - (W - 1)) * x_stride, f);
      } else if (s0) {
        load_vec<T, VEC>(s0 + (long long)m * D, f);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = 0.f;
      }
      store_vec<T, VEC>(sf + (long long)j * D, f);
    }
  }
  if (t0 >= t1) return;

  float wt[W][VEC], bs[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    bs[i] = bias ? bias[c + i] : 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) wt[w][i] = weight[(long long)(c + i) * W + w];
  }
  T *yb = y + b * L * y_stride + c;
  for (int t = t0; t < t1; ++t) {
    load_vec<T, VEC>(xb + t * x_stride, win[W - 1]);
    float o[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      o[i] = bs[i];
#pragma unroll
      for (int w = 0; w < W; ++w) o[i] = fmaf(wt[w][i], win[w][i], o[i]);
      o[i] = activate(act, o[i]);
#pragma unroll
      for (int w = 0; w < W - 1; ++w) win[w][i] = win[w + 1][i];
    }
    store_vec<T, VEC>(yb + t * y_stride, o);
  }
}

template <typename T, int W, int VEC>
cudaError_t launch_v(const ConvArgs &a) {
  const int run = 16;
  const int runs = a.L > 0 ? (a.L + run - 1) / run : 1;  // L = 0 still passes the state on
  const long long threads = (long long)a.B * runs * (a.D / VEC);
  const long long blocks = (threads + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  causal_conv_kernel<T, W, VEC><<<(unsigned)blocks, kThreads, 0, a.stream>>>(
      static_cast<const T *>(a.x), a.x_stride, a.B, a.L, a.D, run, runs, a.weight, a.bias, a.act,
      a.lengths, static_cast<const T *>(a.state0), static_cast<T *>(a.y), a.y_stride,
      static_cast<T *>(a.state_final));
  return cudaGetLastError();
}

template <typename T, int W>
cudaError_t launch_w(const ConvArgs &a) {
  constexpr int V = Pack16<T>::N;
  auto fits = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  const bool vec = a.D % V == 0 && a.x_stride % V == 0 && a.y_stride % V == 0 && fits(a.x) &&
                   fits(a.y) && fits(a.state0) && fits(a.state_final);
  return vec ? launch_v<T, W, V>(a) : launch_v<T, W, 1>(a);
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
