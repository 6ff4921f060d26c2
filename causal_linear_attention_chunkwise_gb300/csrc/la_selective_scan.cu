// la_selective_scan.cu -- selective state space scan.
//
//     delta = softplus(dt + bias);  h_n = exp(delta A_n) h_n + (delta x) B_n
//     y = (sum_n C_n h_n + skip x) silu(z)
//
// for every channel and token, N states per channel.  The decay differs per
// (channel, state) pair, so no matrix product carries the recurrence: per
// state and token it takes one exp and four multiply-adds' worth of fp32 work.
//
// S neighbouring lanes share a channel, each holding P of its states in
// registers; the products with C are summed over the lanes by shuffles.
#include <cstdint>

#include "../../include/la_gb300.h"
#include "la_act.cuh"
#include "la_internal.h"

namespace la {
namespace {

constexpr int kThreads = 128;

template <typename T>
struct ScanParams {
  const T *x, *dt, *z, *Bm, *Cm;
  long long x_stride, dt_stride, z_stride, b_stride, c_stride;
  int L, D, N, groups;
  const float *A, *dt_bias;
  int softplus;
  const float *skip;
  const float *h0;
  const int *lengths;
  T *y;
  long long y_stride;
  float *h_final;
};

template <typename T, int P, int S>
__global__ void __launch_bounds__(kThreads) selective_scan_kernel(const ScanParams<T> p) {
  constexpr int CH = kThreads / S;  // channels per block
  const int per_group = p.D / p.groups;
  const int blocks_g = (per_group + CH - 1) / CH;
  const int blk = blockIdx.x % (blocks_g * p.groups);
  const long long b = blockIdx.x / (blocks_g * p.groups);
  const int g = blk / blocks_g;
  const int cg = blk % blocks_g * CH + threadIdx.x / S;  // channel within the group
  const bool live = cg < per_group;
  const int c = g * per_group + (live ? cg : 0);
  const int n0 = threadIdx.x % S * P;
  const int len = p.lengths ? min(max(p.lengths[b], 0), p.L) : p.L;

  float a[P], h[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const bool in = n0 + i < p.N;
    a[i] = in ? p.A[(long long)c * p.N + n0 + i] * kLog2e : 0.f;
    h[i] = in && p.h0 ? p.h0[(b * p.D + c) * p.N + n0 + i] : 0.f;
  }
  const float bias = p.dt_bias ? p.dt_bias[c] : 0.f;
  const float skip = p.skip ? p.skip[c] : 0.f;
  for (int t = 0; t < len; ++t) {
    const long long row = b * p.L + t;
    const float x = to_f32(p.x[row * p.x_stride + c]);
    float delta = to_f32(p.dt[row * p.dt_stride + c]) + bias;
    if (p.softplus) delta = softplus(delta);
    const float u = delta * x;
    float acc = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const bool in = n0 + i < p.N;
      const float bn = in ? to_f32(p.Bm[row * p.b_stride + g * p.N + n0 + i]) : 0.f;
      const float cn = in ? to_f32(p.Cm[row * p.c_stride + g * p.N + n0 + i]) : 0.f;
      h[i] = fmaf(ex2_approx(delta * a[i]), h[i], u * bn);
      acc = fmaf(cn, h[i], acc);
    }
#pragma unroll
    for (int off = S / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (live && n0 == 0) {
      float o = fmaf(skip, x, acc);
      if (p.z) o *= activate(1, to_f32(p.z[row * p.z_stride + c]));
      p.y[row * p.y_stride + c] = from_f32<T>(o);
    }
  }
  if (live && p.h_final) {
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (n0 + i < p.N) p.h_final[(b * p.D + c) * p.N + n0 + i] = h[i];
  }
}

template <typename T, int P, int S>
cudaError_t launch_ps(const ScanArgs &a) {
  constexpr int CH = kThreads / S;
  const ScanParams<T> p{static_cast<const T *>(a.x), static_cast<const T *>(a.dt),
                        static_cast<const T *>(a.z), static_cast<const T *>(a.Bm),
                        static_cast<const T *>(a.Cm), a.x_stride, a.dt_stride, a.z_stride,
                        a.b_stride, a.c_stride, a.L, a.D, a.N, a.groups, a.A, a.dt_bias,
                        a.softplus, a.skip, a.h0, a.lengths, static_cast<T *>(a.y), a.y_stride,
                        a.h_final};
  const long long blocks =
      (long long)a.B * a.groups * ((a.D / a.groups + CH - 1) / CH);
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  selective_scan_kernel<T, P, S><<<(unsigned)blocks, kThreads, 0, a.stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const ScanArgs &a) {
  if (a.N <= 4) return launch_ps<T, 4, 1>(a);
  if (a.N <= 8) return launch_ps<T, 4, 2>(a);
  if (a.N <= 16) return launch_ps<T, 4, 4>(a);
  if (a.N <= 32) return launch_ps<T, 8, 4>(a);
  if (a.N <= 64) return launch_ps<T, 8, 8>(a);
  if (a.N <= 128) return launch_ps<T, 8, 16>(a);
  return launch_ps<T, 8, 32>(a);
}

}  // namespace

size_t selective_scan_workspace_bytes(int, int, int, int, int) { return 0; }

cudaError_t launch_selective_scan(const ScanArgs &a) {
  return a.dtype == LA_F32 ? launch_t<float>(a) : launch_t<__nv_bfloat16>(a);
}

}  // namespace la
