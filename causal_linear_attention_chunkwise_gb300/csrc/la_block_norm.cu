// la_block_norm.cu -- the norms around a block: the gated norm of a layer's
// heads on their way to the output projection, and the residual step between
// two blocks (post norm, residual scale, addition, next block's norm).
//
// Both are streams over their inputs and outputs with one or two reductions
// per row, held in fp32: a row's mean first, then the mean square about it.
#include <cstdint>

#include "../../include/la_gb300.h"
#include "la_act.cuh"
#include "la_internal.h"

namespace la {
namespace {

constexpr int kThreads = 128;

__device__ float block_sum(float v, float *red) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  __syncthreads();  // red may still be read from the sum before
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}

// mean (0 for RMS) and 1 / sqrt(mean square about it + eps) of row[0..d).
__device__ void moments(const float *row, int d, int norm, float eps, float *red, float *mean,
                        float *rstd) {
  float m = 0.f;
  if (norm == LA_NORM_LAYER) {
    for (int i = threadIdx.x; i < d; i += kThreads) m += row[i];
    m = block_sum(m, red) / d;
  }
  float q = 0.f;
  for (int i = threadIdx.x; i < d; i += kThreads) q = fmaf(row[i] - m, row[i] - m, q);
  *mean = m;
  *rstd = rsqrtf(block_sum(q, red) / d + eps);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
gated_norm_kernel(const T *x, long long x_bs, long long x_hs, long long x_ts, const T *gate,
                  long long gate_stride, int H, int L, int d, int norm, int act, int gate_first,
                  const float *weight, const float *bias, int weight_heads, float eps, T *y,
                  long long y_stride) {
  extern __shared__ float row[];
  __shared__ float red[4];
  const int h = blockIdx.x % H;
  const long long bt = blockIdx.x / H;
  const T *xr = x + bt / L * x_bs + h * x_hs + bt % L * x_ts;
  const T *gr = gate ? gate + bt * gate_stride + (long long)h * d : nullptr;
  T *yr = y + bt * y_stride + (long long)h * d;
  for (int i = threadIdx.x; i < d; i += kThreads) {
    float v = to_f32(xr[i]);
    if (gr && gate_first) v *= activate(act, to_f32(gr[i]));
    row[i] = v;
  }
  float mean, rstd;
  moments(row, d, norm, eps, red, &mean, &rstd);
  const long long w0 = weight_heads > 1 ? (long long)h * d : 0;
  for (int i = threadIdx.x; i < d; i += kThreads) {
    float v = (row[i] - mean) * rstd;
    if (weight) v *= weight[w0 + i];
    if (bias) v += bias[w0 + i];
    if (gr && !gate_first) v *= activate(act, to_f32(gr[i]));
    yr[i] = from_f32<T>(v);
  }
}

template <typename T, typename R>
__global__ void __launch_bounds__(kThreads)
residual_norm_kernel(const T *x, const R *residual, int D, const float *post_weight,
                     const float *scale, float alpha, const float *weight, const float *bias,
                     int norm, float eps, T *y, R *residual_out) {
  extern __shared__ float row[];
  __shared__ float red[4];
  const long long at = (long long)blockIdx.x * D;
  float mean = 0.f, rstd = 1.f;
  for (int i = threadIdx.x; i < D; i += kThreads) row[i] = to_f32(x[at + i]);
  if (post_weight) moments(row, D, norm, eps, red, &mean, &rstd);
  for (int i = threadIdx.x; i < D; i += kThreads) {
    float u = row[i];
    if (post_weight) u = (u - mean) * rstd * post_weight[i];
    if (scale) u *= scale[i];
    const float r = fmaf(alpha, u, residual ? to_f32(residual[at + i]) : 0.f);
    if (residual_out) residual_out[at + i] = from_f32<R>(r);
    row[i] = r;
  }
  moments(row, D, norm, eps, red, &mean, &rstd);
  for (int i = threadIdx.x; i < D; i += kThreads) {
    float v = (row[i] - mean) * rstd;
    if (weight) v *= weight[i];
    if (bias) v += bias[i];
    y[at + i] = from_f32<T>(v);
  }
}

template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T>
cudaError_t launch_gated_t(const GatedNormArgs &a) {
  const long long rows = (long long)a.B * a.L * a.H;
  if (rows > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  const size_t smem = (size_t)a.d * sizeof(float);
  cudaError_t e = allow_smem(gated_norm_kernel<T>, smem);
  if (e != cudaSuccess) return e;
  gated_norm_kernel<T><<<(unsigned)rows, kThreads, smem, a.stream>>>(
      static_cast<const T *>(a.x), a.x_bs, a.x_hs, a.x_ts, static_cast<const T *>(a.gate),
      a.gate_stride, a.H, a.L, a.d, a.norm, a.act, a.gate_first, a.weight, a.bias,
      a.weight_heads, a.eps, static_cast<T *>(a.y), a.y_stride);
  return cudaGetLastError();
}

template <typename T, typename R>
cudaError_t launch_residual_t(const ResidualNormArgs &a) {
  if (a.rows > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  const size_t smem = (size_t)a.D * sizeof(float);
  cudaError_t e = allow_smem(residual_norm_kernel<T, R>, smem);
  if (e != cudaSuccess) return e;
  residual_norm_kernel<T, R><<<(unsigned)a.rows, kThreads, smem, a.stream>>>(
      static_cast<const T *>(a.x), static_cast<const R *>(a.residual), a.D, a.post_weight,
      a.scale, a.alpha, a.weight, a.bias, a.norm, a.eps, static_cast<T *>(a.y),
      static_cast<R *>(a.residual_out));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gated_norm(const GatedNormArgs &a) {
  return a.dtype == LA_F32 ? launch_gated_t<float>(a) : launch_gated_t<__nv_bfloat16>(a);
}

cudaError_t launch_residual_norm(const ResidualNormArgs &a) {
  if (a.dtype == LA_F32) return launch_residual_t<float, float>(a);
  if (a.res_dtype == LA_F32) return launch_residual_t<__nv_bfloat16, float>(a);
  return launch_residual_t<__nv_bfloat16, __nv_bfloat16>(a);
}

}  // namespace la
