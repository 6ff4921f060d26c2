// la_act.cuh -- the activations and the vector loads of the state space block's kernels.
#pragma once

#include "la_common.cuh"

namespace la {

// 2^x on the special-function unit; results below 2^-126 become 0.
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + e^-x): e^-x overflows to infinity for x < -88, whose reciprocal is 0.
__device__ __forceinline__ float sigmoid(float x) {
  return rcp_approx(1.f + ex2_approx(-x * kLog2e));
}

// act: LA_ACT_NONE (x), LA_ACT_SILU (x sigmoid(x)), LA_ACT_SIGMOID.
__device__ __forceinline__ float activate(int act, float x) {
  if (act == 1) return x * sigmoid(x);
  return act == 2 ? sigmoid(x) : x;
}

// log(1 + e^v) = max(v, 0) + log1p(e), e = e^-|v| in (0, 1].  log1p(e) is
// taken as 2 atanh(s) with s = e / (2 + e) <= 1/3, whose odd series to s^13
// leaves a relative remainder below (1/9)^7 / 15 = 1.4e-8: step sizes near
// e^-7 keep their relative precision, which log(1 + e) would lose.
__device__ __forceinline__ float softplus(float v) {
  const float e = expf(-fabsf(v));
  const float s = e * rcp_approx(2.f + e);
  const float q = s * s;
  float p = fmaf(q, 1.f / 13.f, 1.f / 11.f);
  p = fmaf(q, p, 1.f / 9.f);
  p = fmaf(q, p, 1.f / 7.f);
  p = fmaf(q, p, 1.f / 5.f);
  p = fmaf(q, p, 1.f / 3.f);
  p = fmaf(q, p, 1.f);
  return fmaxf(v, 0.f) + 2.f * s * p;
}

// VEC consecutive elements of T (16 bytes, or one element) to and from fp32.
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T *p, float *f) {
  if constexpr (VEC == 1) {
    f[0] = to_f32(*p);
  } else {
    static_assert(VEC == Pack16<T>::N, "16-byte vectors");
    Pack16<T>::unpack(*reinterpret_cast<const uint4 *>(p), f);
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float *f) {
  if constexpr (VEC == 1) {
    *p = from_f32<T>(f[0]);
  } else {
    static_assert(VEC == Pack16<T>::N, "16-byte vectors");
    alignas(16) T u[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) u[i] = from_f32<T>(f[i]);
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(u);
  }
}

}  // namespace la
