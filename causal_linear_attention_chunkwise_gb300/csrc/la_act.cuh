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

// max(a, b), NaN where one of them is (fmaxf gives the other).
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + e^-x), off by at most some 2^-21 relative above x = -87.3.  Below, the
// result has no normal fp32 number and is 0 (e^-x overflows from -88 on).
__device__ __forceinline__ float sigmoid(float x) {
  return rcp_approx(1.f + ex2_approx(-x * kLog2e));
}

// act: LA_ACT_NONE (x), LA_ACT_SILU (x sigmoid(x)), LA_ACT_SIGMOID.
__device__ __forceinline__ float activate(int act, float x) {
  if (act == 1) return x * sigmoid(x);
  return act == 2 ? sigmoid(x) : x;
}

// Two fp32 values in one 64-bit register pair: one instruction for both.
__device__ __forceinline__ unsigned long long pack2(float lo, float hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(unsigned long long v, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b,
                                                   unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long dup2(float v) { return pack2(v, v); }

// act of two values.
__device__ __forceinline__ unsigned long long activate2(int act, unsigned long long v) {
  if (act == 0) return v;
  float a, b;
  unpack2(mul2(v, dup2(-kLog2e)), a, b);
  unpack2(add2(pack2(ex2_approx(a), ex2_approx(b)), dup2(1.f)), a, b);
  const unsigned long long s = pack2(rcp_approx(a), rcp_approx(b));
  return act == 1 ? mul2(v, s) : s;
}

// The same operations where the vectors are single elements.
__device__ __forceinline__ float mul2(float a, float b) { return a * b; }
__device__ __forceinline__ float add2(float a, float b) { return a + b; }
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float activate2(int act, float v) { return activate(act, v); }
template <int VEC> struct CellOf {  // what VEC > 1 holds two values in
  using type = unsigned long long;
  __device__ static __forceinline__ type both(float v) { return dup2(v); }
  __device__ static __forceinline__ float sum(type c) {
    float lo, hi;
    unpack2(c, lo, hi);
    return lo + hi;
  }
};
template <> struct CellOf<1> {
  using type = float;
  __device__ static __forceinline__ type both(float v) { return v; }
  __device__ static __forceinline__ float sum(type c) { return c; }
};

// a / b for a >= 0: in 32 bits where a allows it (a 64-bit division is some
// hundred instructions).
__device__ __forceinline__ long long div_index(long long a, int b) {
  return a >> 32 == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// VEC elements of T as they lie in memory: 16, 8 or 4 bytes, or one element.
template <typename T, int VEC> struct Raw {
  static constexpr int WORDS = VEC * sizeof(T) / 4;
  static_assert(WORDS == 4 || WORDS == 2 || WORDS == 1, "16-, 8- or 4-byte vectors");
  alignas(VEC * sizeof(T)) uint32_t w[WORDS];
  __device__ __forceinline__ void unpack(float *f) const {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      if constexpr (sizeof(T) == 4) f[i] = __uint_as_float(w[i]);
      else f[i] = __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
  }
};
template <typename T> struct Raw<T, 1> {
  T u;
  __device__ __forceinline__ void unpack(float *f) const { f[0] = to_f32(u); }
};

// VEC elements between memory and registers, and from fp32.
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T *p) {
  Raw<T, VEC> r;
  if constexpr (VEC == 1) {
    r.u = *p;
  } else if constexpr (VEC * sizeof(T) == 16) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    r.w[0] = u.x, r.w[1] = u.y, r.w[2] = u.z, r.w[3] = u.w;
  } else if constexpr (VEC * sizeof(T) == 8) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    r.w[0] = u.x, r.w[1] = u.y;
  } else {
    r.w[0] = *reinterpret_cast<const uint32_t *>(p);
  }
  return r;
}
template <typename T, int VEC>
__device__ __forceinline__ void store_raw(T *p, const Raw<T, VEC> &r) {
  if constexpr (VEC == 1) *p = r.u;
  else if constexpr (VEC * sizeof(T) == 16)
    *reinterpret_cast<uint4 *>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  else if constexpr (VEC * sizeof(T) == 8)
    *reinterpret_cast<uint2 *>(p) = make_uint2(r.w[0], r.w[1]);
  else *reinterpret_cast<uint32_t *>(p) = r.w[0];
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float *f) {
  Raw<T, VEC> r;
  if constexpr (VEC == 1) {
    r.u = from_f32<T>(f[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.w[i] = __float_as_uint(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 2) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(f[i], f[i + 1]);
      r.w[i / 2] = *reinterpret_cast<const uint32_t *>(&v);
    }
  }
  store_raw<T, VEC>(p, r);
}

}  // namespace la
