// la_mma.cuh -- warp-level matrix products of bf16 tiles in shared memory: 16-byte
// swizzled tiles, their fragments, and sums of bf16 planes that stand for fp32 values.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "la_ptx.cuh"

namespace la {

// Element (row, col) of a tile with rows of D bf16: 16-byte pieces of a row change
// places with the row, so that the 8 rows of an 8 x 8 matrix lie in different banks.
template <int D> __device__ __forceinline__ uint32_t tile_offset(int row, int col) {
  return (uint32_t)(row * D * 2 + (((col >> 3) ^ (row & 7)) << 4) + ((col & 7) << 1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// The fragments of a 16 x 16 matrix A[m][k], and of two 16 x 8 matrices B[k][n], n in
// n0 .. n0 + 15, each from a tile stored with its own rows or transposed.
template <int D>  // tile [m][k]
__device__ __forceinline__ void frag_a(uint32_t (&r)[4], uint32_t tile, int m0, int k0, int lane) {
  ldsm4(r, tile + tile_offset<D>(m0 + (lane & 15), k0 + (lane >> 4) * 8));
}
template <int D>  // tile [k][m]
__device__ __forceinline__ void frag_a_t(uint32_t (&r)[4], uint32_t tile, int m0, int k0,
                                         int lane) {
  ldsm4_t(r, tile + tile_offset<D>(k0 + (lane & 7) + (lane >> 4) * 8, m0 + (lane >> 3 & 1) * 8));
}
template <int D>  // tile [n][k]
__device__ __forceinline__ void frag_b(uint32_t (&r)[4], uint32_t tile, int n0, int k0, int lane) {
  ldsm4(r, tile + tile_offset<D>(n0 + (lane & 7) + (lane >> 4) * 8, k0 + (lane >> 3 & 1) * 8));
}
template <int D>  // tile [k][n]
__device__ __forceinline__ void frag_b_t(uint32_t (&r)[4], uint32_t tile, int n0, int k0,
                                         int lane) {
  ldsm4_t(r, tile + tile_offset<D>(k0 + (lane & 7) + (lane >> 3 & 1) * 8, n0 + (lane >> 4) * 8));
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
      "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A B for two neighbouring 8-column tiles, A and B sums of bf16 planes: the product of
// the first planes is added to c0, c1, those of planes p, q with 0 < p + q below the
// larger number of planes to s0, s1 (the others are below an fp32 rounding).  The tensor
// cores cut a sum's last bits off instead of rounding it, so the many small products
// get accumulators of their own, and their cuts are as small as they are.
template <int NA, int NB>
__device__ __forceinline__ void mma_planes(float (&c0)[4], float (&c1)[4], float (&s0)[4],
                                           float (&s1)[4], const uint32_t (&a)[NA][4],
                                           const uint32_t (&b)[NB][4]) {
  constexpr int N = NA > NB ? NA : NB;
#pragma unroll
  for (int s = N - 1; s > 0; --s)
#pragma unroll
    for (int p = 0; p < NA; ++p) {
      const int q = s - p;
      if (q < 0 || q >= NB) continue;
      mma16816(s0, a[p], b[q][0], b[q][1]);
      mma16816(s1, a[p], b[q][2], b[q][3]);
    }
  mma16816(c0, a[0], b[0][0], b[0][1]);
  mma16816(c1, a[0], b[0][2], b[0][3]);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Two fp32 values as sums of NP bf16 planes (three hold all 24 bits): plane p at out[p * stride].
// An infinity becomes a NaN.
template <int NP>
__device__ __forceinline__ void split(float x, float y, uint32_t *out, int stride) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const uint32_t v = pack_bf16(x, y);
    out[p * stride] = v;
    if (p + 1 < NP) {
      x -= bf16_lo(v);
      y -= bf16_hi(v);
    }
  }
}

}  // namespace la
