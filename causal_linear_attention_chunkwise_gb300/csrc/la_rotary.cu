// la_rotary.cu -- rotary positions of q and k, forward and backward.
//
//     (x_a, x_b) <- scale * (x_a cos - x_b sin, x_a sin + x_b cos),   angle = position * f
//
// for the pairs of the first `rot` values of a head, the rest copied; the
// backward pass turns by the negative angle.
//
// The angle is kept in turns, as a 64-bit fraction of one: F = f / 2 pi in units
// of 2^-64, so that position * F wraps at whole turns by itself and an angle is
// exact to position * 2^-64 turns however far the position lies (in fp32 a
// position of 10^6 would leave 4 digits of its angle).  The top two bits round to the
// quadrant; sine and cosine of the remainder, |theta| <= pi / 4, are their Taylor
// polynomials (next terms below 2e-9 and 2e-10).
//
// A thread owns V pairs of one token (two vectors) and walks over some of the
// token's heads, so that one sine and cosine serve them all: 8 of them cost 400
// instructions, a head 50.  The bytes bound it: 4 x (16 + 16) x 4096 x 64 bf16 takes 24 us, 5.6 TB/s.  Reading a projection's token-major slices and
// writing [B,H,L,d], or the other way round, changes strides only: a head's
// values of one token are whole 32-byte sectors on either side.
#include <cstdint>

#include "../../include/la_gb300.h"
#include "la_act.cuh"
#include "la_internal.h"

namespace la {
namespace {

constexpr int kThreads = 256;

// f / 2 pi in units of 2^-64, whole turns dropped; f = m 2^e with 24 bits of m.
__device__ __forceinline__ unsigned long long turns_per_token(float f) {
  constexpr unsigned long long k66 = 0xa2f9836e4e44152aull;  // 2^66 / 2 pi, rounded
  const uint32_t bits = __float_as_uint(f);
  const int ex = bits >> 23 & 0xff;
  const unsigned long long m = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int right = 152 - (ex ? ex : 1);  // F = m k66 2^-right
  const unsigned long long lo = m * k66, hi = __umul64hi(m, k66);
  unsigned long long F = 0;
  if (right >= 64) F = right < 128 ? hi >> (right - 64) : 0;
  else if (right > 0) F = lo >> right | hi << (64 - right);
  else if (right > -64) F = lo << -right;
  return bits >> 31 ? 0ull - F : F;
}

// Sine and cosine of a phase in units of 2^-64 turns.
__device__ __forceinline__ void sin_cos(unsigned long long phase, float *sine, float *cosine) {
  const unsigned long long up = phase + (1ull << 61);
  const int quadrant = (int)(up >> 62);
  const long long rest = (long long)((up & ((1ull << 62) - 1)) - (1ull << 61));
  const float t = (float)(int)(rest >> 30) * 3.6572952e-10f;  // 2 pi 2^-34
  const float u = t * t;
  float s = fmaf(u, 2.7557319e-6f, -1.9841270e-4f);
  s = fmaf(u, s, 8.3333333e-3f);
  s = fmaf(u, s, -1.6666667e-1f);
  s = fmaf(t * u, s, t);
  float c = fmaf(u, -2.7557319e-7f, 2.4801587e-5f);
  c = fmaf(u, c, -1.3888889e-3f);
  c = fmaf(u, c, 4.1666667e-2f);
  c = fmaf(u, c, -0.5f);
  c = fmaf(u, c, 1.f);
  const float a = quadrant & 1 ? c : s, b = quadrant & 1 ? s : c;
  *sine = quadrant & 2 ? -a : a;
  *cosine = (quadrant + 1) & 2 ? -b : b;
}

// One head of one token: the slot's two vectors at c0 and c1.
template <typename T, int V, bool INNER>
__device__ __forceinline__ void turn(Raw<T, V> &lo, Raw<T, V> &hi, const float *cosine,
                                     const float *sine, int live, T *y, int c0, int c1) {
  float a[V], b[V], p[V], q[V];
  lo.unpack(a);
  hi.unpack(b);
#pragma unroll
  for (int e = 0; e < V; ++e) p[e] = a[e], q[e] = b[e];
  if constexpr (INNER) {  // pairs of neighbours, V / 2 in each vector
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      if (e < live) {
        p[2 * e] = a[2 * e] * cosine[e] - a[2 * e + 1] * sine[e];
        p[2 * e + 1] = a[2 * e] * sine[e] + a[2 * e + 1] * cosine[e];
      }
      const int f = e + V / 2;
      if (f < live) {
        q[2 * e] = b[2 * e] * cosine[f] - b[2 * e + 1] * sine[f];
        q[2 * e + 1] = b[2 * e] * sine[f] + b[2 * e + 1] * cosine[f];
      }
    }
  } else if (live > 0) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      p[e] = a[e] * cosine[e] - b[e] * sine[e];
      q[e] = a[e] * sine[e] + b[e] * cosine[e];
    }
  }
  store_vec<T, V>(y + c0, p);
  if (c1 >= 0) store_vec<T, V>(y + c1, q);
}

// slots: of V pairs (or of two vectors to copy) in a head; hp: heads a thread
// walks over; groups_q: groups of hp heads of q, in front of k's.
template <typename T, int V, bool INNER>
__global__ void __launch_bounds__(kThreads)
rotary_kernel(const RotaryArgs a, int slots, int hp, int groups_q, long long items) {
  const long long item = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (item >= items) return;
  const long long bt = div_index(item, slots);
  const int slot = (int)(item - bt * slots);
  const long long b = div_index(bt, a.L);
  const int t = (int)(bt - b * a.L);
  if (a.lengths && t >= a.lengths[b]) return;
  const bool second = (int)blockIdx.y >= groups_q;
  const RotaryTensor x = second ? a.k : a.q, y = second ? a.k_out : a.q_out;
  const int heads = second ? a.heads_k : a.heads_q;
  const int h0 = ((int)blockIdx.y - (second ? groups_q : 0)) * hp;
  const int h1 = min(h0 + hp, heads);

  // Where the slot's vectors lie, and how many of its V pairs turn.
  const int half = a.rot / 2;
  int c0, c1, pair, live;
  if (INNER || a.interleaved) {
    c0 = 2 * slot * V, c1 = c0 + V, pair = slot * V, live = half - pair;
  } else if (slot * V < half) {
    c0 = slot * V, c1 = half + c0, pair = c0, live = V;
  } else {
    c0 = a.rot + 2 * (slot * V - half), c1 = c0 + V, pair = 0, live = 0;
  }
  if (c1 >= a.d) c1 = -1;
  float cosine[V], sine[V];
  if (live > 0) {
    long long pos = a.positions ? a.positions[bt] : t;
    if (a.offsets) pos += a.offsets[b];
    if (a.backward) pos = -pos;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float f = e < live ? __ldg(a.inv_freq + pair + e) : 0.f;
      sin_cos((unsigned long long)pos * turns_per_token(f), &sine[e], &cosine[e]);
      sine[e] *= a.scale;
      cosine[e] *= a.scale;
    }
  }
  const T *xp = static_cast<const T *>(x.p) + b * x.bs + t * x.ts + h0 * x.hs;
  T *yp = static_cast<T *>(y.p) + b * y.bs + t * y.ts + h0 * y.hs;
  int h = h0;
  for (; h + 2 <= h1; h += 2, xp += 2 * x.hs, yp += 2 * y.hs) {  // two heads' loads in flight
    Raw<T, V> lo = load_raw<T, V>(xp + c0), lo2 = load_raw<T, V>(xp + x.hs + c0);
    Raw<T, V> hi{}, hi2{};
    if (c1 >= 0) hi = load_raw<T, V>(xp + c1), hi2 = load_raw<T, V>(xp + x.hs + c1);
    turn<T, V, INNER>(lo, hi, cosine, sine, live, yp, c0, c1);
    turn<T, V, INNER>(lo2, hi2, cosine, sine, live, yp + y.hs, c0, c1);
  }
  if (h < h1) {
    Raw<T, V> lo = load_raw<T, V>(xp + c0), hi{};
    if (c1 >= 0) hi = load_raw<T, V>(xp + c1);
    turn<T, V, INNER>(lo, hi, cosine, sine, live, yp, c0, c1);
  }
}

template <typename T, int V, bool INNER>
cudaError_t launch_v(const RotaryArgs &a) {
  const int half = a.rot / 2;
  const int slots = INNER || a.interleaved
                        ? (a.d + 2 * V - 1) / (2 * V)
                        : half / V + ((a.d - a.rot) / V + 1) / 2;
  const long long items = (long long)a.B * a.L * slots;
  const int heads = a.heads_q + a.heads_k;
  // As many heads to a thread as leave 1024 threads to an SM, at most 8 (fp32: 4, whose vectors hold
  // half the pairs).  4 x (16 + 16) x 4096 x 64 bf16: 24 us with 8 and with 16, 26 with 4, 36 with
  // 2; 1 x (16 + 16) x 32767 x 128 fp32, half of each head turned: 169 with 8, 162 with 4, 158 with 2.
  int hp = sizeof(T) == 2 ? 8 : 4;
  while (hp > 1 && items * ((heads + hp - 1) / hp) < 152ll * 1024) hp /= 2;
  const int groups_q = (a.heads_q + hp - 1) / hp, groups_k = (a.heads_k + hp - 1) / hp;
  const long long blocks = (items + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffll || groups_q + groups_k > 65535) return cudaErrorInvalidConfiguration;
  rotary_kernel<T, V, INNER><<<dim3((unsigned)blocks, groups_q + groups_k), kThreads, 0, a.stream>>>(
      a, slots, hp, groups_q, items);
  return cudaGetLastError();
}

// The widest vectors that the alignment, the width and, for pairs half a width apart, the
// turned half allow: 16 bytes, or element by element.
template <typename T>
cudaError_t launch_t(const RotaryArgs &a) {
  constexpr int V = Pack16<T>::N;
  auto fits = [&](const RotaryTensor &x, int heads) {
    return heads == 0 || (reinterpret_cast<uintptr_t>(x.p) % 16 == 0 &&
                          (a.B == 1 || x.bs % V == 0) && (heads == 1 || x.hs % V == 0) &&
                          (a.L == 1 || x.ts % V == 0));
  };
  const bool wide = a.d % V == 0 && fits(a.q, a.heads_q) && fits(a.q_out, a.heads_q) &&
                    fits(a.k, a.heads_k) && fits(a.k_out, a.heads_k);
  if (wide && a.interleaved) return launch_v<T, V, true>(a);
  if (wide && a.rot / 2 % V == 0) return launch_v<T, V, false>(a);
  return launch_v<T, 1, false>(a);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs &a) {
  return a.dtype == LA_F32 ? launch_t<float>(a) : launch_t<__nv_bfloat16>(a);
}

}  // namespace la
