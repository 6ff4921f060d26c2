// la_chunk_bwd.cuh -- backward pass of chunkwise linear attention: the kernels.
//
// With S_t = a_t S_{t-1} + k_t v_t^T, o_t = S_t^T q_t (q, k after phi) and G_t the
// gradient of S_t, G_t = q_t do_t^T + a_{t+1} G_{t+1}:
//
//     dq_t = S_t do_t,   dk_t = G_t v_t,   dv_t = G_t^T k_t,   dlog a_t = a_t <G_t, S_{t-1}>.
//
// In chunks of C tokens, with L_t the sum of the log decays of the chunk's tokens up to t, D_ji =
// e^(L_j - L_i) for j >= i (else 0), S the state before the chunk and G the gradient
// of the state behind it:
//
//     dq = (dO V^T . D) K + e^L dO S^T             S <- e^L_C S + (e^(L_C - L) K)^T V
//     dk = (dO V^T . D)^T Q + e^(L_C - L) V G^T    G <- e^L_C G + (e^L Q)^T dO
//     dv = (Q K^T . D)^T dO + e^(L_C - L) K G
//
// dq needs S, which runs forward; dk and dv need G, which runs backward.  So two
// kernels, each one walk over the chunks with its state in registers (fp32).  A long
// sequence is cut into segments that run side by side: a first kernel forms every
// segment's own share of S and G, a second one strings them together.
//
// Most bf16 calls run in la_chunk_bwd_tc.cu.  The kernels here take what enters as three bf16 planes,
// fp32 tensors and phi = elu + 1 where an fp32 output is wanted (there is no such form there; at
// width 128 three planes of 128 tokens would not fit), and many short bf16 sequences.  A warp owns 16
// tokens of a
// chunk (with others, which take other columns) and computes its rows of the score matrices in the
// orientation that its products need (dO V^T for dq, V dO^T and K Q^T for dk and dv).
//
// A decay's gradient counts the pairs (i < t <= j) that it lies between: pairs within
// the chunk (sums over Q K^T . dO V^T . D), pairs with one token in it (dot
// products of the rows of dq's and dk's second terms with q and k), and pairs
// around it (<G, e^L_C S>, which follows from chunk to chunk by the same sums).
// Those of a chunk are added up pair by pair, so that a token that nearly resets the state, whose
// gradient is small beside its neighbours', has all of its digits; q dq - k dk summed from the
// sequence's end would lose the short decays to the long sums.  Followed from chunk to chunk the
// sums' errors stay, and a per-head decay's gradient adds them up over all tokens: every 512
// tokens, and at every chunk in which one token decays by more than 2^-5, S is kept for the
// backward walk, which forms <G, e^L_C S> anew (2 x 32 x 8192 x 128
// with per-head decays: 4.8e-7 off; 4.5e-6 without, growing with the length to the power 1.5).
//
// Precision.  Products run in bf16 with fp32 sums.  With bf16 inputs and outputs the
// scores, the states and what a decay multiplies round once to bf16 as operands (the state itself
// stays fp32), each about as large as the outputs' own rounding; phi's values of elu + 1 enter dq and dk
// as two planes, for a third such would be theirs (dq and dk 3.0e-3 off with one plane, 2.35e-3
// with two).  The fp32 outputs (ddecay, dS0) take those operands as three bf16
// planes, which hold all of an fp32 value's bits; fp32 inputs, and phi = elu + 1
// where an fp32 output is wanted, enter as three planes too (v and dO of bf16 inputs as one).
//
// What bounds these kernels: mma.sync, 600 TFLOP/s at best, times six for three planes by three
// (grad_kv of 3 x 5 x 777 x 64 x 128 fp32: the tensor pipe 35% busy, with two warps to a scheduler and
// a chunk's steps one after another).
#pragma once

#include <cstdint>

#include "../../include/la_gb300.h"
#include "la_act.cuh"
#include "la_internal.h"
#include "la_mma.cuh"
#include "la_tc_sync.cuh"

namespace la {

constexpr int kShares = 16;  // warps whose sums a <G, S> is left as, at most
constexpr float kStrong = -5.f;  // log2 of a strong decay of one token

// What the kernels get: the tensors, and the plan.
struct ChunkBwd {
  const void *q, *k, *v, *dO;
  void *dq, *dk, *dv;
  const float *decay, *S0, *dSf;
  float *dS0;
  int H, L, n_k, n_v;          // n_k, n_v: d_k and d_v
  int phi, decay_kind;
  int chunks, segments, per;   // per: chunks of a segment
  float *U, *W;                // [seq][segments - 1][d_k d_v]: states between segments
  float *total;                // [seq][segments] log2 of a segment's decay
  float2 *lam;                 // [seq][chunks][C] log2 of the decay from a chunk's start to a
                               // token, as a sum of two floats (unused without a decay)
  // Shares of ddecay [seq][L], or null: the pairs of a token with tokens before its chunk (rq)
  // and behind it (rk), the pairs of its block of the chunk that it lies between (rc), and its
  // pairs with the chunk's blocks before (cs) and behind (rs) its own, where a chunk has blocks.
  float *rq, *rk, *rc, *cs, *rs;
  float2 *across;              // [seq][chunks] pairs of a chunk's blocks around block 1 and block 2
  float *around;               // [seq][segments] <G, e^L_C S> of a segment's last chunk
  unsigned char *strong;       // [seq][chunks] whether a token of the chunk decays by kStrong
  float *kept;                 // [seq][chunks - 1] S before a chunk that keeps() it: d_k d_v
                               // floats, on tcgen05 those of the padded widths
  float *between;              // [seq][chunks - 1][kShares] <G, e^L_C S> of such a chunk
  int every;

  // Whether chunk c, with its segment ending in front of c1, is one that S is kept for: the last
  // of `every` chunks, and one with a strong decay, whose token's gradient is so much smaller
  // than its neighbours' that a difference of theirs would not leave much of it.
  __device__ __forceinline__ bool keeps(int seq, int c, int c1) const {
    return kept && c + 1 < c1 && ((c + 1) % every == 0 || strong[(size_t)seq * chunks + c]);
  }
  __device__ __forceinline__ size_t keep_slot(int seq, int c) const {
    return (size_t)seq * (chunks - 1) + c;
  }
};

// T: element type; D: padded width (d_k, d_v <= D); C: tokens of a chunk; NI: planes of q
// and k after phi (two, for outputs in bf16: phi's own rounding would be added to theirs); NM: planes
// of the states and of what enters them.
template <typename T_, int D_, int C_, int NI_, int NM_> struct BwdConfig {
  using T = T_;
  static constexpr int D = D_, C = C_, NI = NI_, NM = NM_;
  static constexpr int NV = sizeof(T) == 2 ? 1 : NI;  // of v and dO, which are not mapped
  static constexpr int NO = NI < 3 ? 1 : 3;           // planes of scores
  static constexpr int WARPS = D / 16;         // each owns 16 rows of the state
  static constexpr int ROWS = C / 16;          // groups of 16 tokens
  static constexpr int SPLIT = WARPS / ROWS;   // warps that share a group, by columns
  static constexpr int COLS = D / SPLIT;       // columns of a warp's outputs
  static constexpr int THREADS = WARPS * 32;
  static constexpr int BLOCKS = D == 64 ? 3 : 1;  // to an SM
  // Three planes of scores are six products: the warps of a group form 8 of their columns each
  // and share them in shared memory, where four do (2 x 16 x 4096 x 128 fp32: 1237 us before,
  // 1131 after).  At D = 64 two warps share a group, and three blocks an SM.
  static constexpr bool SHARE = NI == 3 && SPLIT == C / 8;
  static constexpr uint32_t SCORE_ROW = C * 2 + 16, SCORES = C * SCORE_ROW;  // bytes
  static constexpr uint32_t TILE = C * D * 2;  // bytes of one plane
  static constexpr uint32_t STATE = D * D * 2;
  static_assert(WARPS % ROWS == 0 && COLS % 16 == 0, "whole column tiles");
};

// The sum of v over the warp's lanes in front of this one (FRONT) or behind it, within groups of
// WIDTH lanes.
template <bool FRONT, int WIDTH> __device__ __forceinline__ float lanes_sum(float v, int lane) {
  const int at = lane % WIDTH;
  float x = v;
#pragma unroll
  for (int off = 1; off < WIDTH; off <<= 1) {
    const float y = FRONT ? __shfl_up_sync(0xffffffffu, x, off, WIDTH)
                          : __shfl_down_sync(0xffffffffu, x, off, WIDTH);
    if (FRONT ? at >= off : at + off < WIDTH) x += y;
  }
  const float y = FRONT ? __shfl_up_sync(0xffffffffu, x, 1, WIDTH)
                        : __shfl_down_sync(0xffffffffu, x, 1, WIDTH);
  return FRONT ? at ? y : 0.f : at < WIDTH - 1 ? y : 0.f;
}
// Their sum over such a group.
template <int WIDTH> __device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = WIDTH / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Per-chunk decay factors in shared memory.
template <int C> struct ChunkDecay {
  float2 lam[C];  // log2 of the decay from the chunk's start, as a sum of two floats
  float head[C];  // e^L
  float tail[C];  // e^(L_C - L)
  float2 all;     // e^L_C, as a sum of two floats
};

// The decay between two tokens.
__device__ __forceinline__ float decay_between(float2 later, float2 earlier) {
  return ex2_approx((later.x - earlier.x) + (later.y - earlier.y));
}

// 2^x as a sum of two floats, to 2^-26 relative.  A state is multiplied by its chunks' decays
// again and again: the 2^-23 that an exponential may be off would add up over the chunks that a
// slow decay spans.  2^n e^t with |t| <= 0.35: 1 + t, whose rounding is kept, and the rest of e^t's
// series.
__device__ __forceinline__ float2 exp2_two(float2 x) {
  if (!(fabsf(x.x) <= 126.f)) return make_float2(ex2_approx(x.x), 0.f);
  const float n = rintf(x.x), f = x.x - n;
  const float t = f * 0.693147182f;  // ln 2 = 0.693147182 - 1.90465421e-9
  const float low = fmaf(f, 0.693147182f, -t) + fmaf(x.y, 0.693147182f, f * -1.90465421e-9f);
  float s = 1.f / 40320;
  s = fmaf(s, t, 1.f / 5040), s = fmaf(s, t, 1.f / 720), s = fmaf(s, t, 1.f / 120);
  s = fmaf(s, t, 1.f / 24), s = fmaf(s, t, 1.f / 6), s = fmaf(s, t, 0.5f);
  s *= t * t;
  const float one = 1.f + t, rest = (t - (one - 1.f)) + fmaf(low, one + s, s);
  const float hi = one + rest, scale = __int_as_float(((int)n + 127) << 23);
  return make_float2(hi * scale, (rest - (hi - one)) * scale);
}
// all s + u
__device__ __forceinline__ float decayed_sum(float2 all, float s, float u) {
  return fmaf(all.x, s, fmaf(all.y, s, u));
}

// The factors of a chunk, by its first C threads.
template <int C>
__device__ __forceinline__ void chunk_decay(const ChunkBwd &p, int seq, int c, ChunkDecay<C> &s) {
  const int t = threadIdx.x;
  if (t >= C) return;
  float2 own = make_float2(0.f, 0.f), end = own;
  if (p.decay_kind != LA_DECAY_NONE) {
    const float2 *lam = p.lam + ((size_t)seq * p.chunks + c) * C;
    own = lam[t], end = lam[C - 1];
  }
  s.lam[t] = own;
  s.head[t] = ex2_approx(own.x);
  s.tail[t] = decay_between(end, own);
  if (t == 0) s.all = exp2_two(end);
}

// Rows t0 .. t0 + C - 1 of a [L, width] tensor on their way to a tile's planes, after phi if
// MAP; zeros past the last token and past the width.  All of a chunk's tiles are fetched before the
// first is put: a fetch behind a put would wait for the one before it (2 x 16 x 4096 x 128
// fp32 with token decays: 1053 us; tile by tile 1126).
template <typename F> struct TileRows {
  using T = typename F::T;
  static constexpr int N = F::C * F::D / 8 / F::THREADS, V = 16 / sizeof(T), K = 8 / V;
  Raw<T, V> v[N][K];

  __device__ __forceinline__ static bool place(const ChunkBwd &p, int width, int t0, int i, int &row,
                                               int &col) {
    const int vec = threadIdx.x + i * F::THREADS;
    row = vec / (F::D / 8), col = vec % (F::D / 8) * 8;
    return t0 + row < p.L && col < width;
  }
  __device__ __forceinline__ void fetch(const T *rows, const ChunkBwd &p, int width, int t0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      int row, col;
      const bool live = place(p, width, t0, i, row, col);
      const T *from = rows + (live ? (long long)(t0 + row) * width + col : 0);
#pragma unroll
      for (int k = 0; k < K; ++k) v[i][k] = load_raw<T, V>(from + k * V);
    }
  }
  template <bool MAP, int NP = MAP ? F::NI : F::NV>
  __device__ __forceinline__ void put(uint32_t tile, const ChunkBwd &p, int width, int t0) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      int row, col;
      const bool live = place(p, width, t0, i, row, col);
      uint32_t out[NP][4];
      if (NP == 1 && !(MAP && p.phi == LA_PHI_ELU1)) {  // bf16 as it is
#pragma unroll
        for (int e = 0; e < 4; ++e) out[0][e] = live ? v[i][0].w[e] : 0;
      } else {
        float f[8];
#pragma unroll
        for (int k = 0; k < K; ++k) v[i][k].unpack(f + k * V);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (MAP) f[e] = NP == 1 ? feature_map(p.phi, f[e]) : feature_map_precise(p.phi, f[e]);
          f[e] = live ? f[e] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) split<NP>(f[2 * e], f[2 * e + 1], &out[0][e], 4);
      }
      const uint32_t to = tile + tile_offset<F::D>(row, col);
#pragma unroll
      for (int n = 0; n < NP; ++n)
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to + n * F::TILE),
                     "r"(out[n][0]), "r"(out[n][1]), "r"(out[n][2]), "r"(out[n][3])
                     : "memory");
    }
  }
};

// A warp's 16 rows of a state, as accumulators: row g or g + 8, columns 8 n + 2 (lane % 4).
template <typename F> struct StateRows {
  float c[F::D / 8][4];

  __device__ __forceinline__ void load(const float *src, const ChunkBwd &p, int warp, int lane) {
#pragma unroll
    for (int n = 0; n < F::D / 8; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = warp * 16 + lane / 4 + 8 * h, col = n * 8 + lane % 4 * 2;
        float2 x = make_float2(0.f, 0.f);
        if (src && row < p.n_k && col < p.n_v)
          x = *reinterpret_cast<const float2 *>(src + (size_t)row * p.n_v + col);
        c[n][2 * h] = x.x, c[n][2 * h + 1] = x.y;
      }
  }
  __device__ __forceinline__ void store(float *dst, const ChunkBwd &p, int warp, int lane) const {
#pragma unroll
    for (int n = 0; n < F::D / 8; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = warp * 16 + lane / 4 + 8 * h, col = n * 8 + lane % 4 * 2;
        if (row < p.n_k && col < p.n_v)
          *reinterpret_cast<float2 *>(dst + (size_t)row * p.n_v + col) =
              make_float2(c[n][2 * h], c[n][2 * h + 1]);
      }
  }
  // The state as planes of a bf16 tile [d_k][d_v].
  __device__ __forceinline__ void planes(char *tile, int warp, int lane) const {
#pragma unroll
    for (int n = 0; n < F::D / 8; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[F::NM];
        split<F::NM>(c[n][2 * h], c[n][2 * h + 1], w, 1);
        const uint32_t at = tile_offset<F::D>(warp * 16 + lane / 4 + 8 * h, n * 8 + lane % 4 * 2);
#pragma unroll
        for (int m = 0; m < F::NM; ++m)
          *reinterpret_cast<uint32_t *>(tile + m * F::STATE + at) = w[m];
      }
  }
  // c <- all c + sum over tokens of weight x (x) y: x's tile [token][d_k], y's [token][d_v].
  // A chunk's sum is formed by itself and then added, with an fp32 rounding: the tensor
  // cores' cuts would add up over the chunks.
  __device__ __forceinline__ void update(uint32_t x, uint32_t y, const float *weight, float2 all,
                                         int warp, int lane) {
    uint32_t w[F::C / 16][F::NM][4];
#pragma unroll
    for (int k = 0; k < F::C / 16; ++k) {
      uint32_t a[F::NI][4];
#pragma unroll
      for (int i = 0; i < F::NI; ++i)
        frag_a_t<F::D>(a[i], x + i * F::TILE, warp * 16, k * 16, lane);
#pragma unroll
      for (int r = 0; r < 4; ++r) {  // registers 2 and 3 hold the tokens 8 further on
        const float2 f =
            *reinterpret_cast<const float2 *>(weight + k * 16 + (r / 2) * 8 + lane % 4 * 2);
        float lo = 0.f, hi = 0.f;
#pragma unroll
        for (int i = F::NI - 1; i >= 0; --i) lo += bf16_lo(a[i][r]), hi += bf16_hi(a[i][r]);
        split<F::NM>(lo * f.x, hi * f.y, &w[k][0][r], 4);
      }
    }
#pragma unroll
    for (int n = 0; n < F::D / 8; n += 2) {
      float sum[2][4] = {}, small[2][4] = {};
#pragma unroll
      for (int k = 0; k < F::C / 16; ++k) {
        uint32_t b[F::NV][4];
#pragma unroll
        for (int i = 0; i < F::NV; ++i)
          frag_b_t<F::D>(b[i], y + i * F::TILE, n * 8, k * 16, lane);
        mma_planes<F::NM, F::NV>(sum[0], sum[1], small[0], small[1], w[k], b);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          c[n + j][e] = decayed_sum(all, c[n + j][e],
                                    F::NM > 1 ? sum[j][e] + small[j][e] : sum[j][e]);
    }
  }
};

// A state from its three planes in shared memory, which hold all of its bits, to global memory,
// and the product of such a one with the state whose planes are there: from the registers,
// both made the walks spill (3 x 5 x 777 x 64 x 128 fp32: 50 and 63 us against 40 and 57).
template <typename F> __device__ __forceinline__ float plane_sum(const char *tile, int row, int col) {
  const uint32_t at = tile_offset<F::D>(row, col);
  float s = 0.f;
#pragma unroll
  for (int m = F::NM - 1; m >= 0; --m)
    s += __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(tile + m * F::STATE + at));
  return s;
}
template <typename F>
__device__ __forceinline__ void keep_state(float *dst, const char *tile, const ChunkBwd &p) {
  const int shift = 31 - __clz(p.n_v), all = p.n_k << shift;  // the widths are powers of two
#pragma unroll 4
  for (int e = threadIdx.x; e < all; e += F::THREADS)
    dst[e] = plane_sum<F>(tile, e >> shift, e & (p.n_v - 1));
}
template <typename F>
__device__ __forceinline__ float dot_kept(const float *src, const char *tile, const ChunkBwd &p) {
  const int shift = 31 - __clz(p.n_v), all = p.n_k << shift;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  for (int e = threadIdx.x; e < all; e += 4 * F::THREADS)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = e + i * F::THREADS;
      if (x < all)
        s[i] = fmaf(src[x], plane_sum<F>(tile, x >> shift, x & (p.n_v - 1)), s[i]);
    }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// acc += small where there were small products.
template <bool ANY, int NT>
__device__ __forceinline__ void add_small(float (&acc)[NT][4], const float (&small)[NT][4]) {
  if constexpr (ANY) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] += small[n][e];
  }
}

// acc[n] += X Y^T over the widths: rows m0 .. of X's tile, rows n0 + 16 j of Y's (live(j)).
template <typename F, int NT, int NX, int NY, typename Live>
__device__ __forceinline__ void rows_times_rows(float (&acc)[NT][4], uint32_t x, uint32_t x_plane,
                                                int m0, uint32_t y, uint32_t y_plane, int n0,
                                                int lane, Live live) {
  float small[NT][4] = {};
#pragma unroll
  for (int k0 = 0; k0 < F::D; k0 += 16) {
    uint32_t a[NX][4];
#pragma unroll
    for (int i = 0; i < NX; ++i) frag_a<F::D>(a[i], x + i * x_plane, m0, k0, lane);
#pragma unroll
    for (int j = 0; j < NT / 2; ++j) {
      if (!live(j)) continue;
      uint32_t b[NY][4];
#pragma unroll
      for (int i = 0; i < NY; ++i) frag_b<F::D>(b[i], y + i * y_plane, n0 + j * 16, k0, lane);
      mma_planes<NX, NY>(acc[2 * j], acc[2 * j + 1], small[2 * j], small[2 * j + 1], a, b);
    }
  }
  add_small<(NX > 1 || NY > 1)>(acc, small);
}

// acc[n] += X Y: rows m0 .. of X's tile, columns n0 + 8 n of Y's.
template <typename F, int NT, int NX, int NY>
__device__ __forceinline__ void rows_times_cols(float (&acc)[NT][4], uint32_t x, uint32_t x_plane,
                                                int m0, uint32_t y, uint32_t y_plane, int n0,
                                                int lane) {
  float small[NT][4] = {};
#pragma unroll
  for (int k0 = 0; k0 < F::D; k0 += 16) {
    uint32_t a[NX][4];
#pragma unroll
    for (int i = 0; i < NX; ++i) frag_a<F::D>(a[i], x + i * x_plane, m0, k0, lane);
#pragma unroll
    for (int n = 0; n < NT; n += 2) {
      uint32_t b[NY][4];
#pragma unroll
      for (int i = 0; i < NY; ++i) frag_b_t<F::D>(b[i], y + i * y_plane, n0 + n * 8, k0, lane);
      mma_planes<NX, NY>(acc[n], acc[n + 1], small[n], small[n + 1], a, b);
    }
  }
  add_small<(NX > 1 || NY > 1)>(acc, small);
}

// 16 x 8 scores: rows m0 .. of X's tile times rows n0 .. of Y's, over the widths.
template <typename F, int NX, int NY>
__device__ __forceinline__ void score_tile(float (&acc)[4], uint32_t x, int m0, uint32_t y, int n0,
                                           int lane) {
  constexpr int N = NX > NY ? NX : NY;
  float small[4] = {};
#pragma unroll
  for (int k0 = 0; k0 < F::D; k0 += 32) {
    uint32_t b[NY][4];
#pragma unroll
    for (int i = 0; i < NY; ++i)
      ldsm4(b[i], y + i * F::TILE + tile_offset<F::D>(n0 + (lane & 7), k0 + (lane >> 3) * 8));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t a[NX][4];
#pragma unroll
      for (int i = 0; i < NX; ++i) frag_a<F::D>(a[i], x + i * F::TILE, m0, k0 + h * 16, lane);
#pragma unroll
      for (int o = N - 1; o > 0; --o)
#pragma unroll
        for (int i = 0; i < NX; ++i)
          if (o - i >= 0 && o - i < NY) mma16816(small, a[i], b[o - i][2 * h], b[o - i][2 * h + 1]);
      mma16816(acc, a[0], b[0][2 * h], b[0][2 * h + 1]);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] += small[e];
}

// Scores as planes of an operand: from accumulators (tiles of 8 tokens), and by shared memory,
// from 16 x 8 tiles.
template <typename F>
__device__ __forceinline__ void score_frag(uint32_t (&a)[F::NO][4], const float (&w)[F::C / 8][4],
                                           int j) {
  split<F::NO>(w[2 * j][0], w[2 * j][1], &a[0][0], 4);
  split<F::NO>(w[2 * j][2], w[2 * j][3], &a[0][1], 4);
  split<F::NO>(w[2 * j + 1][0], w[2 * j + 1][1], &a[0][2], 4);
  split<F::NO>(w[2 * j + 1][2], w[2 * j + 1][3], &a[0][3], 4);
}
template <typename F>
__device__ __forceinline__ void score_frag(uint32_t (&a)[F::NO][4], uint32_t scores, int m0, int j,
                                           int lane) {
#pragma unroll
  for (int m = 0; m < F::NO; ++m)
    ldsm4(a[m], scores + m * F::SCORES + (m0 + (lane & 15)) * F::SCORE_ROW +
                    (j * 16 + (lane >> 4) * 8) * 2);
}
template <typename F>
__device__ __forceinline__ void put_scores(char *scores, const float (&w)[4], int m0, int n0,
                                           int lane) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t o[F::NO];
    split<F::NO>(w[2 * h], w[2 * h + 1], o, 1);
#pragma unroll
    for (int m = 0; m < F::NO; ++m)
      *reinterpret_cast<uint32_t *>(scores + m * F::SCORES + (m0 + lane / 4 + 8 * h) * F::SCORE_ROW +
                                    (n0 + lane % 4 * 2) * 2) = o[m];
  }
}

// acc[n] += W Y over the chunk's tokens: W's operand by frag(planes, 16 tokens), Y's tile
// [token][.], columns n0 + 8 n.
template <typename F, int NT, int NY, typename Frag, typename Live>
__device__ __forceinline__ void scores_times_cols(float (&acc)[NT][4], Frag frag, uint32_t y,
                                                  int n0, int lane, Live live) {
  float small[NT][4] = {};
#pragma unroll
  for (int j = 0; j < F::C / 16; ++j) {
    if (!live(j)) continue;
    uint32_t a[F::NO][4];
    frag(a, j);
#pragma unroll
    for (int n = 0; n < NT; n += 2) {
      uint32_t b[NY][4];
#pragma unroll
      for (int i = 0; i < NY; ++i) frag_b_t<F::D>(b[i], y + i * F::TILE, n0 + n * 8, j * 16, lane);
      mma_planes<F::NO, NY>(acc[n], acc[n + 1], small[n], small[n + 1], a, b);
    }
  }
  add_small<(F::NO > 1 || NY > 1)>(acc, small);
}

// A warp's 16 x COLS outputs to rows t0 + r0 + .. of a [L, width] tensor; with phi = elu + 1
// times its derivative at raw (e^x up to 0, then 1).
template <typename F, int NT>
__device__ __forceinline__ void store_rows(const float (&acc)[NT][4], void *dst, const void *raw,
                                           const ChunkBwd &p, int width, int t, int n0, int lane) {
  using T = typename F::T;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = t + lane / 4 + 8 * h;
    if (row >= p.L) continue;
    T *to = static_cast<T *>(dst) + (long long)row * width;
    const T *x = static_cast<const T *>(raw) + (long long)row * width;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int c = n0 + n * 8 + lane % 4 * 2;
      if (c >= width) continue;
      float f[2] = {acc[n][2 * h], acc[n][2 * h + 1]};
      if (raw && p.phi == LA_PHI_ELU1) {
        float y[2];
        load_raw<T, 2>(x + c).unpack(y);
#pragma unroll
        for (int e = 0; e < 2; ++e) f[e] *= y[e] > 0.f ? 1.f : expf(y[e]);
      }
      store_vec<T, 2>(to + c, f);
    }
  }
}

// <a row of acc, the same row of x after phi>, summed over a warp's columns: rows g and g + 8.
template <typename F, int NT>
__device__ __forceinline__ float2 row_dots(const float (&acc)[NT][4], const void *raw,
                                           const ChunkBwd &p, int width, int t, int n0, int lane) {
  using T = typename F::T;
  float s[2] = {0.f, 0.f};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = t + lane / 4 + 8 * h;
    if (row < p.L) {
      const T *x = static_cast<const T *>(raw) + (long long)row * width;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int c = n0 + n * 8 + lane % 4 * 2;
        if (c >= width) continue;
        float y[2];
        load_raw<T, 2>(x + c).unpack(y);
        s[h] = fmaf(acc[n][2 * h], feature_map_precise(p.phi, y[0]), s[h]);
        s[h] = fmaf(acc[n][2 * h + 1], feature_map_precise(p.phi, y[1]), s[h]);
      }
    }
    s[h] += __shfl_xor_sync(0xffffffffu, s[h], 1);
    s[h] += __shfl_xor_sync(0xffffffffu, s[h], 2);
  }
  return make_float2(s[0], s[1]);
}

template <typename F> struct BwdShared {
  ChunkDecay<F::C> decay;
  float rows[F::SPLIT][F::C];  // row sums of the warps that share a group
  float cols[F::ROWS][F::C];   // pairs of a group's rows that the chunk's tokens lie between
  float pairs[F::SHARE ? F::SPLIT : 1][F::C];  // row sums of the pairs of shared scores
  float sum[F::WARPS];
};
template <typename F> constexpr uint32_t bwd_shared_bytes() {
  return (sizeof(BwdShared<F>) + 127) / 128 * 128;
}

// The segment's own share of S (blockIdx.y = 0: segments 0 .. n - 2) or of G (1: segments 1 .. n - 1).
template <typename F> constexpr uint32_t share_smem() {
  return bwd_shared_bytes<F>() + (F::NI + F::NV) * F::TILE;
}
template <typename F>
__global__ void __launch_bounds__(F::THREADS) segment_share_kernel(const ChunkBwd p) {
  extern __shared__ __align__(128) char smem[];
  auto &sh = *reinterpret_cast<BwdShared<F> *>(smem);
  const uint32_t tiles = smem_u32(smem) + bwd_shared_bytes<F>();
  constexpr uint32_t X = F::NI * F::TILE;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int seq = blockIdx.x / (p.segments - 1), of = blockIdx.x % (p.segments - 1);
  const bool back = blockIdx.y != 0;
  const int seg = back ? of + 1 : of;
  const int c0 = seg * p.per, c1 = min(c0 + p.per, p.chunks), n = c1 - c0;
  const size_t ek = (size_t)seq * p.L * p.n_k, ev = (size_t)seq * p.L * p.n_v;
  using T = typename F::T;
  const T *x = static_cast<const T *>(back ? p.q : p.k) + ek;
  const T *y = static_cast<const T *>(back ? p.dO : p.v) + ev;
  auto token = [&](int i) { return (back ? c1 - 1 - i : c0 + i) * F::C; };
  auto load = [&](int i) {
    TileRows<F> a, b;
    a.fetch(x, p, p.n_k, token(i)), b.fetch(y, p, p.n_v, token(i));
    a.template put<true>(tiles, p, p.n_k, token(i));
    b.template put<false>(tiles + X, p, p.n_v, token(i));
  };
  StateRows<F> state;
  state.load(nullptr, p, warp, lane);
  double total = 0.0;
  for (int i = 0; i < n; ++i) {
    load(i);
    chunk_decay<F::C>(p, seq, token(i) / F::C, sh.decay);
    __syncthreads();
    total += (double)sh.decay.lam[F::C - 1].x + sh.decay.lam[F::C - 1].y;
    state.update(tiles, tiles + X, back ? sh.decay.head : sh.decay.tail, sh.decay.all, warp, lane);
    __syncthreads();
  }
  const size_t slot = (size_t)seq * (p.segments - 1) + of;
  state.store((back ? p.W : p.U) + slot * p.n_k * p.n_v, p, warp, lane);
  if (threadIdx.x == 0 && (!back || seg == p.segments - 1))
    p.total[(size_t)seq * p.segments + seg] = (float)total;
}

// dq: a walk forward over a segment's chunks.
template <typename F> constexpr uint32_t grad_q_smem() {
  return bwd_shared_bytes<F>() + (F::NI + 2 * F::NV) * F::TILE + F::NM * F::STATE +
         F::SHARE * F::NO * F::SCORES;
}
template <typename F>
__global__ void __launch_bounds__(F::THREADS, F::BLOCKS) grad_q_kernel(const ChunkBwd p) {
  extern __shared__ __align__(128) char smem[];
  auto &sh = *reinterpret_cast<BwdShared<F> *>(smem);
  char *state_tile = smem + bwd_shared_bytes<F>();
  const uint32_t S = smem_u32(state_tile), tiles = S + F::NM * F::STATE;
  constexpr uint32_t X = F::NI * F::TILE, Y = F::NV * F::TILE;
  char *scores = state_tile + F::NM * F::STATE + X + 2 * Y;
  constexpr int NT = F::COLS / 8;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int group = warp % F::ROWS, part = warp / F::ROWS;
  const int r0 = group * 16, n0 = part * F::COLS;
  const int seq = blockIdx.x / p.segments, seg = blockIdx.x % p.segments;
  const int c0 = seg * p.per, c1 = min(c0 + p.per, p.chunks);
  const size_t ek = (size_t)seq * p.L * p.n_k, ev = (size_t)seq * p.L * p.n_v;
  const size_t es = (size_t)p.n_k * p.n_v;
  using T = typename F::T;
  const T *k = static_cast<const T *>(p.k) + ek, *v = static_cast<const T *>(p.v) + ev;
  const T *q = static_cast<const T *>(p.q) + ek, *dO = static_cast<const T *>(p.dO) + ev;
  auto load = [&](int t) {
    TileRows<F> a, b, c;
    a.fetch(k, p, p.n_k, t), b.fetch(v, p, p.n_v, t), c.fetch(dO, p, p.n_v, t);
    a.template put<true>(tiles, p, p.n_k, t);
    b.template put<false>(tiles + X, p, p.n_v, t);
    c.template put<false>(tiles + X + Y, p, p.n_v, t);
  };
  StateRows<F> state;
  state.load(seg ? p.U + ((size_t)seq * (p.segments - 1) + seg - 1) * es
                 : p.S0 ? p.S0 + (size_t)seq * es : nullptr, p, warp, lane);
  state.planes(state_tile, warp, lane);
  for (int c = c0; c < c1; ++c) {
    const int t0 = c * F::C;
    const uint32_t tk = tiles, tv = tk + X, td = tv + Y;
    const bool keep = F::NI == 3 && p.keeps(seq, c, c1);
    load(t0);
    chunk_decay<F::C>(p, seq, c, sh.decay);
    __syncthreads();
    if (keep)
      keep_state<F>(p.kept + p.keep_slot(seq, c) * es, state_tile, p);
    // dO V^T . D: rows j of the group, tokens i <= j
    float w[F::C / 8][4] = {};
    auto live = [&](int j) { return j <= group; };
    auto masked = [&](float &x, int e, int col) {
      const int j = r0 + lane / 4 + e / 2 * 8, i = col + lane % 4 * 2 + e % 2;
      if (p.decay_kind != LA_DECAY_NONE)
        x *= decay_between(sh.decay.lam[j], sh.decay.lam[i <= j ? i : j]);
      x = i <= j ? x : 0.f;
    };
    if constexpr (F::SHARE) {
      if (live(part / 2)) {
        float x[4] = {};
        score_tile<F, F::NV, F::NV>(x, td, r0, tv, part * 8, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) masked(x[e], e, part * 8);
        put_scores<F>(scores, x, r0, part * 8, lane);
      }
    } else {
      rows_times_rows<F, F::C / 8, F::NV, F::NV>(w, td, F::TILE, r0, tv, F::TILE, 0, lane, live);
#pragma unroll
      for (int n = 0; n < F::C / 8; ++n) {
        if (n / 2 > group) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) masked(w[n][e], e, n * 8);
      }
    }
    float acc[NT][4] = {};
    rows_times_rows<F, NT, F::NV, F::NM>(acc, td, F::TILE, r0, S, F::STATE, n0, lane,
                                         [](int) { return true; });
    const float h0 = sh.decay.head[r0 + lane / 4], h1 = sh.decay.head[r0 + lane / 4 + 8];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n][0] *= h0, acc[n][1] *= h0, acc[n][2] *= h1, acc[n][3] *= h1;
    if (p.rq) {
      const float2 d = row_dots<F, NT>(acc, q, p, p.n_k, t0 + r0, n0, lane);
      if (lane % 4 == 0) {
        sh.rows[part][r0 + lane / 4] = d.x;
        sh.rows[part][r0 + lane / 4 + 8] = d.y;
      }
    }
    if (F::SHARE) __syncthreads();
    auto frag = [&](uint32_t (&a)[F::NO][4], int j) {
      if constexpr (F::SHARE) score_frag<F>(a, smem_u32(scores), r0, j, lane);
      else score_frag<F>(a, w, j);
    };
    scores_times_cols<F, NT, F::NI>(acc, frag, tk, n0, lane, live);
    store_rows<F, NT>(acc, static_cast<T *>(p.dq) + ek, q, p, p.n_k, t0 + r0, n0, lane);
    float around = 0.f;
    if (c + 1 < c1) {
      state.update(tk, tv, sh.decay.tail, sh.decay.all, warp, lane);
    } else if (p.rq) {  // <G, e^L_C S>: the pairs around the segment's last chunk
      const float *G = seg + 1 < p.segments ? p.W + ((size_t)seq * (p.segments - 1) + seg) * es
                       : p.dSf ? p.dSf + (size_t)seq * es : nullptr;
      if (G) {
        StateRows<F> g;
        g.load(G, p, warp, lane);
#pragma unroll
        for (int n = 0; n < F::D / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) around = fmaf(g.c[n][e], state.c[n][e], around);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) around += __shfl_xor_sync(0xffffffffu, around, off);
      if (lane == 0) sh.sum[warp] = around * sh.decay.all.x;
    }
    __syncthreads();
    if (p.rq && threadIdx.x < F::C && t0 + (int)threadIdx.x < p.L) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < F::SPLIT; ++i) s += sh.rows[i][threadIdx.x];
      p.rq[(size_t)seq * p.L + t0 + threadIdx.x] = s;
    }
    if (c + 1 < c1) state.planes(state_tile, warp, lane);
  }
  if (p.rq && threadIdx.x == 0) {
    float s = 0.f;
    for (int i = 0; i < F::WARPS; ++i) s += sh.sum[i];
    p.around[(size_t)seq * p.segments + seg] = s;
  }
}

// dk and dv: a walk backward over a segment's chunks.
template <typename F> constexpr uint32_t grad_kv_smem() {
  return bwd_shared_bytes<F>() + 2 * (F::NI + F::NV) * F::TILE + F::NM * F::STATE +
         2 * F::SHARE * F::NO * F::SCORES;
}
template <typename F>
__global__ void __launch_bounds__(F::THREADS, F::BLOCKS) grad_kv_kernel(const ChunkBwd p) {
  extern __shared__ __align__(128) char smem[];
  auto &sh = *reinterpret_cast<BwdShared<F> *>(smem);
  char *state_tile = smem + bwd_shared_bytes<F>();
  const uint32_t G = smem_u32(state_tile), tiles = G + F::NM * F::STATE;
  constexpr uint32_t X = F::NI * F::TILE, Y = F::NV * F::TILE;
  char *scores = state_tile + F::NM * F::STATE + 2 * (X + Y);
  constexpr int NT = F::COLS / 8, CT = F::C / 8;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int group = warp % F::ROWS, part = warp / F::ROWS;
  const int r0 = group * 16, n0 = part * F::COLS;
  const int seq = blockIdx.x / p.segments, seg = blockIdx.x % p.segments;
  const int c0 = seg * p.per, c1 = min(c0 + p.per, p.chunks);
  const size_t ek = (size_t)seq * p.L * p.n_k, ev = (size_t)seq * p.L * p.n_v;
  const size_t es = (size_t)p.n_k * p.n_v;
  using T = typename F::T;
  const T *k = static_cast<const T *>(p.k) + ek, *v = static_cast<const T *>(p.v) + ev;
  const T *q = static_cast<const T *>(p.q) + ek, *dO = static_cast<const T *>(p.dO) + ev;
  auto load = [&](int t) {
    TileRows<F> a, b, c, d;
    a.fetch(q, p, p.n_k, t), b.fetch(k, p, p.n_k, t);
    c.fetch(v, p, p.n_v, t), d.fetch(dO, p, p.n_v, t);
    a.template put<true>(tiles, p, p.n_k, t);
    // of phi(k), for dv alone, its rounding averages out
    b.template put<true, F::NO>(tiles + X, p, p.n_k, t);
    c.template put<false>(tiles + 2 * X, p, p.n_v, t);
    d.template put<false>(tiles + 2 * X + Y, p, p.n_v, t);
  };
  StateRows<F> state;
  state.load(seg + 1 < p.segments ? p.W + ((size_t)seq * (p.segments - 1) + seg) * es
             : p.dSf ? p.dSf + (size_t)seq * es : nullptr, p, warp, lane);
  state.planes(state_tile, warp, lane);
  for (int c = c1 - 1; c >= c0; --c) {
    const int t0 = c * F::C;
    const uint32_t tq = tiles;
    const uint32_t tk = tq + X, tv = tk + X, td = tv + Y;
    const bool keep = F::NI == 3 && p.keeps(seq, c, c1);
    load(t0);
    chunk_decay<F::C>(p, seq, c, sh.decay);
    __syncthreads();
    if (keep) {
      float s = dot_kept<F>(p.kept + p.keep_slot(seq, c) * es, state_tile, p);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      float *to = p.between + p.keep_slot(seq, c) * kShares;
      if (lane == 0)
        for (int i = warp; i < kShares; i += F::WARPS) to[i] = i == warp ? s * sh.decay.all.x : 0.f;
    }
    // K Q^T . D and V dO^T . D: rows i of the group, tokens j >= i
    float w[CT][4] = {}, dw[CT][4] = {};
    auto live = [&](int j) { return j >= group; };
    // Four scores of both, masked and decayed, and their pairs.
    auto masked = [&](float (&x)[4], float (&y)[4], int col, float (&pair)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = r0 + lane / 4 + e / 2 * 8, j = col + lane % 4 * 2 + e % 2;
        float f = 1.f;
        if (p.decay_kind != LA_DECAY_NONE)
          f = decay_between(sh.decay.lam[j], sh.decay.lam[i <= j ? i : j]);
        pair[e] = i < j ? x[e] * y[e] * f : 0.f;
        x[e] = i <= j ? x[e] * f : 0.f;
        y[e] = i <= j ? y[e] * f : 0.f;
      }
    };
    // The pairs i < t <= j for the tokens t of eight columns: j in them or, by `behind`, the sum of
    // a row's pairs with the columns behind them.  A row's sum from each column on, which joins
    // `behind`, then for each column the sum over the rows before it.
    auto put_crossing = [&](const float (&pair)[4], int col, float (&behind)[2]) {
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = lane % 4, i = r0 + lane / 4 + 8 * h, t = col + at * 2;
        float from = pair[2 * h] + pair[2 * h + 1];  // on to the sum of this lane's and those behind
        float x = __shfl_down_sync(0xffffffffu, from, 1, 4);
        from += at < 3 ? x : 0.f;
        x = __shfl_down_sync(0xffffffffu, from, 2, 4);
        from += at < 2 ? x : 0.f;
        x = __shfl_down_sync(0xffffffffu, from, 1, 4);
        const float last = pair[2 * h + 1] + ((at < 3 ? x : 0.f) + behind[h]);
        sum[0] += i < t ? pair[2 * h] + last : 0.f;
        sum[1] += i < t + 1 ? last : 0.f;
        behind[h] += __shfl_sync(0xffffffffu, from, 0, 4);
      }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], off);
        sum[1] += __shfl_xor_sync(0xffffffffu, sum[1], off);
      }
      if (lane < 4) {
        sh.cols[group][col + lane * 2] = sum[0];
        sh.cols[group][col + lane * 2 + 1] = sum[1];
      }
    };
    float behind[2] = {0.f, 0.f};
    if constexpr (F::SHARE) {
      float pair[4] = {};
      if (live(part / 2)) {
        float x[4] = {}, y[4] = {};
        score_tile<F, F::NI, F::NI>(x, tk, r0, tq, part * 8, lane);
        score_tile<F, F::NV, F::NV>(y, tv, r0, td, part * 8, lane);
        masked(x, y, part * 8, pair);
        put_scores<F>(scores, x, r0, part * 8, lane);
        put_scores<F>(scores + F::NO * F::SCORES, y, r0, part * 8, lane);
      }
      if (p.rc) {
        put_crossing(pair, part * 8, behind);
#pragma unroll
        for (int h = 0; h < 2; ++h)  // a row's pairs with the warp's columns, for those before them
          if (lane % 4 == 0) sh.pairs[part][r0 + lane / 4 + 8 * h] = behind[h];
      }
    } else {
      rows_times_rows<F, CT, F::NO, F::NO>(w, tk, F::TILE, r0, tq, F::TILE, 0, lane, live);
      rows_times_rows<F, CT, F::NV, F::NV>(dw, tv, F::TILE, r0, td, F::TILE, 0, lane, live);
      constexpr int OWN = CT / F::SPLIT;  // columns (by 8) whose tokens a warp of the group adds up
      float later[2] = {0.f, 0.f};
#pragma unroll
      for (int n = CT - 1; n >= 0; --n) {
        float pair[4] = {};
        if (n / 2 >= group) masked(w[n], dw[n], n * 8, pair);
        if (!p.rc || n / OWN < part) continue;
        if (n / OWN > part) {
          later[0] += pair[0] + pair[1], later[1] += pair[2] + pair[3];
          continue;
        }
        if (n % OWN == OWN - 1) behind[0] = group_sum<4>(later[0]), behind[1] = group_sum<4>(later[1]);
        put_crossing(pair, n * 8, behind);
      }
    }
    auto frag = [&](uint32_t (&a)[F::NO][4], int j) {
      if constexpr (F::SHARE) score_frag<F>(a, smem_u32(scores), r0, j, lane);
      else score_frag<F>(a, w, j);
    };
    auto dfrag = [&](uint32_t (&a)[F::NO][4], int j) {
      if constexpr (F::SHARE) score_frag<F>(a, smem_u32(scores) + F::NO * F::SCORES, r0, j, lane);
      else score_frag<F>(a, dw, j);
    };
    const float t_0 = sh.decay.tail[r0 + lane / 4], t_1 = sh.decay.tail[r0 + lane / 4 + 8];
    {
      float acc[NT][4] = {};
      rows_times_cols<F, NT, F::NO, F::NO>(acc, tk, F::TILE, r0, G, F::STATE, n0, lane);
#pragma unroll
      for (int n = 0; n < NT; ++n)
        acc[n][0] *= t_0, acc[n][1] *= t_0, acc[n][2] *= t_1, acc[n][3] *= t_1;
      if (F::SHARE) __syncthreads();
      scores_times_cols<F, NT, F::NV>(acc, frag, td, n0, lane, live);
      store_rows<F, NT>(acc, static_cast<T *>(p.dv) + ev, nullptr, p, p.n_v, t0 + r0, n0, lane);
    }
    {
      float acc[NT][4] = {};
      rows_times_rows<F, NT, F::NV, F::NM>(acc, tv, F::TILE, r0, G, F::STATE, n0, lane,
                                           [](int) { return true; });
#pragma unroll
      for (int n = 0; n < NT; ++n)
        acc[n][0] *= t_0, acc[n][1] *= t_0, acc[n][2] *= t_1, acc[n][3] *= t_1;
      if (p.rk) {
        const float2 d = row_dots<F, NT>(acc, k, p, p.n_k, t0 + r0, n0, lane);
        if (lane % 4 == 0) {
          sh.rows[part][r0 + lane / 4] = d.x;
          sh.rows[part][r0 + lane / 4 + 8] = d.y;
        }
      }
      scores_times_cols<F, NT, F::NI>(acc, dfrag, tq, n0, lane, live);
      store_rows<F, NT>(acc, static_cast<T *>(p.dk) + ek, k, p, p.n_k, t0 + r0, n0, lane);
    }
    const bool more = c > c0;
    if (more || (p.dS0 && seg == 0)) state.update(tq, td, sh.decay.head, sh.decay.all, warp, lane);
    __syncthreads();
    if (p.rk) {
      const int t = threadIdx.x;
      float others = 0.f;  // pairs of the rows before t with the columns of the warps behind t's
      if constexpr (F::SHARE) {
        static_assert(F::C == 32, "a warp holds a row of each");
        if (warp == 0) {
#pragma unroll
          for (int i = 1; i < F::SPLIT; ++i) {
            const float before = lanes_sum<true, 32>(sh.pairs[i][lane], lane);
            if (i > lane / 8) others += before;
          }
        }
      }
      if (t < F::C && t0 + t < p.L) {
        float s = 0.f, cols = 0.f;
#pragma unroll
        for (int i = 0; i < F::SPLIT; ++i) s += sh.rows[i][t];
#pragma unroll
        for (int i = 0; i < F::ROWS; ++i) cols += sh.cols[i][t];
        p.rk[(size_t)seq * p.L + t0 + t] = s;
        p.rc[(size_t)seq * p.L + t0 + t] = cols + others;
      }
    }
    if (more) state.planes(state_tile, warp, lane);
  }
  if (p.dS0 && seg == 0) state.store(p.dS0 + (size_t)seq * es, p, warp, lane);
}

cudaError_t launch_segment_scan(const ChunkBwd &p, int seqs, cudaStream_t stream);

// The launches of one configuration.
template <typename F> cudaError_t run_chunk_bwd(const ChunkBwd &p, int seqs, cudaStream_t stream) {
  [[maybe_unused]] static int set_share[64];
  static int set_q[64], set_kv[64];
  cudaError_t e;
  if constexpr (F::NI == 3) {  // else there is one chunk
    if (p.segments > 1) {
      auto share = segment_share_kernel<F>;
      if ((e = tc::set_smem_once(share, share_smem<F>(), set_share)) != cudaSuccess) return e;
      share<<<dim3((unsigned)(seqs * (p.segments - 1)), 2), F::THREADS, share_smem<F>(), stream>>>(p);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
      if ((e = launch_segment_scan(p, seqs, stream)) != cudaSuccess) return e;
    }
  }
  auto gq = grad_q_kernel<F>;
  auto gkv = grad_kv_kernel<F>;
  if ((e = tc::set_smem_once(gq, grad_q_smem<F>(), set_q)) != cudaSuccess) return e;
  if ((e = tc::set_smem_once(gkv, grad_kv_smem<F>(), set_kv)) != cudaSuccess) return e;
  gq<<<seqs * p.segments, F::THREADS, grad_q_smem<F>(), stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  gkv<<<seqs * p.segments, F::THREADS, grad_kv_smem<F>(), stream>>>(p);
  return cudaGetLastError();
}

}  // namespace la
