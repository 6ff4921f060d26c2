// la_selective_scan.cu -- selective state space scan.
//
//     delta = softplus(dt + bias);  h_n = exp(delta A_n) h_n + (delta x) B_n
//     y = (sum_n C_n h_n + skip x) silu(z)
//
// for every channel and token, N states per channel.  The decay differs per
// (channel, state) pair, so no matrix product carries the recurrence: per
// state and token it takes one exp and four multiply-adds' worth of fp32 work.
//
// A block holds CH channels of one sequence and walks it in tiles of T tokens.
// Four staging warps turn a tile's inputs into delta and delta x, once per
// (token, channel), and into fp32 B and C, in shared memory; four recurrence
// warps run the states over the tile, each lane holding P states of NC
// channels in registers, S lanes to a channel; the staging warps sum the
// lanes' parts of y, apply skip and gate, and store.  The tiles are double
// buffered, so the recurrence of one tile runs beside the staging of the next
// and the output of the one before.
//
// A sequence too long for the channels there are to fill the GPU runs as
// segments: a first launch gives every segment's own end state (and all of the
// first segment's output), a second the other segments' outputs, each starting
// from the states of the segments before it, decayed by exp(A sum delta).
//
// What bounds it: per 4 states of 32 lanes and token, 16 cycles of the
// special-function unit for the exps (32 lanes a clock on an SM) and 16 of the
// fp32 pipe (128 lanes a clock; 22 as three-operand packed instructions issue).
// Both floors are 57 us for 4 x 2048 x 4096 (N = 16, bf16; its bytes take 40): it
// runs 185 us, and 1 x 16384 x 2048 280 us.  The counters show no unit full
// (issue slots and shared-memory wavefronts about 70% on an SM with two
// blocks): the recurrence warps' own instruction stream sets the pace, and taking
// out staging work (softplus, gate, address arithmetic) does not change the time.
// A block has 64 channels, so 256 blocks leave 48 of the 152 SMs with one
// instead of two (14%).  Measured on the first case: lanes with 4 states of two
// channels 198 us, of one 260, with 8 of two 202; blocks of 2 + 2 warps 195; one
// role for all threads (no staging warps) 262; a token's loads not ahead of the
// token before 213.
#include <cstdint>

#include "../../include/la_gb300.h"
#include "la_act.cuh"
#include "la_internal.h"

namespace la {
namespace {

constexpr int kStage = 128;           // staging threads
constexpr int kMain = 128;            // recurrence threads
constexpr int kThreads = kStage + kMain;
constexpr int kRing = 5;              // tiles of inputs in shared memory: the one whose output is
                                      // due, the one being staged, and three on their way

template <int I> struct Int { static constexpr int value = I; };

// Block barriers between the staging and the recurrence warps: one side
// arrives, the other waits.
__device__ __forceinline__ void bar_arrive(int id) {
  asm volatile("barrier.cta.arrive %0, %1;" ::"r"(id), "n"(kThreads) : "memory");
}
__device__ __forceinline__ void bar_wait(int id) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "n"(kThreads) : "memory");
}

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
  // Segments: nseg of seg_len tokens; states [nseg - 1][B][D][N] and sums of
  // delta [nseg - 1][B][D] in the workspace.
  int B, nseg, seg_len;
  float *seg_state, *seg_sum;
};

// softplus of two values: log(1 + e^v) = max(v, 0) + e p(e), e = e^-|v| in (0,
// 1].  e's exponent is taken in two parts, -|v| log2 e = hi + lo, where a fused
// multiply-add gives the rounding error of the product hi exactly, so that it
// does not reach e.  p(e) = log1p(e) / e is the polynomial of degree 9 through
// the ten Chebyshev nodes of [0, 1]; with the constant 1 and the other
// coefficients in fp32 it errs by 1.43e-8 before rounding, relative (as computed
// in 64 bits), so steps near e^-7 keep the precision that log(1 + e) would lose.
// (2 atanh(e / (2 + e)) by its series took a reciprocal more.)
// |v| counts as 128 beyond it: e is 0 there in fp32, and hi stays finite for
// infinities and for the lowest values that a mask writes.
__device__ __forceinline__ void softplus2(float &v0, float &v1) {
  const unsigned long long v = pack2(max_nan(-fabsf(v0), -128.f), max_nan(-fabsf(v1), -128.f));
  const unsigned long long hi = mul2(v, dup2(kLog2e));
  unsigned long long lo = fma2(v, dup2(kLog2e), mul2(hi, dup2(-1.f)));
  lo = fma2(v, dup2(1.925963033500e-8f), lo);  // log2 e - float(log2 e)
  float h0, h1;
  unpack2(hi, h0, h1);
  unsigned long long e = pack2(ex2_approx(h0), ex2_approx(h1));
  e = fma2(e, mul2(lo, dup2(0.6931471805599453f)), e);  // 2^lo = 1 + lo ln 2
  unsigned long long p = fma2(e, dup2(-0.0031760570127516985f), dup2(0.019542526453733444f));
  p = fma2(e, p, dup2(-0.056373611092567444f));
  p = fma2(e, p, dup2(0.10543623566627502f));
  p = fma2(e, p, dup2(-0.1526966691017151f));
  p = fma2(e, p, dup2(0.1966327428817749f));
  p = fma2(e, p, dup2(-0.24951615929603577f));
  p = fma2(e, p, dup2(0.33329710364341736f));
  p = fma2(e, p, dup2(-0.49999892711639404f));
  p = fma2(e, p, dup2(1.f));
  unpack2(fma2(e, p, pack2(fmaxf(v0, 0.f), fmaxf(v1, 0.f))), v0, v1);
}

__device__ __forceinline__ uint32_t bits(float v) { return __float_as_uint(v); }
__device__ __forceinline__ uint32_t bits(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }

constexpr int min_c(int a, int b) { return a < b ? a : b; }

// P states of NC channels per lane, S lanes per channel, elements of E bytes.
template <int P, int S, int NC, int E>
struct ScanShape {
  static constexpr int NP = P * S;                              // states, padded
  static constexpr int LC = 32 / S;                             // lanes side by side in channels
  static constexpr int WCH = LC * NC;                           // channels per warp
  static constexpr int CH = kMain / 32 * WCH;                   // channels per block
  static constexpr int T = min_c(CH * E >= 256 ? 8 : 16, 1024 / NP);  // tokens per tile
  static constexpr int Q = min_c(S, 4);                         // parts of y per (token, channel)
  static constexpr int V = 16 / E;                              // channels a thread stages at once
  static constexpr int K = CH / V;                              // such chunks per token
  static constexpr int XR = (T * K + kStage - 1) / kStage;      // chunks per thread
  static constexpr int BV = min_c(16 / E, NP);                  // states of B or C staged at once
  static constexpr int BK = NP / BV;
  static constexpr int BR = (2 * T * BK + kStage - 1) / kStage;
  // The parts of a warp's channels lie together, [Q][WCH]; its row is padded so
  // that the staging threads, V channels each, read them from different banks.
  static constexpr int GROUP = Q * WCH + 4;
  static constexpr int SLOT_BYTES = T * CH * 8;
  static constexpr int BC_BYTES = 2 * T * NP * 4;
  static constexpr int PART_BYTES = T * (kMain / 32) * GROUP * 4;
  // The inputs as fetched: a ring of kRing tiles, in which every staging thread
  // has places of its own (x, dt and z chunks, then its B and C chunks).
  static constexpr int RAW_X = XR * kStage * 16;
  static constexpr int RAW_BYTES = 3 * RAW_X + BR * kStage * 16;
  static constexpr int SMEM = 2 * (SLOT_BYTES + BC_BYTES + PART_BYTES) + kRing * RAW_BYTES;
  static_assert(WCH % 4 == 0 && CH % V == 0 && kStage % K == 0 && NP % 4 == 0, "tile shape");
  static_assert(SMEM <= 113 * 1024, "two blocks per SM");
};

// N elements of T as they lie in memory, in 32-bit words.
template <typename T, int N> struct alignas(sizeof(T) * N) Chunk {
  uint32_t w[N * sizeof(T) / 4];
  __device__ __forceinline__ float get(int i) const {  // i known at compile time
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  __device__ __forceinline__ void set2(int i, float lo, float hi) {  // elements i, i + 1
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(lo), w[i + 1] = __float_as_uint(hi);
    } else {
      const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
      w[i / 2] = *reinterpret_cast<const uint32_t *>(&v);
    }
  }
};

// How the rows of the inputs are aligned: to 16 bytes, to 4 bytes, or to an element.
enum : int { ALIGN16 = 16, ALIGN4 = 4, ALIGN_ELT = 1 };

// Bring `count` of N elements of T into this thread's 16-byte (or smaller)
// place in shared memory; the rest of it becomes 0.  Asynchronous where the
// alignment allows it.
template <typename T, int N, int ALIGN>
__device__ __forceinline__ void fetch_chunk(void *dst, const T *src, int count) {
  constexpr int BYTES = N * sizeof(T);
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (ALIGN == ALIGN16 && BYTES == 16) {
    const int bytes = count * (int)sizeof(T);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes)
                 : "memory");
  } else if constexpr (ALIGN >= 4) {
#pragma unroll
    for (int i = 0; i < BYTES / 4; ++i) {
      const int bytes = min(max(count * (int)sizeof(T) - 4 * i, 0), 4);
      const T *from = src + (bytes > 0 ? i * 4 / (int)sizeof(T) : 0);
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d + 4 * i), "l"(from),
                   "r"(bytes)
                   : "memory");
    }
  } else {
    T *out = static_cast<T *>(dst);
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = i < count ? src[i] : from_f32<T>(0.f);
  }
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING> __device__ __forceinline__ void fetch_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// Where the 16 bytes (delta and delta x of channels 2g, 2g + 1) of granule g
// lie in a token's row: the 8 staging threads of a quarter warp, four granules
// apart, write to different banks, and neighbouring lanes read neighbours.
__device__ __forceinline__ int slot_granule(int g) { return g ^ (g >> 3 & 3); }

// The state behind a segment that starts in h: exp2(a sum) h + end, end being the
// segment's end state from zero.  Where a state grows (a sum > 0) the factor may
// pass fp32's range although its product with a small h or with 0 does not: it
// is then applied in three parts.  A state that does not decay (a = 0) stays h
// where the sum is infinite.
__device__ __forceinline__ float after_segment(float h, float a, float sum, float end) {
  const float e = a * sum;
  if (e <= 120.f) return fmaf(ex2_approx(e), h, end);
  if (a == 0.f) return h + end;
  if (h == 0.f) return end;
  const float third = ex2_approx(e * (1.f / 3.f));
  return fmaf(third, third * (third * h), end);
}

// One block's share of one segment.  FULL: outputs from the state `from` the
// segment starts in; else only its end state, from zero, and its sum of delta.
template <typename T, int P, int S, int NC, int ALIGN, bool FULL>
__device__ __forceinline__ void scan_segment(const ScanParams<T> &p, long long b, int g, int cg0,
                                             int seg, int s0, int s1, int len, char *smem) {
  using Sh = ScanShape<P, S, NC, sizeof(T)>;
  constexpr int CH = Sh::CH, NP = Sh::NP, TT = Sh::T, Q = Sh::Q, V = Sh::V, K = Sh::K;
  constexpr int BV = Sh::BV, BK = Sh::BK, WCH = Sh::WCH;
  const int per_group = p.D / p.groups;
  const int nch = min(CH, per_group - cg0);
  const int c0 = g * per_group + cg0;
  const int end = min(s1, len);  // s0 < end
  const int tiles = (end - s0 + TT - 1) / TT;
  char *slots = smem, *bcs = smem + 2 * Sh::SLOT_BYTES, *prt = bcs + 2 * Sh::BC_BYTES;
  char *raw = prt + 2 * Sh::PART_BYTES;

  if (threadIdx.x >= kMain) {
    // ------------------------------------------------------------ staging warps
    const int tid = threadIdx.x - kMain;
    const int k = tid % K;                        // the chunk of channels it stages in every tile
    const int sc = k * V;                         // its first channel in the block
    const int st = tid / K;                       // its first token in the tile
    const int have = min(max(nch - sc, 0), V);    // channels past the last are staged as zeros
    float bias[V], skip[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      bias[e] = p.dt_bias && e < have ? p.dt_bias[c0 + sc + e] : 0.f;
      skip[e] = p.skip && e < have ? p.skip[c0 + sc + e] : 0.f;
    }
    const int from_c = c0 + (have > 0 ? sc : 0);  // an address in bounds even where nothing is read
    const T *xb = p.x + b * p.L * p.x_stride + from_c;
    const T *db = p.dt + b * p.L * p.dt_stride + from_c;
    const T *zb = p.z ? p.z + b * p.L * p.z_stride + from_c : nullptr;
    T *yb = p.y + b * p.L * p.y_stride + c0 + sc;
    const T *Bb = p.Bm + b * p.L * p.b_stride + (long long)g * p.N;
    const T *Cb = p.Cm + b * p.L * p.c_stride + (long long)g * p.N;

    char *mine = raw + tid * 16;
    auto fetch = [&](int tile) {  // rows past the last token repeat it
      if (tile < tiles) {
        char *to = mine + tile % kRing * Sh::RAW_BYTES;
        const int t0 = s0 + tile * TT;
#pragma unroll
        for (int r = 0; r < Sh::XR; ++r) {
          const long long t = min(t0 + st + r * (kStage / K), end - 1);
          char *at = to + r * kStage * 16;
          fetch_chunk<T, V, ALIGN>(at, xb + t * p.x_stride, have);
          fetch_chunk<T, V, ALIGN>(at + Sh::RAW_X, db + t * p.dt_stride, have);
          if (FULL && zb) fetch_chunk<T, V, ALIGN>(at + 2 * Sh::RAW_X, zb + t * p.z_stride, have);
        }
#pragma unroll
        for (int r = 0; r < Sh::BR; ++r) {
          const int i = tid + r * kStage;
          const bool is_c = i / BK >= TT;
          if (!FULL && is_c) break;
          const int cnt = min(max(p.N - i % BK * BV, 0), BV), n = cnt > 0 ? i % BK * BV : 0;
          const long long t = min(t0 + i / BK % TT, end - 1);
          const T *src = is_c ? Cb + t * p.c_stride : Bb + t * p.b_stride;
          fetch_chunk<T, BV, ALIGN>(to + 3 * Sh::RAW_X + r * kStage * 16, src + n, cnt);
        }
      }
      fetch_commit();
    };

    auto output = [&](int tile) {
      const int t0 = s0 + tile * TT;
      const float *pt = reinterpret_cast<const float *>(prt + (tile & 1) * Sh::PART_BYTES);
#pragma unroll
      for (int r = 0; r < Sh::XR; ++r) {
        const int t = st + r * (kStage / K);
        if (t >= TT || t0 + t >= end) break;
        float v[V];
#pragma unroll
        for (int e = 0; e < V; e += 4) {
          const int c = sc + e;
          const float *s = pt + (t * (kMain / 32) + c / WCH) * Sh::GROUP + c % WCH;
          float4 f = *reinterpret_cast<const float4 *>(s);
#pragma unroll
          for (int i = 1; i < Q; ++i) {
            const float4 o = *reinterpret_cast<const float4 *>(s + i * WCH);
            f.x += o.x, f.y += o.y, f.z += o.z, f.w += o.w;
          }
          v[e] = f.x, v[e + 1] = f.y, v[e + 2] = f.z, v[e + 3] = f.w;
        }
        const char *from = mine + tile % kRing * Sh::RAW_BYTES + r * kStage * 16;
        const auto x = *reinterpret_cast<const Chunk<T, V> *>(from);
        const auto z = *reinterpret_cast<const Chunk<T, V> *>(from + 2 * Sh::RAW_X);
        Chunk<T, V> o;
#pragma unroll
        for (int e = 0; e < V; e += 2) {
#pragma unroll
          for (int f = e; f < e + 2; ++f) {
            v[f] = fmaf(skip[f], x.get(f), v[f]);
            if (zb) v[f] *= activate(LA_ACT_SILU, z.get(f));
          }
          o.set2(e, v[e], v[e + 1]);
        }
        T *yr = yb + (long long)(t0 + t) * p.y_stride;
        if (ALIGN == ALIGN16 && have == V) {
          *reinterpret_cast<uint4 *>(yr) = *reinterpret_cast<const uint4 *>(&o);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e)
            if (e < have) yr[e] = from_f32<T>(o.get(e));
        }
      }
    };

    for (int i = 0; i < kRing - 2; ++i) fetch(i);
    for (int tile = 0; tile < tiles; ++tile) {
      const int buf = tile & 1;
      fetch(tile + kRing - 2);  // into the place of the tile whose output came last
      fetch_wait<kRing - 2>();
      const char *in = mine + tile % kRing * Sh::RAW_BYTES;
      if (!FULL && tile >= 2) bar_wait(3 + buf);  // the recurrence is done with this buffer
      char *sl = slots + buf * Sh::SLOT_BYTES;
#pragma unroll
      for (int r = 0; r < Sh::XR; ++r) {
        const int t = st + r * (kStage / K);
        if (t >= TT) break;
        const auto rx = *reinterpret_cast<const Chunk<T, V> *>(in + r * kStage * 16);
        const auto rd = *reinterpret_cast<const Chunk<T, V> *>(in + Sh::RAW_X + r * kStage * 16);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          float d0 = rd.get(e) + bias[e], d1 = rd.get(e + 1) + bias[e + 1];
          if (p.softplus) softplus2(d0, d1);
          *reinterpret_cast<float4 *>(sl + t * CH * 8 + slot_granule((sc + e) / 2) * 16) =
              make_float4(d0, d0 * rx.get(e), d1, d1 * rx.get(e + 1));
        }
      }
      float4 *bc = reinterpret_cast<float4 *>(bcs + buf * Sh::BC_BYTES);
#pragma unroll
      for (int r = 0; r < Sh::BR; ++r) {
        const int i = tid + r * kStage;
        if (i >= (FULL ? 2 : 1) * TT * BK) break;
        const auto v = *reinterpret_cast<const Chunk<T, BV> *>(in + 3 * Sh::RAW_X +
                                                               r * kStage * 16);
#pragma unroll
        for (int e = 0; e < BV; e += 4)
          bc[(i * BV + e) / 4] = make_float4(v.get(e), v.get(e + 1), v.get(e + 2), v.get(e + 3));
      }
      bar_arrive(1 + buf);
      if (FULL && tile >= 1) {
        bar_wait(3 + (buf ^ 1));
        output(tile - 1);
      }
    }
    if (FULL) {
      bar_wait(3 + ((tiles - 1) & 1));
      output(tiles - 1);
    } else {  // leave no arrival behind
      if (tiles >= 2) bar_wait(3 + (tiles & 1));
      bar_wait(3 + ((tiles - 1) & 1));
    }
    return;
  }

  // -------------------------------------------------------------- recurrence warps
  // Lane (q, cl): lanes that read the same B and C are neighbours.  It holds the
  // states 4 (q + S j) + i of the channels lc + m.
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int q = lane / Sh::LC, cl = lane % Sh::LC;
  const int lc = warp * WCH + cl * NC;
  unsigned long long a[NC][P / 2], h[NC][P / 2];
#pragma unroll
  for (int m = 0; m < NC; ++m) {
    const bool on = lc + m < nch;
    const long long ch = c0 + (on ? lc + m : 0);
    const long long at = (b * p.D + ch) * p.N;
    const long long pitch = (long long)p.B * p.D * p.N;
#pragma unroll
    for (int k = 0; k < P; k += 2) {
      float av[2], hv[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int n = 4 * (q + S * (k / 4)) + k % 4 + e;
        const bool in = on && n < p.N;
        av[e] = in ? p.A[ch * p.N + n] * kLog2e : 0.f;
        hv[e] = 0.f;
        if (FULL && in) {
          if (seg == 0) {
            if (p.h0) hv[e] = p.h0[at + n];
          } else {
            hv[e] = p.seg_state[at + n];
            for (int i = 1; i < seg; ++i)
              hv[e] = after_segment(hv[e], av[e],
                                    p.seg_sum[((long long)i * p.B + b) * p.D + ch],
                                    p.seg_state[i * pitch + at + n]);
          }
        }
      }
      a[m][k / 2] = pack2(av[0], av[1]);
      h[m][k / 2] = pack2(hv[0], hv[1]);
    }
  }
  float sum[NC];
#pragma unroll
  for (int m = 0; m < NC; ++m) sum[m] = 0.f;

  for (int tile = 0; tile < tiles; ++tile) {
    const int buf = tile & 1;
    const char *sl = slots + buf * Sh::SLOT_BYTES;
    const float4 *bc = reinterpret_cast<const float4 *>(bcs + buf * Sh::BC_BYTES);
    float *pt = reinterpret_cast<float *>(prt + buf * Sh::PART_BYTES) + warp * Sh::GROUP +
                q * WCH + cl * NC;
    float part_sum[NC];
#pragma unroll
    for (int m = 0; m < NC; ++m) part_sum[m] = 0.f;
    bar_wait(1 + buf);
    // A token passes three stages, one token apart: its loads; its decays and
    // writes, which do not wait for the state; the recurrence and the read.
    // A warp alone on its scheduler so keeps loads, exponentials and products
    // of three tokens in flight.
    struct Loaded {
      float d[NC], dx[NC];
      float4 b[P / 4], c[P / 4];
    };
    struct Ready {
      unsigned long long dec[NC][P / 2], w[NC][P / 2];
    };
    auto load = [&](Loaded &l, int t) {
      const char *row = sl + t * CH * 8;
      if constexpr (NC == 1) {
        const float2 s =
            *reinterpret_cast<const float2 *>(row + slot_granule(lc / 2) * 16 + lc % 2 * 8);
        l.d[0] = s.x, l.dx[0] = s.y;
      } else {
#pragma unroll
        for (int m = 0; m < NC; m += 2) {
          const float4 s = *reinterpret_cast<const float4 *>(row + slot_granule((lc + m) / 2) * 16);
          l.d[m] = s.x, l.dx[m] = s.y, l.d[m + 1] = s.z, l.dx[m + 1] = s.w;
        }
      }
#pragma unroll
      for (int j = 0; j < P / 4; ++j) {
        l.b[j] = bc[t * (NP / 4) + q + S * j];
        if (FULL) l.c[j] = bc[(TT + t) * (NP / 4) + q + S * j];
      }
    };
    auto prepare = [&](Ready &r, const Loaded &l) {
#pragma unroll
      for (int m = 0; m < NC; ++m) {
        const unsigned long long d2 = dup2(l.d[m]), x2 = dup2(l.dx[m]);
#pragma unroll
        for (int j = 0; j < P / 4; ++j) {
          float e0, e1, e2, e3;
          unpack2(mul2(d2, a[m][2 * j]), e0, e1);
          unpack2(mul2(d2, a[m][2 * j + 1]), e2, e3);
          r.dec[m][2 * j] = pack2(ex2_approx(e0), ex2_approx(e1));
          r.dec[m][2 * j + 1] = pack2(ex2_approx(e2), ex2_approx(e3));
          r.w[m][2 * j] = mul2(x2, pack2(l.b[j].x, l.b[j].y));
          r.w[m][2 * j + 1] = mul2(x2, pack2(l.b[j].z, l.b[j].w));
        }
        if (!FULL) part_sum[m] += l.d[m];
      }
    };
    auto advance = [&](const Ready &r, const Loaded &l, int t) {
      float part[NC];
#pragma unroll
      for (int m = 0; m < NC; ++m) {
        unsigned long long acc;
#pragma unroll
        for (int k = 0; k < P / 2; ++k) {
          h[m][k] = fma2(r.dec[m][k], h[m][k], r.w[m][k]);
          if (FULL) {
            const float4 cv = l.c[k / 2];
            const unsigned long long c2 = k % 2 ? pack2(cv.z, cv.w) : pack2(cv.x, cv.y);
            acc = k == 0 ? mul2(c2, h[m][0]) : fma2(c2, h[m][k], acc);
          }
        }
        if (FULL) {
          float lo, hi;
          unpack2(acc, lo, hi);
          part[m] = lo + hi;
#pragma unroll
          for (int off = 16; off >= Q * Sh::LC; off >>= 1)
            part[m] += __shfl_xor_sync(0xffffffffu, part[m], off);
        }
      }
      if (FULL && q < Q) {
        float *o = pt + t * (kMain / 32) * Sh::GROUP;
        if constexpr (NC == 1) o[0] = part[0];
        else if constexpr (NC == 2) *reinterpret_cast<float2 *>(o) = make_float2(part[0], part[1]);
        else *reinterpret_cast<float4 *>(o) = make_float4(part[0], part[1], part[2], part[3]);
      }
    };
    const int tend = min(TT, end - s0 - tile * TT);
    Loaded l[3];
    Ready r[2];
    if (P * NC <= 16 && tend == TT) {  // more states than that leave no registers for it
      load(l[0], 0);
      if (TT > 1) load(l[1], 1);
      prepare(r[0], l[0]);
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        if (t + 2 < TT) load(l[(t + 2) % 3], t + 2);
        if (t + 1 < TT) prepare(r[(t + 1) % 2], l[(t + 1) % 3]);
        advance(r[t % 2], l[t % 3], t);
      }
    } else {
#pragma unroll 1
      for (int t = 0; t < tend; ++t) {
        load(l[0], t);
        prepare(r[0], l[0]);
        advance(r[0], l[0], t);
      }
    }
    bar_arrive(3 + buf);
#pragma unroll
    for (int m = 0; m < NC; ++m) sum[m] += part_sum[m];
  }

  // The state after the last token, or what later segments start from (a
  // segment that pass 1 outputs has left its own in pass 0).
  float *dst = s1 >= len ? p.h_final : nullptr;
  if (s1 < len && (!FULL || seg == 0))
    dst = p.seg_state + (long long)seg * p.B * p.D * p.N;
#pragma unroll
  for (int m = 0; m < NC; ++m) {
    if (lc + m >= nch) continue;
    const long long ch = c0 + lc + m, at = (b * p.D + ch) * p.N;
    if (!FULL && q == 0) p.seg_sum[((long long)seg * p.B + b) * p.D + ch] = sum[m];
    if (!dst) continue;
#pragma unroll
    for (int k = 0; k < P; k += 2) {
      const int n = 4 * (q + S * (k / 4)) + k % 4;
      float lo, hi;
      unpack2(h[m][k / 2], lo, hi);
      if (n < p.N) dst[at + n] = lo;
      if (n + 1 < p.N) dst[at + n + 1] = hi;
    }
  }
}

// Pass 0: segments 0 .. max(nseg - 2, 0), the first in full, the others for
// their end states.  Pass 1: the outputs of segments 1 .. nseg - 1.
template <typename T, int P, int S, int NC, int ALIGN>
__global__ void __launch_bounds__(kThreads, 2)
selective_scan_kernel(const ScanParams<T> p, int pass) {
  extern __shared__ __align__(16) char smem[];
  constexpr int CH = ScanShape<P, S, NC, sizeof(T)>::CH;
  const int per_group = p.D / p.groups;
  const int blocks_g = (per_group + CH - 1) / CH;
  const int blk = blockIdx.x % (blocks_g * p.groups);
  const long long b = blockIdx.x / (blocks_g * p.groups);
  const int g = blk / blocks_g;
  const int cg0 = blk % blocks_g * CH;  // the block's first channel within its group
  const int seg = blockIdx.y + pass;
  const int len = p.lengths ? min(max(p.lengths[b], 0), p.L) : p.L;
  const int s0 = seg * p.seg_len;
  const int s1 = seg == p.nseg - 1 ? p.L : s0 + p.seg_len;
  if (seg == 0 && len == 0) {  // no tokens: the state passes through
    const long long at = (b * p.D + g * per_group + cg0) * p.N;
    const int n = min(CH, per_group - cg0) * p.N;
    if (p.h_final && p.h_final != p.h0)
      for (int i = threadIdx.x; i < n; i += kThreads)
        p.h_final[at + i] = p.h0 ? p.h0[at + i] : 0.f;
    return;
  }
  if (s0 >= len) return;
  if (seg == 0 || pass == 1)
    scan_segment<T, P, S, NC, ALIGN, true>(p, b, g, cg0, seg, s0, s1, len, smem);
  else if (s1 < len)  // a segment after this one needs its state
    scan_segment<T, P, S, NC, ALIGN, false>(p, b, g, cg0, seg, s0, s1, len, smem);
}

// A few tokens (a decode step): the states are read and written once, and that
// is the cost.  S neighbouring lanes share a channel, four or eight states each
// in one or two 16-byte vectors, so a warp reads 512 consecutive bytes of state.
// A thread takes R <= S sequences, whose loads are all in flight at once and
// which share its A; the scalars of sequence r (delta, delta x, and the output)
// are worked out by the channel's lane r and passed on by shuffles.  256
// sequences of 4096 x 16 states, one token: bf16 32 us, 4.5 TB/s, fp32 37; with
// one sequence a thread 47 and 53; when it took 33, with four blocks per SM
// instead of five 38, two sequences a thread 42, packed fp32 pairs 42.  Latency
// bounds it: the loads of a thread's sequences leave together and wait in
// registers, which limits the threads (48 registers with 48 to 60 bytes spilled
// in bf16's aligned form of one token, 64 with 56 to 72 in fp32's; 64 with 16
// and 144 for more tokens, whose loads all wait for the token before).
template <typename T, int P, int S, int R, bool VEC, bool ONE>
__global__ void __launch_bounds__(256, ONE && sizeof(T) == 2 && P == 4 ? 5 : 4)
selective_step_kernel(const ScanParams<T> p, unsigned blocks) {  // blocks: per row of sequences
  static_assert(R == 1 || R == 2 || R == 4, "halvings");
  // Channel and lane apart: D S places would pass 32 bits.
  const unsigned row = blockIdx.x / blocks;
  const unsigned place = (blockIdx.x - row * blocks) * (256 / S) + threadIdx.x / S;
  const int q = threadIdx.x % S;
  const bool live = place < (unsigned)p.D;
  const int c = live ? place : 0;
  const int g = p.groups == 1 ? 0 : c / (p.D / p.groups);
  const int b0 = row * R;
  const int mine = min(b0 + q % R, p.B - 1);  // the sequence whose scalars this lane works out
  const bool real = b0 + q % R < p.B;
  // This lane's states are 4 (q + S j) + i: the vector j lies 4 S j values on.
  auto inside = [&](int j) { return 4 * (q + S * j) < p.N; };
  const long long per_seq = (long long)p.D * p.N, at0 = b0 * per_seq + (long long)c * p.N + 4 * q;

  auto load_states = [&](float *f, const float *src) {
#pragma unroll
    for (int j = 0; j < P / 4; ++j) {
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if constexpr (VEC) {
        if (inside(j)) load_raw<float, 4>(src + 4 * S * j).unpack(v);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (4 * (q + S * j) + e < p.N) v[e] = src[4 * S * j + e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) f[4 * j + e] = v[e];
    }
  };
  auto load_row = [&](Raw<T, 4> *f, const T *src) {  // the same of T
#pragma unroll
    for (int j = 0; j < P / 4; ++j) {
      f[j] = Raw<T, 4>{};
      if constexpr (VEC) {
        if (inside(j)) f[j] = load_raw<T, 4>(src + 4 * S * j);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (4 * (q + S * j) + e < p.N)
            f[j].w[e * sizeof(T) / 4] |= bits(src[4 * S * j + e]) << (e * sizeof(T) % 4 * 8);
      }
    }
  };
  float a[P], h[R][P];
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int k = 0; k < P; ++k) h[r][k] = 0.f;
    if (p.h0 && b0 + r < p.B) load_states(h[r], p.h0 + at0 + r * per_seq);
  }
  load_states(a, p.A + (long long)c * p.N + 4 * q);
#pragma unroll
  for (int k = 0; k < P; ++k) a[k] *= kLog2e;
  const float bias = p.dt_bias ? p.dt_bias[c] : 0.f;
  const float skip = p.skip ? p.skip[c] : 0.f;
  const int len = !real ? 0 : p.lengths ? min(max(p.lengths[mine], 0), p.L) : p.L;
  const long long tok = (long long)mine * p.L;
  const T *xp = p.x + tok * p.x_stride + c, *dp = p.dt + tok * p.dt_stride + c;
  const T *zp = p.z ? p.z + tok * p.z_stride + c : nullptr;
  T *yp = p.y + tok * p.y_stride + c;
  const long long tok0 = (long long)b0 * p.L, bstep = p.L * p.b_stride, cstep = p.L * p.c_stride;
  const T *bp = p.Bm + tok0 * p.b_stride + (long long)g * p.N + 4 * q;
  const T *cp = p.Cm + tok0 * p.c_stride + (long long)g * p.N + 4 * q;
  for (int t = 0; t < (ONE ? 1 : p.L); ++t) {
    const bool on = t < len;
    float x = 0.f, d = 0.f, z = 0.f;
    if (on) {
      x = to_f32(*xp);
      d = to_f32(*dp) + bias;
      if (zp) z = to_f32(*zp);
    }
    Raw<T, 4> bn[R][P / 4], cn[R][P / 4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      // Rows behind a sequence's end are not read.
      if (R == 1 ? on : __shfl_sync(0xffffffffu, (int)on, r, S)) {
        load_row(bn[r], bp + r * bstep);
        load_row(cn[r], cp + r * cstep);
      } else {
#pragma unroll
        for (int j = 0; j < P / 4; ++j) bn[r][j] = cn[r][j] = Raw<T, 4>{};
      }
    }
    float unused = 0.f;
    if (p.softplus) softplus2(d, unused);
    if (!on) d = 0.f;  // a step of zero keeps the state
    const float u = d * x;
    float y[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float dr = R == 1 ? d : __shfl_sync(0xffffffffu, d, r, S);
      const float ur = R == 1 ? u : __shfl_sync(0xffffffffu, u, r, S);
      y[r] = 0.f;
#pragma unroll
      for (int j = 0; j < P / 4; ++j) {
        float bf[4], cf[4];
        bn[r][j].unpack(bf);
        cn[r][j].unpack(cf);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = 4 * j + e;
          h[r][k] = fmaf(ex2_approx(dr * a[k]), h[r][k], ur * bf[e]);
          y[r] = fmaf(cf[e], h[r][k], y[r]);
        }
      }
    }
    // Sum over the S lanes; lane r ends with sequence r's.
#pragma unroll
    for (int off = S / 2; off >= R && off > 0; off >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) y[r] += __shfl_xor_sync(0xffffffffu, y[r], off);
#pragma unroll
    for (int off = R / 2; off > 0; off >>= 1)
#pragma unroll
      for (int r = 0; r < off; ++r) {
        const float keep = q & off ? y[r + off] : y[r], send = q & off ? y[r] : y[r + off];
        y[r] = keep + __shfl_xor_sync(0xffffffffu, send, off);
      }
    if (on && live && q < R) {
      float o = fmaf(skip, x, y[0]);
      if (zp) o *= activate(LA_ACT_SILU, z);
      *yp = from_f32<T>(o);
    }
    if (ONE) break;
    xp += p.x_stride, dp += p.dt_stride, yp += p.y_stride;
    if (zp) zp += p.z_stride;
    bp += p.b_stride, cp += p.c_stride;
  }
  if (!p.h_final || !live) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (b0 + r >= p.B) break;
    float *dst = p.h_final + at0 + r * per_seq;
#pragma unroll
    for (int j = 0; j < P / 4; ++j) {
      const float *v = h[r] + 4 * j;
      if constexpr (VEC) {
        if (inside(j)) store_vec<float, 4>(dst + 4 * S * j, v);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (4 * (q + S * j) + e < p.N) dst[4 * S * j + e] = v[e];
      }
    }
  }
}

template <typename T, int P, int S>
cudaError_t launch_step(const ScanParams<T> &p, cudaStream_t stream) {
  constexpr int R = P > 4 ? 1 : min_c(S, 4);  // more states leave no registers for more
  auto fits = [](const void *q) {
    return (reinterpret_cast<uintptr_t>(q) & (4 * sizeof(T) - 1)) == 0;
  };
  const bool vec = p.N % 4 == 0 && p.b_stride % 4 == 0 && p.c_stride % 4 == 0 && fits(p.Bm) &&
                   fits(p.Cm);
  const long long blocks = ((long long)p.D * S + 255) / 256;
  // R sequences a thread once there are enough threads without them, against one
  // (bf16, one token, us): 38 x 4096 x 16 states 7.0 and 9.0, 64 x 4096 x 16 11.1
  // and 13.8, 16 x 4096 x 128 19.4 and 24.7.
  const bool many = (double)p.B / R * p.D * S >= 152 * 1024;
  const long long rows = many ? (p.B + R - 1ll) / R : p.B;
  if (blocks * rows > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  auto pick = [&](auto one) {
    constexpr bool ONE = decltype(one)::value;
    return many ? (vec ? selective_step_kernel<T, P, S, R, true, ONE>
                       : selective_step_kernel<T, P, S, R, false, ONE>)
                : (vec ? selective_step_kernel<T, P, S, 1, true, ONE>
                       : selective_step_kernel<T, P, S, 1, false, ONE>);
  };
  auto *kernel = p.L == 1 ? pick(Int<1>{}) : pick(Int<0>{});
  kernel<<<(unsigned)(blocks * rows), 256, 0, stream>>>(p, (unsigned)blocks);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_steps(const ScanParams<T> &p, cudaStream_t stream) {
  if (p.N <= 4) return launch_step<T, 4, 1>(p, stream);
  if (p.N <= 8) return launch_step<T, 4, 2>(p, stream);
  if (p.N <= 16) return launch_step<T, 4, 4>(p, stream);
  if (p.N <= 32) return launch_step<T, 4, 8>(p, stream);
  if (p.N <= 64) return launch_step<T, 4, 16>(p, stream);
  if (p.N <= 128) return launch_step<T, 4, 32>(p, stream);
  return launch_step<T, 8, 32>(p, stream);
}

// Channels per block, by the number of states.
constexpr int block_channels(int N) { return N <= 4 ? 128 : N <= 16 ? 64 : N <= 32 ? 32 : 16; }

// Up to this many tokens the step kernel runs.  It and the tiled kernel, us:
//                                L = 2      4          8          16
//   64 x L x 4096, N 16, bf16    15, 40     22, 41     37, 45     67, 49
//                        fp32    17, 36     26, 39     43, 41     77, 50
//   16 x L x 4096, N 16, bf16    7.4, 13    11, 13     18, 14     31, 15
//    1 x L x 4096, N 16, bf16    2.2, 3.1   3.0, 3.1   4.5, 3.4   7.8, 4.0
//   64 x L x 4096, N 128, bf16   84, 241    133, 254   236, 270   443, 328
//                        fp32    104, 235   164, 250   288, 267   541, 322
// The crossing lies between 4 and 16 tokens; one limit serves all sizes.
constexpr int kStepTokens = 8;

struct ScanPlan {
  int nseg, seg_len;
};

// How many segments.  One block on an SM takes a token in about 50 ns, two in
// 90 (N = 16, bf16: 1 x 16384 x 2048 in one piece 878 us, 4 x 2048 x 4096 185
// us), and the SMs hold two, so n blocks take rounds(n) ns per token of theirs.  One
// piece costs that over L tokens; nseg > 1 segments cost it twice, for nseg - 1
// segments side by side, over L / nseg tokens, and a launch.  1 x 16384 x 2048
// (32 blocks): 444 us in 4, 277 in 10 (the first that fills both blocks of all
// SMs), 325 in 12 (a round and a bit), 292 in 20.  4 x 2048 x 4096 (256 blocks) is
// fastest in one piece: 185 us, 228 in 3.  The same prices serve every N and
// type, and sequences count as full whatever their lengths are.  In segments and
// in one piece, us:
//   1 x 512 x 512, N 16, 8 segments      bf16 17.5, 29.5   fp32 18.7, 33.8
//   2 x 2048 x 2048, N 16, 3             bf16 82, 113      fp32 93, 128
//   1 x 4096 x 2048, N 4, 20             bf16 76, 418      fp32 63, 326
//   1 x 4096 x 1024, N 64, 3             bf16 173, 253     fp32 144, 206
//   1 x 4096 x 1024, N 128, 3            bf16 351, 512     fp32 285, 411
ScanPlan make_plan(int B, int L, int D, int N, int groups) {
  constexpr int kSMs = 152, kMinLen = 64, kMaxSeg = 64;
  const int CH = block_channels(N);
  const double blocks = (double)B * groups * ((D / groups + CH - 1) / CH);
  auto rounds = [&](double n) {
    const double full = (double)(long long)(n / (2 * kSMs)), rest = n - full * 2 * kSMs;
    return 90 * full + (rest > kSMs ? 90 : rest > 0 ? 50 : 0);
  };
  ScanPlan best{1, L};
  double cost = rounds(blocks) * L;
  for (int n = 2; n <= kMaxSeg && L / n >= kMinLen; ++n) {
    const int len = ((L + n - 1) / n + 15) / 16 * 16;
    const double c = 2 * rounds(blocks * (n - 1)) * len + 12000 + 100 * n;
    if (c < cost && (L + len - 1) / len == n) cost = c, best = {n, len};
  }
  return best;
}

template <typename T, int P, int S, int NC, int ALIGN>
cudaError_t launch_kernel(const ScanParams<T> &p, cudaStream_t stream) {
  using Sh = ScanShape<P, S, NC, sizeof(T)>;
  const int per_group = p.D / p.groups;
  const long long blocks = (long long)p.B * p.groups * ((per_group + Sh::CH - 1) / Sh::CH);
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  auto *kernel = selective_scan_kernel<T, P, S, NC, ALIGN>;
  if (Sh::SMEM > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM);
    if (e != cudaSuccess) return e;
  }
  const unsigned segs = p.nseg > 1 ? p.nseg - 1 : 1;
  kernel<<<dim3((unsigned)blocks, segs), kThreads, Sh::SMEM, stream>>>(p, 0);
  if (p.nseg > 1) kernel<<<dim3((unsigned)blocks, segs), kThreads, Sh::SMEM, stream>>>(p, 1);
  return cudaGetLastError();
}

template <typename T, int P, int S, int NC>
cudaError_t launch_ps(const ScanArgs &a, const ScanParams<T> &p) {
  static_assert(ScanShape<P, S, NC, sizeof(T)>::CH == block_channels(P * S), "the plan's blocks");
  // The widest loads that the alignment of every row, and of every group in it,
  // allows (a block's first channel is a multiple of 16 bytes into its group).
  const int per_group = a.D / a.groups;
  auto rows_fit = [&](int bytes) {
    const int v = bytes / (int)sizeof(T);
    auto fits = [&](const void *q, long long stride) {
      return (reinterpret_cast<uintptr_t>(q) & (bytes - 1)) == 0 && stride % v == 0;
    };
    return (a.groups == 1 || (per_group % v == 0 && a.N % v == 0)) && fits(a.x, a.x_stride) &&
           fits(a.dt, a.dt_stride) && fits(a.z, a.z_stride) && fits(a.y, a.y_stride) &&
           fits(a.Bm, a.b_stride) && fits(a.Cm, a.c_stride);
  };
  if (rows_fit(16)) return launch_kernel<T, P, S, NC, ALIGN16>(p, a.stream);
  if constexpr (sizeof(T) < 4) {  // an fp32 row is always on 4-byte boundaries
    if (!rows_fit(4)) return launch_kernel<T, P, S, NC, ALIGN_ELT>(p, a.stream);
  }
  return launch_kernel<T, P, S, NC, ALIGN4>(p, a.stream);
}

template <typename T>
cudaError_t launch_t(const ScanArgs &a) {
  ScanPlan plan{1, a.L};
  if (a.workspace) plan = make_plan(a.B, a.L, a.D, a.N, a.groups);
  float *ws = static_cast<float *>(a.workspace);
  const size_t states = (size_t)(plan.nseg - 1) * a.B * a.D * a.N;
  const ScanParams<T> p{static_cast<const T *>(a.x), static_cast<const T *>(a.dt),
                        static_cast<const T *>(a.z), static_cast<const T *>(a.Bm),
                        static_cast<const T *>(a.Cm), a.x_stride, a.dt_stride, a.z_stride,
                        a.b_stride, a.c_stride, a.L, a.D, a.N, a.groups, a.A, a.dt_bias,
                        a.softplus, a.skip, a.h0, a.lengths, static_cast<T *>(a.y), a.y_stride,
                        a.h_final, a.B, plan.nseg, plan.seg_len, ws, ws ? ws + states : nullptr};
  if (a.L <= kStepTokens) return launch_steps<T>(p, a.stream);
  if (a.N <= 4) return launch_ps<T, 4, 1, 1>(a, p);
  if (a.N <= 8) return launch_ps<T, 4, 2, 1>(a, p);
  if (a.N <= 16) return launch_ps<T, 8, 2, 1>(a, p);
  if (a.N <= 32) return launch_ps<T, 8, 4, 1>(a, p);
  if (a.N <= 64) return launch_ps<T, 8, 8, 1>(a, p);
  if (a.N <= 128) return launch_ps<T, 8, 16, 2>(a, p);
  return launch_ps<T, 8, 32, 4>(a, p);
}

}  // namespace

// The fp32 kernels are a translation unit of their own (la_selective_scan_f32.cu
// includes this file), so that the two compile side by side.
#ifdef LA_SELECTIVE_SCAN_F32
cudaError_t launch_selective_scan_f32(const ScanArgs &a) { return launch_t<float>(a); }
#else
size_t selective_scan_workspace_bytes(int B, int L, int D, int N, int groups) {
  const ScanPlan plan = make_plan(B, L, D, N, groups);
  return (size_t)(plan.nseg - 1) * B * D * (N + 1) * sizeof(float);
}

cudaError_t launch_selective_scan(const ScanArgs &a) {
  return a.dtype == LA_F32 ? launch_selective_scan_f32(a) : launch_t<__nv_bfloat16>(a);
}
#endif

}  // namespace la
