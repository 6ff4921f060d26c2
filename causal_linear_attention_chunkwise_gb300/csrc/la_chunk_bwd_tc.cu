// la_chunk_bwd_tc.cu -- the backward walks on the 5th-gen tensor cores: bf16 inputs,
// d_k = d_v = D in {64, 128}, chunks of 128 tokens.
//
// The mathematics is la_chunk_bwd.cuh's, a chunk being one 128-row tile.  A
// block of 256 threads owns a segment of a sequence and one chunk of it at a time, in
// steps that all its threads take together:
//
//   1. one thread issues the products that need only the tiles and the state: the scores
//      (dO V^T; K Q^T and V dO^T, transposed, for dk and dv) and the state's
//      share of the gradients (dO S^T; K G and V G^T);
//   2. all threads turn the scores into operands (mask, decay, bf16) in tensor memory,
//      scale the state's share by each token's decay, and write the decayed K
//      (or Q) into the room of the state's operand;
//   3. one thread issues the products with the scores and the state's update;
//   4. all threads write the gradients out, add the update to the state, which they hold
//      in registers (fp32), and write it as the next chunk's operand, while the next tiles
//      arrive.
//
// Thread (warp w, lane l) owns row 32 (w % 4) + l of every accumulator and the
// columns of half w / 4, so a mask, a decay or a dot product is a row's own affair
// and a state row stays in one thread.  Operands are 128-byte swizzled tiles;
// each is read in both orientations (K-major and MN-major), none is transposed.
//
// NM = 3: the state and the decayed operand as three bf16 planes, which hold all
// of an fp32 value's bits, for the fp32 outputs (ddecay, dS0); one product each.
#include <cuda.h>

#include <algorithm>

#include "la_chunk_bwd.cuh"
#include "la_tc_sync.cuh"
#include "la_tma_host.h"

namespace la {
namespace {
using tc::Ctl;

constexpr int CT = 128;       // tokens of a chunk
constexpr int kThreads = 256;
constexpr uint32_t HI = smem_desc_sw128_hi(1024);

// Shared memory of a walk with TILES input tiles (in STAGES sets).  The planes come first:
// a D = 64 operand is read as one of 128 rows, whose other half may be anything.
template <int D, int NM, int TILES, int STAGES> struct Smem {
  static constexpr uint32_t BOX = CT * 128;         // 128 tokens x 64 columns
  static constexpr uint32_t TILE = D / 64 * BOX;
  static constexpr uint32_t SBOX = D * 128;         // 64 columns of a state
  static constexpr uint32_t SPLANE = D / 64 * SBOX;
  static constexpr uint32_t OFF_TILES = NM * TILE;  // planes: of the decayed tile or the state
  static constexpr uint32_t STAGE = TILES * TILE;
  static constexpr uint32_t OFF_LAM = OFF_TILES + STAGES * STAGE;
  static constexpr uint32_t OFF_COLS = OFF_LAM + CT * 8;
  static constexpr uint32_t OFF_BAR = OFF_COLS + 2 * CT * 4;
  static constexpr uint32_t BYTES = OFF_BAR + 128;
  static_assert(BYTES <= 232448, "exceeds the per-block shared memory limit");
};

struct Maps {
  CUtensorMap q, k, v, dO;
};

// A walk's block: its place, barriers and tensor memory.
struct Block {
  unsigned char *smem;
  uint32_t base;       // its shared address
  uint64_t *full;      // [2] tiles have landed
  uint64_t *mma;       // products are done
  Ctl *ctl;
  unsigned int *err;
  uint32_t tmem;
  uint32_t mma_phase;
  int warp, lane, quarter, half, row;
  bool failed;

  __device__ __forceinline__ void start(unsigned char *s, uint32_t off_bar, uint32_t columns,
                                        unsigned int *error) {
    smem = s;
    base = smem_u32(s);
    full = reinterpret_cast<uint64_t *>(s + off_bar);
    mma = full + 2;
    ctl = reinterpret_cast<Ctl *>(s + off_bar + 64);
    err = error;
    warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    quarter = warp % 4, half = warp / 4, row = quarter * 32 + lane;
    mma_phase = 0;
    failed = false;
    if (threadIdx.x == 0) {
      mbar_init(&full[0], 1);
      mbar_init(&full[1], 1);
      mbar_init(mma, 1);
      ctl->abort = 0;
      fence_mbarrier_init();
    }
    __syncwarp();
    if (warp == 0) {
      tmem_alloc(&ctl->tmem_base, columns);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    tmem = ctl->tmem_base;
  }
  __device__ __forceinline__ void finish(uint32_t columns) {
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, columns);
  }
  __device__ __forceinline__ void wait_full(int stage, uint32_t parity) {
    if (!tc::wait1(&full[stage], parity, ctl, err, KID_CHUNK_BWD_TC, 1)) failed = true;
    __syncwarp();
  }
  // The products issued since the last call are done.
  __device__ __forceinline__ void wait_mma() {
    if (!tc::wait1(mma, mma_phase, ctl, err, KID_CHUNK_BWD_TC, 2)) failed = true;
    mma_phase ^= 1;
    __syncwarp();
    tc_fence_after();
  }
  // TMEM address of column `col` in this warp's lanes.
  __device__ __forceinline__ uint32_t at(uint32_t col) const {
    return tmem + col + ((uint32_t)quarter << 21);
  }
};

// ---------------------------------------------------------------- products
// Operands as low descriptor words (start address, distance of 64-element blocks).
struct Operand {
  uint32_t lo, step;  // step: for 16 more along the contraction
  uint32_t wrap;      // K-major: extra per 64 of it
};
template <uint32_t BOX> __device__ __forceinline__ Operand along_row(uint32_t addr) {
  return {smem_desc_sw128_lo(addr, 16), 32 >> 4, (BOX - 128) >> 4};
}
template <uint32_t BOX> __device__ __forceinline__ Operand along_col(uint32_t addr) {
  return {smem_desc_sw128_lo(addr, BOX), 2048 >> 4, 0};
}
__device__ __forceinline__ uint32_t word(const Operand &o, int kk) {
  return o.lo + kk * o.step + kk / 4 * o.wrap;
}

// C[tmem] (+)= A B over a contraction of K.
template <int K>
__device__ __forceinline__ void product(uint32_t c, const Operand &a, const Operand &b,
                                        uint32_t idesc, bool add) {
#pragma unroll
  for (int kk = 0; kk < K / 16; ++kk)
    mma_bf16_w(c, word(a, kk), word(b, kk), HI, idesc, add || kk > 0);
}
// The same with A in tensor memory.
template <int K>
__device__ __forceinline__ void product_ta(uint32_t c, uint32_t a, const Operand &b,
                                           uint32_t idesc, bool add) {
#pragma unroll
  for (int kk = 0; kk < K / 16; ++kk)
    mma_bf16_ta_w(c, a + kk * 8, word(b, kk), HI, idesc, add || kk > 0);
}

// ---------------------------------------------------------------- tiles
template <int D>
__device__ __forceinline__ void load_tile_tma(const Block &b, uint32_t off, const CUtensorMap *map,
                                              uint64_t *bar, int token, int seq) {
#pragma unroll
  for (int x = 0; x < D / 64; ++x)
    tma_load_3d(b.smem + off + x * CT * 128, map, bar, x * 64, token, seq);
}

// phi = elu + 1 of a tile in place; rows past the last token stay zero.
template <int D> __device__ __forceinline__ void map_tile_tc(unsigned char *tile, int rows) {
#pragma unroll
  for (int i = 0; i < CT * D / 8 / kThreads; ++i) {
    const int x = threadIdx.x + i * kThreads;
    if ((x / 8) % CT >= rows) continue;
    uint4 *at = reinterpret_cast<uint4 *>(tile) + x;
    const uint4 u = *at;
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = la::pack_bf16(tc::elu1_fast(bf16_lo(w[e])), tc::elu1_fast(bf16_hi(w[e])));
    *at = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// dst (NM planes) = weight(token) * tile, at the tile's own places.
template <int D, int NM, typename Weight>
__device__ __forceinline__ void decayed_planes(const unsigned char *tile, unsigned char *dst,
                                               Weight weight) {
  constexpr uint32_t TILE = CT * D * 2;
#pragma unroll 4
  for (int i = 0; i < CT * D / 8 / kThreads; ++i) {
    const int x = threadIdx.x + i * kThreads;
    const uint4 u = reinterpret_cast<const uint4 *>(tile)[x];
    const float f = weight((x / 8) % CT);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t out[NM][4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      split<NM>(bf16_lo(w[e]) * f, bf16_hi(w[e]) * f, &out[0][e], 4);
#pragma unroll
    for (int m = 0; m < NM; ++m)
      reinterpret_cast<uint4 *>(dst + m * TILE)[x] =
          make_uint4(out[m][0], out[m][1], out[m][2], out[m][3]);
  }
}

// log2 decays of a chunk by one warp: lam[t] from the chunk's start, as two floats.
__device__ __forceinline__ void chunk_lam(const ChunkBwd &p, int seq, int t0, float2 *lam,
                                          int lane) {
  constexpr int N = CT / 32;
  double a[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    a[i] = log2_decay(p, seq, t0 + lane * N + i);
    if (i) a[i] += a[i - 1];
  }
  double run = a[N - 1];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const double x = __shfl_up_sync(0xffffffffu, run, off);
    if (lane >= off) run += x;
  }
  const double before = run - a[N - 1];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const double x = before + a[i];
    const float hi = (float)x;
    lam[lane * N + i] = make_float2(hi, (float)(x - hi));
  }
}

// ---------------------------------------------------------------- the state
// A thread's part of the state: row `row` (rows < D), columns half D/2 ..
template <int D, int NM> struct StateRow {
  static constexpr int N = D / 2;
  float c[N];

  __device__ __forceinline__ void load(const float *src, const Block &b) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (src && b.row < D)
        x = *reinterpret_cast<const float4 *>(src + (size_t)b.row * D + b.half * N + i);
      c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
    }
  }
  __device__ __forceinline__ void store(float *dst, const Block &b) const {
    if (b.row >= D) return;
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4 *>(dst + (size_t)b.row * D + b.half * N + i) =
          make_float4(c[i], c[i + 1], c[i + 2], c[i + 3]);
  }
  // As planes of operand tiles [D][D] (64-column boxes).
  __device__ __forceinline__ void planes(const Block &b) const {
    if (b.row >= D) return;
#pragma unroll
    for (int i = 0; i < N; i += 8) {
      const int col = b.half * N + i;
      uint32_t w[NM][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split<NM>(c[i + 2 * e], c[i + 2 * e + 1], &w[0][e], 4);
      unsigned char *at = b.smem + col / 64 * (D * 128) + b.row * 128 +
                          (((col % 64 / 8) ^ (b.row & 7)) << 4);
#pragma unroll
      for (int m = 0; m < NM; ++m)
        *reinterpret_cast<uint4 *>(at + m * (D * D * 2)) =
            make_uint4(w[m][0], w[m][1], w[m][2], w[m][3]);
    }
  }
  // c <- all c + the update in tensor memory.  The tensor cores cut a sum's last bits
  // off; formed chunk by chunk and added here, the cuts do not add up.
  __device__ __forceinline__ void update(const Block &b, uint32_t col, float all) {
    uint32_t r[32];
#pragma unroll
    for (int i = 0; i < N; i += 32) {
      tmem_ld32(b.at(col + b.half * N + i), r);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 32; ++e) c[i + e] = fmaf(all, c[i + e], __uint_as_float(r[e]));
    }
  }
  __device__ __forceinline__ float dot(const float *src, const Block &b) const {
    float s = 0.f;
    if (b.row < D) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const float4 x =
            *reinterpret_cast<const float4 *>(src + (size_t)b.row * D + b.half * N + i);
        s = fmaf(x.x, c[i], fmaf(x.y, c[i + 1], fmaf(x.z, c[i + 2], fmaf(x.w, c[i + 3], s))));
      }
    }
    return s;
  }
};

// 32 columns of a gradient row, in bf16, times phi's derivative at raw (elu + 1: e^x up
// to 0, then 1).
template <bool PHI>
__device__ __forceinline__ void store_32(__nv_bfloat16 *dst, const __nv_bfloat16 *raw,
                                         const float *f) {
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = f[i + e];
    if constexpr (PHI) {
      float x[8];
      load_raw<__nv_bfloat16, 8>(raw + i).unpack(x);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= x[e] > 0.f ? 1.f : __expf(x[e]);
    }
    store_vec<__nv_bfloat16, 8>(dst + i, y);
  }
}

// The dot product of 32 columns with a bf16 row.
__device__ __forceinline__ float dot_32(const __nv_bfloat16 *x, const float *f, float s) {
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    float y[8];
    load_raw<__nv_bfloat16, 8>(x + i).unpack(y);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(f[i + e], y[e], s);
  }
  return s;
}

__device__ __forceinline__ void as_floats(const uint32_t (&r)[32], float (&f)[32]) {
#pragma unroll
  for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(r[e]);
}

// ---------------------------------------------------------------- a segment's own share
template <int D, int NM>
__global__ void __launch_bounds__(kThreads, 1)
segment_share_tc_kernel(const __grid_constant__ Maps maps, const ChunkBwd p, unsigned int *err) {
  using SM = Smem<D, NM, 2, 2>;
  constexpr uint32_t id_kv = idesc_bf16_f32(128, D, true, true);
  constexpr bool PHI = NM == 1;  // elu + 1 comes with one plane alone
  extern __shared__ __align__(1024) unsigned char smem[];
  Block b;
  b.start(smem, SM::OFF_BAR, D, err);
  float2 *lam = reinterpret_cast<float2 *>(smem + SM::OFF_LAM);
  const int seq = blockIdx.x / (p.segments - 1), of = blockIdx.x % (p.segments - 1);
  const bool back = blockIdx.y != 0;
  const int seg = back ? of + 1 : of;
  const int c0 = seg * p.per, c1 = min(c0 + p.per, p.chunks), n = c1 - c0;
  const bool decays = p.decay_kind != LA_DECAY_NONE, phi = PHI && p.phi == LA_PHI_ELU1;
  auto token = [&](int i) { return (back ? c1 - 1 - i : c0 + i) * CT; };
  auto load = [&](int i) {
    const uint32_t at = SM::OFF_TILES + (i & 1) * SM::STAGE;
    mbar_arrive_expect_tx(&b.full[i & 1], SM::STAGE);
    load_tile_tma<D>(b, at, back ? &maps.q : &maps.k, &b.full[i & 1], token(i), seq);
    load_tile_tma<D>(b, at + SM::TILE, back ? &maps.dO : &maps.v, &b.full[i & 1], token(i), seq);
  };
  if (threadIdx.x == 0) load(0);
  StateRow<D, NM> state;
  state.load(nullptr, b);
  double total = 0.0;
  int i = 0;
  for (; i < n; ++i) {
    if (threadIdx.x == 0 && i + 1 < n) load(i + 1);  // its stage was read two chunks ago
    if (b.warp == 4 && decays) chunk_lam(p, seq, token(i), lam, b.lane);
    b.wait_full(i & 1, (i >> 1) & 1);
    unsigned char *tile = smem + SM::OFF_TILES + (i & 1) * SM::STAGE;
    if (phi) map_tile_tc<D>(tile, p.L - token(i));
    __syncthreads();
    const float2 end = decays ? lam[CT - 1] : make_float2(0.f, 0.f);
    if (decays) {
      if (back)
        decayed_planes<D, NM>(tile, smem, [&](int t) { return ex2_approx(lam[t].x); });
      else
        decayed_planes<D, NM>(tile, smem, [&](int t) { return decay_between(end, lam[t]); });
    }
    total += (double)end.x + end.y;
    fence_proxy_async_smem();
    tc_fence_before();
    if (__syncthreads_or(b.failed)) break;
    if (threadIdx.x == 0) {
      tc_fence_after();
      const uint32_t tile_at = smem_u32(tile);
      const Operand y = along_col<SM::BOX>(tile_at + SM::TILE);
      if (decays) {
#pragma unroll
        for (int m = NM - 1; m >= 0; --m)
          product<CT>(b.tmem, along_col<SM::BOX>(b.base + m * SM::TILE), y, id_kv, m < NM - 1);
      } else {
        product<CT>(b.tmem, along_col<SM::BOX>(tile_at), y, id_kv, false);
      }
      mma_commit(b.mma);
    }
    b.wait_mma();
    state.update(b, 0, decays ? ex2_approx(end.x) : 1.f);
    tc_fence_before();
    __syncthreads();  // lam and the planes are free, the update is read
  }
  if (i == n) {
    const size_t slot = (size_t)seq * (p.segments - 1) + of;
    state.store((back ? p.W : p.U) + slot * D * D, b);
    if (threadIdx.x == 0 && (!back || seg == p.segments - 1))
      p.total[(size_t)seq * p.segments + seg] = (float)total;
  } else if (threadIdx.x == 0) {  // the copies in flight end before their memory does
    for (int j = i; j < min(i + 2, n); ++j) tc::drain_wait(&b.full[j & 1], (j >> 1) & 1);
  }
  b.finish(D);
}

// ---------------------------------------------------------------- dq
template <int D, int NM>
__global__ void __launch_bounds__(kThreads, 1)
grad_q_tc_kernel(const __grid_constant__ Maps maps, const ChunkBwd p, unsigned int *err) {
  using SM = Smem<D, NM, 3, 1>;
  // Tensor memory: dO V^T, the state's share, the scores' share, the scores as operand; the
  // state's update takes the place of dO V^T.
  constexpr uint32_t T_S = 0, T_IN = 128, T_OUT = 128 + D, T_A = 128 + 2 * D, COLUMNS = 512;
  constexpr uint32_t id_s = idesc_bf16_f32(128, 128, false, false);
  constexpr uint32_t id_in = idesc_bf16_f32(128, D, false, false);
  constexpr uint32_t id_out = idesc_bf16_f32(128, D, false, true);
  constexpr uint32_t id_kv = idesc_bf16_f32(128, D, true, true);
  constexpr int N = D / 2;
  constexpr bool PHI = NM == 1;
  static_assert(T_A + 64 <= COLUMNS, "tensor memory");
  extern __shared__ __align__(1024) unsigned char smem[];
  Block b;
  b.start(smem, SM::OFF_BAR, COLUMNS, err);
  float2 *lam = reinterpret_cast<float2 *>(smem + SM::OFF_LAM);
  float *sums = reinterpret_cast<float *>(smem + SM::OFF_COLS);
  const int seq = blockIdx.x / p.segments, seg = blockIdx.x % p.segments;
  const int c0 = seg * p.per, c1 = min(c0 + p.per, p.chunks);
  const size_t e0 = (size_t)seq * p.L * D, es = (size_t)D * D;
  const bool decays = p.decay_kind != LA_DECAY_NONE, phi = PHI && p.phi == LA_PHI_ELU1;
  const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + e0;
  __nv_bfloat16 *dq = static_cast<__nv_bfloat16 *>(p.dq) + e0;
  constexpr uint32_t TK = SM::OFF_TILES, TV = TK + SM::TILE, TD = TV + SM::TILE;
  auto load = [&](int c) {
    mbar_arrive_expect_tx(&b.full[0], SM::STAGE);
    load_tile_tma<D>(b, TK, &maps.k, &b.full[0], c * CT, seq);
    load_tile_tma<D>(b, TV, &maps.v, &b.full[0], c * CT, seq);
    load_tile_tma<D>(b, TD, &maps.dO, &b.full[0], c * CT, seq);
  };
  if (threadIdx.x == 0) load(c0);
  StateRow<D, NM> state;
  state.load(seg ? p.U + ((size_t)seq * (p.segments - 1) + seg - 1) * es
                 : p.S0 ? p.S0 + (size_t)seq * es : nullptr, b);
  state.planes(b);
  int c = c0;
  for (; c < c1; ++c) {
    const int t0 = c * CT, t = t0 + b.row;
    b.wait_full(0, (c - c0) & 1);
    if (phi) map_tile_tc<D>(smem + TK, p.L - t0);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
      tc_fence_after();
      const Operand a = along_row<SM::BOX>(b.base + TD);
      product<D>(b.tmem + T_S, a, along_row<SM::BOX>(b.base + TV), id_s, false);
#pragma unroll
      for (int m = NM - 1; m >= 0; --m)
        product<D>(b.tmem + T_IN, a, along_row<SM::SBOX>(b.base + m * SM::SPLANE), id_in,
                   m < NM - 1);
      mma_commit(b.mma);
    }
    if (b.warp == 4 && decays) chunk_lam(p, seq, t0, lam, b.lane);
    __syncthreads();
    const float2 own = decays ? lam[b.row] : make_float2(0.f, 0.f);
    const float2 end = decays ? lam[CT - 1] : make_float2(0.f, 0.f);
    b.wait_mma();
    // the scores as operand: row j, tokens i <= j
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int i0 = b.half * 64 + x * 32;
      uint32_t w[16];
      if (i0 / 32 > b.quarter) {  // all behind the warp's rows
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = 0;
      } else {
        uint32_t r[32];
        float f[32];
        tmem_ld32(b.at(T_S + i0), r);
        tmem_ld_wait();
        as_floats(r, f);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int i = i0 + e;
          if (decays) f[e] *= decay_between(own, i <= b.row ? lam[i] : own);
          f[e] = i <= b.row ? f[e] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = la::pack_bf16(f[2 * e], f[2 * e + 1]);
      }
      tmem_st16(b.at(T_A + i0 / 2), w);
    }
    const bool more = c + 1 < c1;
    if (more && decays)
      decayed_planes<D, NM>(smem + TK, smem, [&](int i) { return decay_between(end, lam[i]); });
    tmem_st_wait();
    fence_proxy_async_smem();
    tc_fence_before();
    if (__syncthreads_or(b.failed)) break;
    if (threadIdx.x == 0) {
      tc_fence_after();
      const Operand k = along_col<SM::BOX>(b.base + TK), v = along_col<SM::BOX>(b.base + TV);
      product_ta<CT>(b.tmem + T_OUT, b.tmem + T_A, k, id_out, false);
      if (more) {
        if (decays) {
#pragma unroll
          for (int m = NM - 1; m >= 0; --m)
            product<CT>(b.tmem + T_S, along_col<SM::BOX>(b.base + m * SM::TILE), v, id_kv,
                        m < NM - 1);
        } else {
          product<CT>(b.tmem + T_S, k, v, id_kv, false);
        }
      }
      mma_commit(b.mma);
    }
    b.wait_mma();
    if (threadIdx.x == 0 && more && !b.failed) load(c + 1);
    const float head = ex2_approx(own.x), all = ex2_approx(end.x);
    float dot = 0.f;
#pragma unroll
    for (int x = 0; x < N; x += 32) {
      uint32_t r[32];
      float f[32], g[32];
      tmem_ld32(b.at(T_IN + b.half * N + x), r);
      tmem_ld_wait();
      as_floats(r, f);
      tmem_ld32(b.at(T_OUT + b.half * N + x), r);
      tmem_ld_wait();
      as_floats(r, g);
#pragma unroll
      for (int e = 0; e < 32; ++e) f[e] *= head;
      if (t < p.L) {
        const size_t at = (size_t)t * D + b.half * N + x;
        if (p.rq) dot = dot_32(q + at, f, dot);
#pragma unroll
        for (int e = 0; e < 32; ++e) g[e] += f[e];
        if (phi) store_32<PHI>(dq + at, q + at, g);
        else store_32<false>(dq + at, nullptr, g);
      }
    }
    float around = 0.f;
    if (more) {
      state.update(b, T_S, decays ? all : 1.f);
      state.planes(b);
    } else if (p.rq) {  // <G, e^L_C S>: the pairs around the segment's last chunk
      const float *G = seg + 1 < p.segments ? p.W + ((size_t)seq * (p.segments - 1) + seg) * es
                       : p.dSf ? p.dSf + (size_t)seq * es : nullptr;
      if (G) around = state.dot(G, b);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) around += __shfl_xor_sync(0xffffffffu, around, off);
      if (b.lane == 0) sums[CT + b.warp] = around * all;
    }
    if (p.rq) {
      if (b.half == 1) sums[b.row] = dot;
      __syncthreads();
      if (b.half == 0 && t < p.L) p.rq[(size_t)seq * p.L + t] = dot + sums[b.row];
      if (!more && threadIdx.x == 0) {
        float s = 0.f;
        for (int i = 0; i < kThreads / 32; ++i) s += sums[CT + i];
        p.around[(size_t)seq * p.segments + seg] = s;
      }
    }
  }
  if (c < c1 && threadIdx.x == 0) {
    tc::drain_wait(&b.full[0], (c - c0) & 1);
    tc::drain_wait(b.mma, b.mma_phase ^ 1);
  }
  b.finish(COLUMNS);
}

// ---------------------------------------------------------------- dk and dv
template <int D, int NM>
__global__ void __launch_bounds__(kThreads, 1)
grad_kv_tc_kernel(const __grid_constant__ Maps maps, const ChunkBwd p, unsigned int *err) {
  using SM = Smem<D, NM, 4, 1>;
  // Tensor memory: K Q^T and V dO^T, dv, dk.  When the scores have been read their operands
  // take columns 0..63 and 192..255, the state's update those between.
  constexpr uint32_t T_P = 0, T_DP = 128, T_V = 256, T_K = 256 + D, COLUMNS = 512;
  constexpr uint32_t T_AP = 0, T_ADP = 192, T_U = 64;
  constexpr uint32_t id_s = idesc_bf16_f32(128, 128, false, false);
  constexpr uint32_t id_in = idesc_bf16_f32(128, D, false, false);
  constexpr uint32_t id_out = idesc_bf16_f32(128, D, false, true);
  constexpr uint32_t id_kv = idesc_bf16_f32(128, D, true, true);
  constexpr int N = D / 2;
  constexpr bool PHI = NM == 1;
  extern __shared__ __align__(1024) unsigned char smem[];
  Block b;
  b.start(smem, SM::OFF_BAR, COLUMNS, err);
  float2 *lam = reinterpret_cast<float2 *>(smem + SM::OFF_LAM);
  float *part = reinterpret_cast<float *>(smem + SM::OFF_LAM);  // [4][CT], once lam is used
  const int seq = blockIdx.x / p.segments, seg = blockIdx.x % p.segments;
  const int c0 = seg * p.per, c1 = min(c0 + p.per, p.chunks), n = c1 - c0;
  const size_t e0 = (size_t)seq * p.L * D, es = (size_t)D * D;
  const bool decays = p.decay_kind != LA_DECAY_NONE, phi = PHI && p.phi == LA_PHI_ELU1;
  const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(p.k) + e0;
  __nv_bfloat16 *dk = static_cast<__nv_bfloat16 *>(p.dk) + e0;
  __nv_bfloat16 *dv = static_cast<__nv_bfloat16 *>(p.dv) + e0;
  constexpr uint32_t TQ = SM::OFF_TILES, TK = TQ + SM::TILE, TV = TK + SM::TILE,
                     TD = TV + SM::TILE;
  auto load = [&](int c) {
    mbar_arrive_expect_tx(&b.full[0], SM::STAGE);
    load_tile_tma<D>(b, TQ, &maps.q, &b.full[0], c * CT, seq);
    load_tile_tma<D>(b, TK, &maps.k, &b.full[0], c * CT, seq);
    load_tile_tma<D>(b, TV, &maps.v, &b.full[0], c * CT, seq);
    load_tile_tma<D>(b, TD, &maps.dO, &b.full[0], c * CT, seq);
  };
  if (threadIdx.x == 0) load(c1 - 1);
  StateRow<D, NM> state;
  state.load(seg + 1 < p.segments ? p.W + ((size_t)seq * (p.segments - 1) + seg) * es
             : p.dSf ? p.dSf + (size_t)seq * es : nullptr, b);
  state.planes(b);
  int done = 0;
  for (; done < n; ++done) {
    const int c = c1 - 1 - done, t0 = c * CT, t = t0 + b.row;
    b.wait_full(0, done & 1);
    if (phi) {
      map_tile_tc<D>(smem + TQ, p.L - t0);
      map_tile_tc<D>(smem + TK, p.L - t0);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
      tc_fence_after();
      const Operand ak = along_row<SM::BOX>(b.base + TK), av = along_row<SM::BOX>(b.base + TV);
      product<D>(b.tmem + T_P, ak, along_row<SM::BOX>(b.base + TQ), id_s, false);
      product<D>(b.tmem + T_DP, av, along_row<SM::BOX>(b.base + TD), id_s, false);
      product<D>(b.tmem + T_V, ak, along_col<SM::SBOX>(b.base), id_out, false);
#pragma unroll
      for (int m = NM - 1; m >= 0; --m)
        product<D>(b.tmem + T_K, av, along_row<SM::SBOX>(b.base + m * SM::SPLANE), id_in,
                   m < NM - 1);
      mma_commit(b.mma);
    }
    if (b.warp == 4 && decays) chunk_lam(p, seq, t0, lam, b.lane);
    __syncthreads();
    const float2 own = decays ? lam[b.row] : make_float2(0.f, 0.f);
    const float2 end = decays ? lam[CT - 1] : make_float2(0.f, 0.f);
    b.wait_mma();
    // the scores as operands: row i, tokens j >= i
    uint32_t wp[2][16], wd[2][16];
    float row_sum = 0.f, col_sum[2] = {0.f, 0.f};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int j0 = b.half * 64 + x * 32;
      if (j0 / 32 < b.quarter) {  // all in front of the warp's rows
#pragma unroll
        for (int e = 0; e < 16; ++e) wp[x][e] = wd[x][e] = 0;
        continue;
      }
      uint32_t r[32];
      float f[32], g[32];
      tmem_ld32(b.at(T_P + j0), r);
      tmem_ld_wait();
      as_floats(r, f);
      tmem_ld32(b.at(T_DP + j0), r);
      tmem_ld_wait();
      as_floats(r, g);
      float pair[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const int j = j0 + e;
        const float d = decays ? decay_between(j >= b.row ? lam[j] : own, own) : 1.f;
        pair[e] = j > b.row ? f[e] * g[e] * d : 0.f;
        f[e] = j >= b.row ? f[e] * d : 0.f;
        g[e] = j >= b.row ? g[e] * d : 0.f;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        wp[x][e] = la::pack_bf16(f[2 * e], f[2 * e + 1]);
        wd[x][e] = la::pack_bf16(g[2 * e], g[2 * e + 1]);
      }
      if (p.rc) {
#pragma unroll
        for (int e = 0; e < 32; ++e) row_sum += pair[e];
        // sums over the warp's rows: lane e ends with column e's
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
          const bool up = b.lane & off;
#pragma unroll
          for (int e = 0; e < off; ++e) {
            const float give = up ? pair[e] : pair[e + off];
            pair[e] = (up ? pair[e + off] : pair[e]) + __shfl_xor_sync(0xffffffffu, give, off);
          }
        }
        col_sum[x] = pair[0];
      }
    }
    tc_fence_before();
    __syncthreads();  // the scores are read: their operands may take their place
    tc_fence_after();
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      tmem_st16(b.at(T_AP + b.half * 32 + x * 16), wp[x]);
      tmem_st16(b.at(T_ADP + b.half * 32 + x * 16), wd[x]);
    }
    const float tail = decay_between(end, own);
    float dot = 0.f;
    if (decays) {  // the state's share, by each token's decay to the chunk's end
#pragma unroll
      for (int x = 0; x < 2 * N; x += 32) {
        const bool of_k = x >= N;
        const uint32_t at = b.at((of_k ? T_K : T_V) + b.half * N + x % N);
        uint32_t r[32];
        float f[32];
        tmem_ld32(at, r);
        tmem_ld_wait();
        as_floats(r, f);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          f[e] *= tail;
          r[e] = __float_as_uint(f[e]);
        }
        tmem_st32(at, r);
        if (of_k && p.rk && t < p.L) dot = dot_32(k + (size_t)t * D + b.half * N + x % N, f, dot);
      }
    }
    const bool more = done + 1 < n, update = more || (p.dS0 && seg == 0);
    if (update && decays)
      decayed_planes<D, NM>(smem + TQ, smem, [&](int i) { return ex2_approx(lam[i].x); });
    tmem_st_wait();
    fence_proxy_async_smem();
    tc_fence_before();
    if (__syncthreads_or(b.failed)) break;
    if (threadIdx.x == 0) {
      tc_fence_after();
      const Operand q = along_col<SM::BOX>(b.base + TQ), dO = along_col<SM::BOX>(b.base + TD);
      product_ta<CT>(b.tmem + T_V, b.tmem + T_AP, dO, id_out, true);
      product_ta<CT>(b.tmem + T_K, b.tmem + T_ADP, q, id_out, true);
      if (update) {
        if (decays) {
#pragma unroll
          for (int m = NM - 1; m >= 0; --m)
            product<CT>(b.tmem + T_U, along_col<SM::BOX>(b.base + m * SM::TILE), dO, id_kv,
                        m < NM - 1);
        } else {
          product<CT>(b.tmem + T_U, q, dO, id_kv, false);
        }
      }
      mma_commit(b.mma);
    }
    if (p.rk) {  // over the halves of a row and the quarters of a column, by way of lam's room
      const size_t to = (size_t)seq * p.L + t;
      part[b.quarter * CT + b.half * 64 + b.lane] = col_sum[0];
      part[b.quarter * CT + b.half * 64 + 32 + b.lane] = col_sum[1];
      __syncthreads();
      float col = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) col += part[i * CT + b.row];
      __syncthreads();
      if (b.half == 1) part[b.row] = row_sum, part[CT + b.row] = dot;
      __syncthreads();
      if (b.half == 0 && t < p.L) {
        p.rc[to] = col - (row_sum + part[b.row]);
        p.rk[to] = dot + part[CT + b.row];
      }
    }
    b.wait_mma();
    if (threadIdx.x == 0 && more && !b.failed) load(c - 1);
#pragma unroll
    for (int x = 0; x < N; x += 32) {
      uint32_t r[32];
      float f[32];
      const size_t at = (size_t)t * D + b.half * N + x;
      tmem_ld32(b.at(T_V + b.half * N + x), r);
      tmem_ld_wait();
      as_floats(r, f);
      if (t < p.L) store_32<false>(dv + at, nullptr, f);
      tmem_ld32(b.at(T_K + b.half * N + x), r);
      tmem_ld_wait();
      as_floats(r, f);
      if (t < p.L) {
        if (phi) store_32<PHI>(dk + at, k + at, f);
        else store_32<false>(dk + at, nullptr, f);
      }
    }
    if (update) state.update(b, T_U, decays ? ex2_approx(end.x) : 1.f);
    if (more) state.planes(b);
  }
  if (done == n) {
    if (p.dS0 && seg == 0) state.store(p.dS0 + (size_t)seq * es, b);
  } else if (threadIdx.x == 0) {
    tc::drain_wait(&b.full[0], done & 1);
    tc::drain_wait(b.mma, b.mma_phase ^ 1);
  }
  b.finish(COLUMNS);
}

template <int D, int NM>
cudaError_t launch_tc(const ChunkBwd &p, int seqs, cudaStream_t stream) {
  using SS = Smem<D, NM, 2, 2>;
  using SQ = Smem<D, NM, 3, 1>;
  using SK = Smem<D, NM, 4, 1>;
  Maps m;
  if (!make_tmap_bf16_3d(&m.q, p.q, D, p.L, seqs, 64, CT) ||
      !make_tmap_bf16_3d(&m.k, p.k, D, p.L, seqs, 64, CT) ||
      !make_tmap_bf16_3d(&m.v, p.v, D, p.L, seqs, 64, CT) ||
      !make_tmap_bf16_3d(&m.dO, p.dO, D, p.L, seqs, 64, CT))
    return cudaErrorInvalidValue;
  unsigned int *err = device_error_word();
  cudaError_t e;
  if (p.segments > 1) {
    auto share = segment_share_tc_kernel<D, NM>;
    static int set[64];
    if ((e = tc::set_smem_once(share, SS::BYTES, set)) != cudaSuccess) return e;
    share<<<dim3((unsigned)(seqs * (p.segments - 1)), 2), kThreads, SS::BYTES, stream>>>(m, p, err);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_segment_scan(p, seqs, stream)) != cudaSuccess) return e;
  }
  auto gq = grad_q_tc_kernel<D, NM>;
  auto gkv = grad_kv_tc_kernel<D, NM>;
  static int set_q[64], set_kv[64];
  if ((e = tc::set_smem_once(gq, SQ::BYTES, set_q)) != cudaSuccess) return e;
  if ((e = tc::set_smem_once(gkv, SK::BYTES, set_kv)) != cudaSuccess) return e;
  gq<<<seqs * p.segments, kThreads, SQ::BYTES, stream>>>(m, p, err);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  gkv<<<seqs * p.segments, kThreads, SK::BYTES, stream>>>(m, p, err);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chunk_bwd_tc(const ChunkBwd &p, int seqs, bool planes, cudaStream_t stream) {
  if (p.n_k == 128)
    return planes ? launch_tc<128, 3>(p, seqs, stream) : launch_tc<128, 1>(p, seqs, stream);
  return planes ? launch_tc<64, 3>(p, seqs, stream) : launch_tc<64, 1>(p, seqs, stream);
}

}  // namespace la
