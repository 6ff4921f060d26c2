// la_chunk_bwd_tc.cu -- the backward walks on the 5th-gen tensor cores: bf16 inputs,
// chunks of 128 tokens, widths padded to D = 64 or 128 (the copies fill with zeros and
// leave out what lies past a row's end; mma.sync at these widths took 361 us for 4 x 16 x 4096 x
// 32 x 64 with token decays, 468 for 2 x 16 x 4096 x 64 x 128, where these take 198 and 163).
//
// The mathematics is la_chunk_bwd.cuh's, a chunk being one 128-row tile.  A
// block of 512 threads owns a segment of a sequence and one chunk of it at a time, in
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
// Thread (warp w, lane l) owns row 32 (w % 4) + l of every accumulator and the columns
// of part w / 4, so a mask and a decay are a row's own affair and a state's row stays in four
// threads.  With 256 threads, half a row each, the steps between the products waited longer for
// tensor memory (2 x 32 x 8192 x 128 with per-head decays: grad_q 211 us against 188,
// grad_kv 257 against 228).  Operands are 128-byte swizzled tiles;
// each is read in both orientations (K-major and MN-major), none is transposed.
//
// NM = 3: the state and the decayed operand as three bf16 planes, which hold all
// of an fp32 value's bits, for the fp32 outputs (ddecay, dS0); one product each.
//
// What bounds it at D = 128, NM = 3: no unit by itself, but shared memory and the steps' order
// together.  A chunk of grad_kv moves some 1.1 MB through shared memory (640 KB of them operands of
// the products, each of which takes its 512 clocks' whole bandwidth), 9000 clocks of 13200; the
// other third goes into five barriers of a block's 512 threads, and an SM holds one block (tensor
// pipe 38% busy, shared memory 31% by the products and 22% by loads and stores, DRAM 48%).  Loads
// issued earlier, or dv's share scaled while dk's products run, changed nothing (545 us, when it
// took that, for 1 x 16 x 32768 x 128 gates with either, both or none).
//
// A call that wants dS0 alone leaves out the pairs and the row sums of ddecay (2 x 32 x 8192 x 128
// with per-head decays and states: 478 us, with them 502).
#include <cuda.h>

#include <algorithm>

#include "la_chunk_bwd.cuh"
#include "la_tc_sync.cuh"
#include "la_tma_host.h"

namespace la {
namespace {
using tc::Ctl;

constexpr int CT = 128;       // tokens of a chunk
// Parts of a row: 32 tokens' scores, D / PARTS columns.
constexpr int PARTS = 4, kThreads = CT * PARTS;
// The thread that issues products and copies waits when their queue is full: it is one of a warp
// that has no scores to work on, all of its columns lying outside the mask.
constexpr int kLeaderQ = 384, kLeaderKV = 96;
constexpr uint32_t HI = smem_desc_sw128_hi(1024);
static_assert(kThreads / 32 == kShares, "a share for each warp");

// Shared memory of a walk with TILES input tiles (in STAGES sets) and MORE others.  The planes come
// first: a D = 64 operand is read as one of 128 rows, whose other half may be anything.
template <int D, int NM, int TILES, int STAGES, int MORE = 0> struct Smem {
  static constexpr uint32_t BOX = CT * 128;         // 128 tokens x 64 columns
  static constexpr uint32_t TILE = D / 64 * BOX;
  static constexpr uint32_t OFF_TILES = NM * TILE;  // planes: of the decayed tile or the state
  static constexpr uint32_t STAGE = TILES * TILE;
  static constexpr uint32_t OFF_EXTRA = OFF_TILES + STAGES * STAGE;
  static constexpr uint32_t OFF_LAM = OFF_EXTRA + MORE * TILE;     // float2 [CT]
  static constexpr uint32_t OFF_FAC = OFF_LAM + CT * 8;            // float [CT]
  static constexpr uint32_t OFF_MORE = OFF_FAC + CT * 4;           // float [2 CT]
  static constexpr uint32_t OFF_BAR = OFF_MORE + 2 * CT * 4;
  static constexpr uint32_t BYTES = OFF_BAR + 128;
  static_assert(BYTES <= 232448, "exceeds the per-block shared memory limit");
};
// phi's values lie in shared memory as bf16, and what that rounding leaves out in a tile of its own
// (low): with one plane alone, phi's rounding would be added to the outputs' own, 3.0e-3 of dq and dk
// instead of 2.35e-3 (outputs rounded from fp32: 1.7e-3).  The products of scores take it as a second
// product.  A state of 64 rows leaves half of the lanes of its update free, and the rows of low's share
// take these (SPLIT): without a product more they become the state's second plane (4 x 16 x 4096 x 64:
// 140 us; with a product of its own for low's share 150, without low 132).
template <int D, bool PHI, bool DECAY> constexpr bool kSplit = PHI && !DECAY && D == 64;
template <int D> struct StateTile {
  static constexpr uint32_t BOX = D * 128;  // 64 columns of a state
  static constexpr uint32_t PLANE = D / 64 * BOX;
};

struct Maps {
  CUtensorMap q, k, v, dO, dq, dk, dv;
};

// A walk's block: its place, barriers and tensor memory.
struct Block {
  unsigned char *smem;
  uint32_t base;       // its shared address
  uint64_t *full;      // [2] tiles have landed
  uint64_t *mma;       // [4] products are done
  int *narrow;         // [4] whether a block of 32 tokens takes factors on its diagonal
  Ctl *ctl;
  unsigned int *err;
  uint32_t tmem;
  int warp, lane, quarter, part, row;
  bool failed;

  __device__ __forceinline__ void start(unsigned char *s, uint32_t off_bar, uint32_t columns,
                                        unsigned int *error) {
    smem = s;
    base = smem_u32(s);
    full = reinterpret_cast<uint64_t *>(s + off_bar);
    mma = full + 2;
    narrow = reinterpret_cast<int *>(s + off_bar + 80);
    ctl = reinterpret_cast<Ctl *>(s + off_bar + 64);
    err = error;
    warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    quarter = warp % 4, part = warp / 4, row = quarter * 32 + lane;
    failed = false;
    if (threadIdx.x == 0) {
      mbar_init(&full[0], 1);
      mbar_init(&full[1], 1);
      for (int i = 0; i < 4; ++i) mbar_init(&mma[i], 1);
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
  // The products committed to mma[i] are done.
  __device__ __forceinline__ void wait_mma(int i, uint32_t parity) {
    if (!tc::wait1(&mma[i], parity, ctl, err, KID_CHUNK_BWD_TC, 2 + i)) failed = true;
    __syncwarp();
    tc_fence_after();
  }
  // TMEM address of column `col` in this warp's lanes.
  __device__ __forceinline__ uint32_t at(uint32_t col) const {
    return tmem + col + ((uint32_t)quarter << 21);
  }
  // Two sums of each part of a row, by tensor memory's columns from `col` on: left by the parts
  // behind the first, and added to the first one's (a barrier later).
  __device__ __forceinline__ void leave(uint32_t col, float x, float y) const {
    if (part) tmem_st2(at(col + (part - 1) * 2), __float_as_uint(x), __float_as_uint(y));
    tmem_st_wait();
  }
  __device__ __forceinline__ void gather(uint32_t col, float &x, float &y) const {
    uint32_t r[8];
    tc_fence_after();
    tmem_ld8(at(col), r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < PARTS - 1; ++i)
      x += __uint_as_float(r[2 * i]), y += __uint_as_float(r[2 * i + 1]);
  }
  // 16 bytes at column `col` (a multiple of 8) of this thread's row in a tile of tokens.
  __device__ __forceinline__ uint4 *cell(uint32_t tile, int col) const {
    return reinterpret_cast<uint4 *>(smem + tile + col / 64 * (CT * 128) + row * 128 +
                                     (((col % 64 / 8) ^ (row & 7)) << 4));
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
// 64 columns at addr and 64 at next, which lies behind it.
__device__ __forceinline__ Operand along_cols(uint32_t addr, uint32_t next) {
  return {smem_desc_sw128_lo(addr, next - addr), 2048 >> 4, 0};
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
template <int D>
__device__ __forceinline__ void prefetch_tile(const CUtensorMap *map, int token, int seq,
                                              int width) {
#pragma unroll
  for (int x = 0; x < D / 64; ++x)
    if (x * 64 < width) tma_prefetch_3d(map, x * 64, token, seq);
}
// Rows past the last token, and columns past the width, are not written.
template <int D>
__device__ __forceinline__ void store_tile_tma(const Block &b, uint32_t off,
                                               const CUtensorMap *map, int token, int seq,
                                               int width) {
#pragma unroll
  for (int x = 0; x < D / 64; ++x)
    if (x * 64 < width) tma_store_3d(map, b.smem + off + x * CT * 128, x * 64, token, seq);
}

// dst = elu + 1 of a tile (dst may be the tile) as bf16, and, LOW, low = what that rounding left out;
// rows past the last token and columns past the width are zero.
template <int D, bool LOW>
__device__ __forceinline__ void map_tile_tc(const unsigned char *tile, unsigned char *dst,
                                            unsigned char *low, int rows, int width) {
#pragma unroll
  for (int i = 0; i < CT * D / 8 / kThreads; ++i) {
    const int x = threadIdx.x + i * kThreads;
    const int row = x / 8 % CT, col = x / 8 / CT * 64 + ((x % 8) ^ (row & 7)) * 8;
    const bool live = row < rows && col < width;
    const uint4 u = reinterpret_cast<const uint4 *>(tile)[x];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t out[1 + LOW][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      split<1 + LOW>(tc::elu1_fast(bf16_lo(w[e])), tc::elu1_fast(bf16_hi(w[e])), &out[0][e], 4);
#pragma unroll
      for (int n = 0; n < 1 + LOW; ++n)
        if (!live) out[n][e] = 0;
    }
    reinterpret_cast<uint4 *>(dst)[x] = make_uint4(out[0][0], out[0][1], out[0][2], out[0][3]);
    if constexpr (LOW)
      reinterpret_cast<uint4 *>(low)[x] = make_uint4(out[1][0], out[1][1], out[1][2], out[1][3]);
  }
}

// dst (NM planes) = weight(token) * (tile + low), at the tile's own places: ROWS tokens from row0
// on.  LOW: there is a low.
template <int D, int NM, int ROWS, bool LOW, typename Weight>
__device__ __forceinline__ void decayed_rows(const unsigned char *tile, const unsigned char *low,
                                             unsigned char *dst, int row0, Weight weight) {
  constexpr uint32_t TILE = CT * D * 2;
#pragma unroll 4
  for (int i = 0; i < ROWS * D / 8 / kThreads; ++i) {
    const int x = threadIdx.x + i * kThreads, row = row0 + x / 8 % ROWS;
    const int at = x / 8 / ROWS * (CT * 8) + row * 8 + x % 8;  // in 16-byte cells
    const uint4 u = reinterpret_cast<const uint4 *>(tile)[at];
    const float f = weight(row);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t l[4] = {0, 0, 0, 0};
    if constexpr (LOW) {
      const uint4 v = reinterpret_cast<const uint4 *>(low)[at];
      l[0] = v.x, l[1] = v.y, l[2] = v.z, l[3] = v.w;
    }
    uint32_t out[NM][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = LOW ? bf16_lo(w[e]) + bf16_lo(l[e]) : bf16_lo(w[e]);
      const float y = LOW ? bf16_hi(w[e]) + bf16_hi(l[e]) : bf16_hi(w[e]);
      split<NM>(x * f, y * f, &out[0][e], 4);
    }
#pragma unroll
    for (int m = 0; m < NM; ++m)
      reinterpret_cast<uint4 *>(dst + m * TILE)[at] =
          make_uint4(out[m][0], out[m][1], out[m][2], out[m][3]);
  }
}

__device__ __forceinline__ void load_16(const Block &b, uint32_t col, float (&f)[16]) {
  uint32_t r[16];
  tmem_ld16(b.at(col), r);
  tmem_ld_wait();
#pragma unroll
  for (int e = 0; e < 16; ++e) f[e] = __uint_as_float(r[e]);
}
// ---------------------------------------------------------------- decays
// A chunk's log2 decays on their way to shared memory: the threads of part 0 hold a
// token each, loaded a chunk ahead.  A decay is the product of a factor of the row and one of the
// column, e^(L_j - E) e^(E - L_i) with E at the end of a block of 32 tokens between them, so
// both are at most 1.  Pairs of one block take their own block's end (dq) or the
// end before it: one factor is then above 1, up to what the block decays by.  A block
// that decays by more than 2^60 takes an exponential for each pair instead.
struct TokenDecay {
  float2 own, before;  // at the token, and at the end of the block in front of it

  __device__ __forceinline__ void load(const ChunkBwd &p, const Block &b, int seq, int c) {
    own = before = make_float2(0.f, 0.f);
    if (b.part || p.decay_kind == LA_DECAY_NONE) return;
    const float2 *lam = p.lam + ((size_t)seq * p.chunks + c) * CT;
    own = lam[b.row];
    if (b.quarter) before = lam[b.quarter * 32 - 1];
  }
  // LATER: for columns behind the rows (e^(L - E) of the block before), else e^(E - L).
  template <bool LATER>
  __device__ __forceinline__ void put(const Block &b, float2 *lam, float *fac) const {
    float2 at = before;
    if (!LATER) {
      at.x = __shfl_sync(0xffffffffu, own.x, 31);
      at.y = __shfl_sync(0xffffffffu, own.y, 31);
    }
    lam[b.row] = own;
    fac[b.row] = LATER ? decay_between(own, at) : decay_between(at, own);
    const bool all = __all_sync(0xffffffffu, fabsf(own.x - before.x) < 60.f);
    if (b.lane == 0) b.narrow[b.quarter] = all;
  }
};

// The decays of a thread's row and a column block's 32 tokens, by its columns.
struct RowDecay {
  const float *factors;  // of the columns, or null: an exponential for each pair
  float mine;
  const float2 *lam;
  float2 own;
  bool later;

  // LATER: the columns come after the row (else before it); anything outside the mask.
  template <bool LATER>
  __device__ __forceinline__ void start(const Block &b, int block, const float2 *lams,
                                        const float *fac, float2 o) {
    factors = nullptr, mine = 0.f, own = o, later = LATER;
    lam = lams + block * 32;
    if (block == b.quarter && !b.narrow[block]) return;
    float2 at = make_float2(0.f, 0.f);
    if (!LATER || block) at = lams[LATER ? block * 32 - 1 : block * 32 + 31];
    mine = LATER ? decay_between(at, own) : decay_between(own, at);
    factors = fac + block * 32;
  }
  template <int W> __device__ __forceinline__ void get(int at, float (&d)[W]) const {
    if (factors) {
#pragma unroll
      for (int e = 0; e < W; e += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(factors + at + e);
        d[e] = mine * x.x, d[e + 1] = mine * x.y, d[e + 2] = mine * x.z, d[e + 3] = mine * x.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float2 other = lam[at + e];
        const float x = (own.x - other.x) + (own.y - other.y);
        d[e] = ex2_approx(later ? -x : x);
      }
    }
  }
};

// ---------------------------------------------------------------- the state
// A thread's part of the state: row `row` (rows < D), N columns from N part on.  SPLIT: the rows from D
// on hold the share of phi's low parts.
template <int D, int NM, bool SPLIT = false> struct StateRow {
  static constexpr int N = D / PARTS;
  float c[N];

  // The same of a [n_k][n_v] tensor: element `at` of it, or none of its.
  __device__ __forceinline__ static bool place(const Block &b, const ChunkBwd &p, int i,
                                               size_t &at) {
    const int col = b.part * N + i;
    at = (size_t)b.row * p.n_v + col;
    return b.row < p.n_k && col < p.n_v;
  }
  __device__ __forceinline__ void load(const float *src, const Block &b, const ChunkBwd &p) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      size_t at;
      if (src && place(b, p, i, at)) x = *reinterpret_cast<const float4 *>(src + at);
      c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
    }
  }
  __device__ __forceinline__ void store(float *dst, const Block &b, const ChunkBwd &p) const {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      size_t at;
      if (place(b, p, i, at))
        *reinterpret_cast<float4 *>(dst + at) = make_float4(c[i], c[i + 1], c[i + 2], c[i + 3]);
    }
  }
  // As planes of operand tiles [D][D] (64-column boxes).
  __device__ __forceinline__ void planes(const Block &b) const {
    static_assert(!SPLIT || (NM == 1 && D == 64), "two planes, of 64 rows each");
    if (!SPLIT && b.row >= D) return;
#pragma unroll
    for (int i = 0; i < N; i += 8) {
      const int col = b.part * N + i;
      uint32_t w[NM][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split<NM>(c[i + 2 * e], c[i + 2 * e + 1], &w[0][e], 4);
      // SPLIT: row 64 is the second plane's first
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
  __device__ __forceinline__ void update(const Block &b, uint32_t col, float2 all) {
    if (!SPLIT && b.quarter * 32 >= D) return;
    uint32_t r[N];
    if constexpr (N == 32) tmem_ld32(b.at(col + b.part * N), r);
    else tmem_ld16(b.at(col + b.part * N), r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = decayed_sum(all, c[i], __uint_as_float(r[i]));
  }
  // The state as it lies in a block's threads, and its product with such a one.
  __device__ __forceinline__ void keep(float *dst, const Block &b) const {
    if (b.row >= D) return;
#pragma unroll
    for (int i = 0; i < N; i += 4)
      reinterpret_cast<float4 *>(dst)[i / 4 * (PARTS * D) + b.part * D + b.row] =
          make_float4(c[i], c[i + 1], c[i + 2], c[i + 3]);
  }
  __device__ __forceinline__ float dot_kept(const float *src, const Block &b) const {
    float s = 0.f;
    if (b.row < D) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const float4 x =
            reinterpret_cast<const float4 *>(src)[i / 4 * (PARTS * D) + b.part * D + b.row];
        s = fmaf(x.x, c[i], fmaf(x.y, c[i + 1], fmaf(x.z, c[i + 2], fmaf(x.w, c[i + 3], s))));
      }
    }
    return s;
  }
  __device__ __forceinline__ float dot(const float *src, const Block &b, const ChunkBwd &p) const {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      size_t at;
      if (!place(b, p, i, at)) continue;
      const float4 x = *reinterpret_cast<const float4 *>(src + at);
      s = fmaf(x.x, c[i], fmaf(x.y, c[i + 1], fmaf(x.z, c[i + 2], fmaf(x.w, c[i + 3], s))));
    }
    return s;
  }
};

// 8 values of a gradient into a staging cell; SLOPE: times phi's derivative at the raw values
// that another cell, or the same, holds (elu + 1: e^x up to 0, then 1).
template <bool SLOPE>
__device__ __forceinline__ void stage_8(uint4 *cell, const uint4 *raw, const float *f) {
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = f[e];
  if constexpr (SLOPE) {
    const uint4 u = *raw;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = e % 2 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
      y[e] *= x > 0.f ? 1.f : __expf(x);
    }
  }
  *cell = make_uint4(la::pack_bf16(y[0], y[1]), la::pack_bf16(y[2], y[3]),
                     la::pack_bf16(y[4], y[5]), la::pack_bf16(y[6], y[7]));
}
// 16 values in each lane: the sum of value l % 16 over the 16 lanes of this half of the warp.  Each
// step halves the values that a lane keeps.
__device__ __forceinline__ float lanes_of_16(float (&v)[16], int lane) {
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) {
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < off; ++i)
      v[i] = (up ? v[i + off] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + off], off);
  }
  return v[0];
}
// The same of two: lo in the lanes below 16, hi in the others, each over both halves.
__device__ __forceinline__ float lanes_of_2(float lo, float hi, int lane) {
  const bool up = lane & 16;
  return (up ? hi : lo) + __shfl_xor_sync(0xffffffffu, up ? lo : hi, 16);
}
__device__ __forceinline__ float dot_8(const uint4 &u, const float *f, float s) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    s = fmaf(f[2 * e], bf16_lo(w[e]), fmaf(f[2 * e + 1], bf16_hi(w[e]), s));
  return s;
}

// ---------------------------------------------------------------- a segment's own share
// The decayed tile is formed in two halves of 64 tokens, each while the products of the other
// run; a chunk's sum is added to the state while the next one's products run.
template <int D, int NM, bool PHI, bool DECAY>
using ShareSmem = Smem<D, DECAY ? NM : 0, 2, 2, PHI ? DECAY ? 1 : 2 : 0>;
template <int D, int NM, bool PHI, bool DECAY>
__global__ void __launch_bounds__(kThreads, 1)
segment_share_tc_kernel(const __grid_constant__ Maps maps, const ChunkBwd p, unsigned int *err) {
  using SM = ShareSmem<D, NM, PHI, DECAY>;
  constexpr bool SPLIT = kSplit<D, PHI, DECAY>;
  constexpr uint32_t id_kv = idesc_bf16_f32(128, D, true, true), COLUMNS = 2 * D;
  extern __shared__ __align__(1024) unsigned char smem[];
  Block b;
  b.start(smem, SM::OFF_BAR, COLUMNS, err);
  float *weights = reinterpret_cast<float *>(smem + SM::OFF_LAM);   // [2][CT]
  float2 *ends = reinterpret_cast<float2 *>(smem + SM::OFF_FAC);    // [2] the chunk's log decay
  const int seq = blockIdx.x / (p.segments - 1), of = blockIdx.x % (p.segments - 1);
  const bool back = blockIdx.y != 0;
  const int seg = back ? of + 1 : of;
  const int c0 = seg * p.per, c1 = min(c0 + p.per, p.chunks), n = c1 - c0;
  const CUtensorMap *mx = back ? &maps.q : &maps.k, *my = back ? &maps.dO : &maps.v;
  auto chunk = [&](int i) { return back ? c1 - 1 - i : c0 + i; };
  auto load = [&](int i) {
    const uint32_t at = SM::OFF_TILES + (i & 1) * SM::STAGE;
    mbar_arrive_expect_tx(&b.full[i & 1], SM::STAGE);
    load_tile_tma<D>(b, at, mx, &b.full[i & 1], chunk(i) * CT, seq);
    load_tile_tma<D>(b, at + SM::TILE, my, &b.full[i & 1], chunk(i) * CT, seq);
  };
  if (threadIdx.x == 0) {
    load(0);
    if (n > 1) load(1);
  }
  StateRow<D, NM, SPLIT> state;
  state.load(nullptr, b, p);
  double total = 0.0;
  // each thread of part 0: its token's log decay and the chunk's, a chunk ahead
  float2 own = make_float2(0.f, 0.f), end = own;
  auto fetch = [&](int i) {
    if (!DECAY || b.part) return;
    const float2 *lam = p.lam + ((size_t)seq * p.chunks + chunk(i)) * CT;
    own = lam[b.row], end = lam[CT - 1];
  };
  auto put = [&](int i) {
    if (!DECAY || b.part) return;
    weights[(i & 1) * CT + b.row] = back ? ex2_approx(own.x) : decay_between(end, own);
    if (b.row == 0) ends[i & 1] = end;
  };
  fetch(0);
  put(0);
  if (n > 1) fetch(1);
  __syncthreads();
  float2 last = make_float2(0.f, 0.f);  // of the chunk whose sum is not yet added
  int i = 0;
  bool stop = false;
  for (; i < n; ++i) {
    const float2 all = exp2_two(last);
    b.wait_full(i & 1, (i >> 1) & 1);
    unsigned char *tile = smem + SM::OFF_TILES + (i & 1) * SM::STAGE;
    const uint32_t tile_at = smem_u32(tile), sum = b.tmem + (i & 1) * D;
    const Operand y = along_col<SM::BOX>(tile_at + SM::TILE);
    // phi's low parts: without decays one of two tiles in turn, since the last chunk's may still be read
    const uint32_t low = SM::OFF_EXTRA + (DECAY ? 0 : (i & 1) * SM::TILE);
    if (PHI) {
      map_tile_tc<D, true>(tile, tile, smem + low, p.L - chunk(i) * CT, p.n_k);
      if (DECAY) __syncthreads();
    }
    if (DECAY) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (i > 0) b.wait_mma(h, (i - 1) & 1);
        if (h == 1) {
          if (threadIdx.x == 0 && i > 0 && i + 1 < n) load(i + 1);
          __syncwarp();
          if (i + 1 < n) {
            put(i + 1);
            if (i + 2 < n) fetch(i + 2);
          }
        }
        const float *w = weights + (i & 1) * CT;
        decayed_rows<D, NM, 64, PHI>(tile, smem + low, smem, h * 64, [&](int t) { return w[t]; });
        fence_proxy_async_smem();
        tc_fence_before();
        if ((stop = __syncthreads_or(b.failed))) break;
        if (threadIdx.x == 0) {
          tc_fence_after();
#pragma unroll
          for (int m = NM - 1; m >= 0; --m) {
            const Operand x = along_col<SM::BOX>(b.base + m * SM::TILE);
#pragma unroll
            for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
              mma_bf16_w(sum, word(x, kk), word(y, kk), HI, id_kv, h > 0 || m < NM - 1 || kk > 0);
          }
          mma_commit(&b.mma[h]);
        }
      }
      if (stop) break;
    } else {
      if (i > 0) b.wait_mma(1, (i - 1) & 1);
      if (threadIdx.x == 0 && i > 0 && i + 1 < n) load(i + 1);
      __syncwarp();
      fence_proxy_async_smem();
      tc_fence_before();
      if ((stop = __syncthreads_or(b.failed))) break;
      if (threadIdx.x == 0) {
        tc_fence_after();
        constexpr bool TWO = PHI && !SPLIT;
        if (TWO) product<CT>(sum, along_col<SM::BOX>(b.base + low), y, id_kv, false);
        product<CT>(sum, SPLIT ? along_cols(tile_at, b.base + low) : along_col<SM::BOX>(tile_at), y,
                    id_kv, TWO);
        mma_commit(&b.mma[1]);
      }
    }
    if (i > 0) state.update(b, ((i - 1) & 1) * D, all);
    tc_fence_before();
    if (DECAY) {
      last = ends[i & 1];
      total += (double)last.x + last.y;
    }
  }
  if (!stop) {
    b.wait_mma(1, (n - 1) & 1);
    state.update(b, ((n - 1) & 1) * D, exp2_two(last));
    const size_t slot = (size_t)seq * (p.segments - 1) + of;
    if constexpr (SPLIT) {  // both shares of the state in one
      float *other = reinterpret_cast<float *>(smem) + b.row % D * D + b.part * (D / PARTS);
      if (b.row >= D)
#pragma unroll
        for (int j = 0; j < D / PARTS; ++j) other[j] = state.c[j];
      __syncthreads();
      if (b.row < D)
#pragma unroll
        for (int j = 0; j < D / PARTS; ++j) state.c[j] += other[j];
    }
    state.store((back ? p.W : p.U) + slot * p.n_k * p.n_v, b, p);
    if (threadIdx.x == 0 && (!back || seg == p.segments - 1))
      p.total[(size_t)seq * p.segments + seg] = (float)total;
  } else if (threadIdx.x == 0) {  // the copies in flight end before their memory does
    for (int j = i; j < min(i + 2, n); ++j) tc::drain_wait(&b.full[j & 1], (j >> 1) & 1);
  }
  b.finish(COLUMNS);
}

// Sets of input tiles of the walks below: with two, which D = 64 has room for, a chunk's tiles are
// loaded while the last chunk is worked on (4 x 16 x 4096 x 64 elu1, before phi's low parts: grad_q 45
// us, grad_kv 58; with one set 53 and 70).
template <int D> constexpr int kStages = D == 64 ? 2 : 1;

// ---------------------------------------------------------------- dq
template <int D, int NM, bool PHI, bool DECAY>
__global__ void __launch_bounds__(kThreads, 1)
grad_q_tc_kernel(const __grid_constant__ Maps maps, const ChunkBwd p, unsigned int *err) {
  // The fourth tile: q, where it is needed (for ddecay, for phi's derivative), then dq on its way
  // out.
  using SM = Smem<D, NM, 4, kStages<D>, PHI>;
  using ST = StateTile<D>;
  constexpr bool SPLIT = kSplit<D, PHI, DECAY>;
  constexpr int NS = SPLIT ? 2 : NM;  // planes of the state
  constexpr bool TWO = kStages<D> == 2, HAS_Q = (NM == 3 && DECAY) || PHI;
  // Tensor memory: dO V^T, the state's share, the scores' share, the scores as operand; the
  // state's update takes the place of dO V^T.
  constexpr uint32_t T_S = 0, T_IN = 128, T_OUT = 128 + D, T_A = 128 + 2 * D, COLUMNS = 512;
  constexpr uint32_t id_s = idesc_bf16_f32(128, 128, false, false);
  constexpr uint32_t id_in = idesc_bf16_f32(128, D, false, false);
  constexpr uint32_t id_out = idesc_bf16_f32(128, D, false, true);
  constexpr uint32_t id_kv = idesc_bf16_f32(128, D, true, true);
  constexpr int N = D / PARTS;
  // NM = 3: Q K^T as well, in the scores' share's place or behind everything.
  constexpr uint32_t T_P = D == 128 ? T_OUT : 384;
  // the parts' sums of a row
  constexpr uint32_t LOW = SM::OFF_EXTRA;  // of phi(k)
  constexpr uint32_t T_MORE = T_A + 64, T_CROSS = T_MORE + 8;
  static_assert(T_CROSS + 32 <= (D == 128 ? COLUMNS : T_P), "tensor memory");
  extern __shared__ __align__(1024) unsigned char smem[];
  Block b;
  b.start(smem, SM::OFF_BAR, COLUMNS, err);
  float2 *lam = reinterpret_cast<float2 *>(smem + SM::OFF_LAM);
  float *fac = reinterpret_cast<float *>(smem + SM::OFF_FAC);
  float *sums = reinterpret_cast<float *>(smem + SM::OFF_MORE);  // of warps
  const int seq = blockIdx.x / p.segments, seg = blockIdx.x % p.segments;
  const int c0 = seg * p.per, c1 = min(c0 + p.per, p.chunks);
  const size_t es = (size_t)p.n_k * p.n_v;
  const bool shares = NM == 3 && DECAY && p.rq;  // of ddecay
  auto stage = [&](int c) { return TWO ? (c - c0) & 1 : 0; };
  auto tile = [&](int c, int i) {  // k, v, dO, q
    return SM::OFF_TILES + stage(c) * SM::STAGE + i * SM::TILE;
  };
  // A chunk's tiles: all into the set that the last chunk had, or, with one set, each as soon as
  // the last one's place is free; then into L2 a chunk earlier: all blocks load at about
  // the same time, and DRAM would make them wait.
  auto load_dO = [&](int c) {
    mbar_arrive_expect_tx(&b.full[stage(c)], (HAS_Q ? 4 : 3) * SM::TILE);
    load_tile_tma<D>(b, tile(c, 2), &maps.dO, &b.full[stage(c)], c * CT, seq);
  };
  auto load_k = [&](int c) {
    load_tile_tma<D>(b, tile(c, 0), &maps.k, &b.full[stage(c)], c * CT, seq);
  };
  auto load_vq = [&](int c) {
    load_tile_tma<D>(b, tile(c, 1), &maps.v, &b.full[stage(c)], c * CT, seq);
    if (HAS_Q) load_tile_tma<D>(b, tile(c, 3), &maps.q, &b.full[stage(c)], c * CT, seq);
  };
  auto prefetch = [&](int c) {
    prefetch_tile<D>(&maps.dO, c * CT, seq, p.n_v);
    prefetch_tile<D>(&maps.k, c * CT, seq, p.n_k);
    prefetch_tile<D>(&maps.v, c * CT, seq, p.n_v);
    if (HAS_Q) prefetch_tile<D>(&maps.q, c * CT, seq, p.n_k);
  };
  if (threadIdx.x == kLeaderQ) {
    load_dO(c0);
    load_k(c0);
    load_vq(c0);
  }
  TokenDecay next;
  next.load(p, b, seq, c0);
  StateRow<D, NM, SPLIT> state;
  state.load(seg ? p.U + ((size_t)seq * (p.segments - 1) + seg - 1) * es
                 : p.S0 ? p.S0 + (size_t)seq * es : nullptr, b, p);
  state.planes(b);
  float around = 0.f;
  int c = c0;
  for (; c < c1; ++c) {
    const int t0 = c * CT, t = t0 + b.row;
    const uint32_t phase = (c - c0) & 1;
    const uint32_t TK = tile(c, 0), TV = tile(c, 1), TD = tile(c, 2), TQ = tile(c, 3);
    const bool more = c + 1 < c1;
    if (DECAY && b.part == 0) {
      next.put<false>(b, lam, fac);
      if (more) next.load(p, b, seq, c + 1);
    }
    const bool keep = NM == 3 && DECAY && p.keeps(seq, c, c1);
    b.wait_full(stage(c), TWO ? (c - c0) >> 1 & 1 : phase);
    if (PHI) map_tile_tc<D, true>(smem + TK, smem + TK, smem + LOW, p.L - t0, p.n_k);
    fence_proxy_async_smem();
    tc_fence_before();
    if (__syncthreads_or(b.failed)) break;
    if (threadIdx.x == kLeaderQ) {
      tc_fence_after();
      const Operand a = along_row<SM::BOX>(b.base + TD);
      product<D>(b.tmem + T_S, a, along_row<SM::BOX>(b.base + TV), id_s, false);
      if (shares)
        product<D>(b.tmem + T_P, along_row<SM::BOX>(b.base + TQ), along_row<SM::BOX>(b.base + TK),
                   id_s, false);
      mma_commit(&b.mma[0]);
#pragma unroll
      for (int m = NS - 1; m >= 0; --m)
        product<D>(b.tmem + T_IN, a, along_row<ST::BOX>(b.base + m * ST::PLANE), id_in,
                   m < NS - 1);
      mma_commit(&b.mma[1]);
      if (more && TWO) {
        tma_store_wait_read_all();  // the last chunk's dq
        load_dO(c + 1);
        load_k(c + 1);
        load_vq(c + 1);
      } else if (more) {
        prefetch(c + 1);
      }
    }
    const float2 own = DECAY ? lam[b.row] : make_float2(0.f, 0.f);
    const float2 end = DECAY ? lam[CT - 1] : make_float2(0.f, 0.f);
    const float2 all = exp2_two(end);
    if (keep) state.keep(p.kept + p.keep_slot(seq, c) * (D * D), b);
    b.wait_mma(0, phase);
    // the scores as operand: row j, tokens i <= j
    float pairs = 0.f;  // with tokens of the blocks before
    {
      const int block = b.part;
      const bool diagonal = block == b.quarter;
      uint32_t w[16];
      if (block > b.quarter) {  // all behind the warp's rows
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = 0;
      } else {
        RowDecay decay;
        if (DECAY) decay.start<false>(b, block, lam, fac, own);
        float run = 0.f;
#pragma unroll
        for (int y = 0; y < 32; y += 16) {
          float f[16], d[16];
          load_16(b, T_S + block * 32 + y, f);
          if (DECAY) decay.get(y, d);
          if (shares) {
            float g[16];
            load_16(b, T_P + block * 32 + y, g);
#pragma unroll
            for (int e = 0; e < 16; ++e) g[e] *= d[e] * f[e];
            if (diagonal) {
              // Row j's pairs with the tokens in front of t, for the t that are not behind it: added
              // over the rows they are the pairs i < t <= j, while the state's update runs.
              uint32_t r[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                r[e] = __float_as_uint(y + e <= b.lane ? run : 0.f);
                run += g[e];
              }
              tmem_st16(b.at(T_CROSS + y), r);
            } else {
              float s[2] = {0.f, 0.f};
#pragma unroll
              for (int e = 0; e < 16; ++e) s[e % 2] += g[e];
              pairs += s[0] + s[1];
            }
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if (DECAY) f[e] *= d[e];
            if (diagonal) f[e] = y + e <= b.lane ? f[e] : 0.f;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) w[y / 2 + e] = la::pack_bf16(f[2 * e], f[2 * e + 1]);
        }
      }
      tmem_st16(b.at(T_A + block * 16), w);
    }
    tmem_st_wait();
    tc_fence_before();
    __syncthreads();
    const Operand k = along_col<SM::BOX>(b.base + TK), v = along_col<SM::BOX>(b.base + TV);
    const Operand k_low = along_col<SM::BOX>(b.base + LOW);
    if (threadIdx.x == kLeaderQ) {  // the scores' share, while the decayed K is formed
      tc_fence_after();
      if (PHI) product_ta<CT>(b.tmem + T_OUT, b.tmem + T_A, k_low, id_out, false);
      product_ta<CT>(b.tmem + T_OUT, b.tmem + T_A, k, id_out, PHI);
      mma_commit(&b.mma[2]);
    }
    b.wait_mma(1, phase);  // the state's planes and dO are read
    if (threadIdx.x == kLeaderQ && more && !TWO) load_dO(c + 1);
    __syncwarp();
    if (more) {
      if (DECAY) {
        decayed_rows<D, NM, CT, PHI>(smem + TK, smem + LOW, smem, 0,
                                     [&](int i) { return decay_between(end, lam[i]); });
        fence_proxy_async_smem();
        __syncthreads();
      }
      if (threadIdx.x == kLeaderQ) {  // the state's update, while dq leaves
        tc_fence_after();
        if (DECAY) {
#pragma unroll
          for (int m = NM - 1; m >= 0; --m)
            product<CT>(b.tmem + T_S, along_col<SM::BOX>(b.base + m * SM::TILE), v, id_kv,
                        m < NM - 1);
        } else {
          constexpr bool BOTH = PHI && !SPLIT;
          if (BOTH) product<CT>(b.tmem + T_S, k_low, v, id_kv, false);
          product<CT>(b.tmem + T_S, SPLIT ? along_cols(b.base + TK, b.base + LOW) : k, v, id_kv, BOTH);
        }
        mma_commit(&b.mma[3]);
      }
    }
    b.wait_mma(2, phase);
    if (threadIdx.x == kLeaderQ && more && DECAY && !TWO) load_k(c + 1);
    __syncwarp();
    const float head = ex2_approx(own.x);
    float dot = 0.f;
#pragma unroll
    for (int x = 0; x < N; x += 16) {
      float f[16], g[16];
      load_16(b, T_IN + b.part * N + x, f);
      load_16(b, T_OUT + b.part * N + x, g);
#pragma unroll
      for (int e = 0; e < 16; ++e) f[e] *= head;
#pragma unroll
      for (int e = 0; e < 16; ++e) g[e] += f[e];
#pragma unroll
      for (int e = 0; e < 16; e += 8) {
        uint4 *cell = b.cell(TQ, b.part * N + x + e);
        if (shares) dot = dot_8(*cell, f + e, dot);
        stage_8<PHI>(cell, cell, g + e);
      }
    }
    if (shares) {
      b.leave(T_MORE, dot, pairs);
      if (b.quarter >= b.part + 2) {  // pairs of blocks with others between them
        float s = pairs;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        if (b.lane == 0) sums[b.quarter - 2 + b.part] = s;  // 2 and 0, 3 and 0, 3 and 1
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == kLeaderQ) {
      store_tile_tma<D>(b, TQ, &maps.dq, t0, seq, p.n_k);
      tma_store_commit();
    }
    if (shares && b.part == 0) b.gather(T_MORE, dot, pairs);
    if (shares) {
      const size_t to = (size_t)seq * p.L + t;
      if (b.part == 0 && t < p.L) p.rq[to] = dot, p.cs[to] = pairs;
      if (b.part == b.quarter) {  // who has the diagonal: lane t of 32 sums over the rows
        float f[16], g[16];
        load_16(b, T_CROSS, f);
        load_16(b, T_CROSS + 16, g);
        const float x = lanes_of_2(lanes_of_16(f, b.lane), lanes_of_16(g, b.lane), b.lane);
        if (t < p.L) p.rc[to] = x;
      }
      if (threadIdx.x == 0)
        p.across[(size_t)seq * p.chunks + c] = make_float2(sums[0] + sums[1], sums[1] + sums[2]);
    }
    if (more) {
      b.wait_mma(3, phase);
      if (threadIdx.x == kLeaderQ && !TWO) {
        tma_store_wait_read_all();  // the fourth tile
        if (!DECAY) load_k(c + 1);
        load_vq(c + 1);
      }
      __syncwarp();
      state.update(b, T_S, all);
      state.planes(b);
    } else if (shares) {  // <G, e^L_C S>: the pairs around the segment's last chunk
      const float *G = seg + 1 < p.segments ? p.W + ((size_t)seq * (p.segments - 1) + seg) * es
                       : p.dSf ? p.dSf + (size_t)seq * es : nullptr;
      if (G) around = state.dot(G, b, p) * all.x;
    }
  }
  if (threadIdx.x == kLeaderQ) {
    if (c < c1) tc::drain_wait(&b.full[stage(c)], (TWO ? (c - c0) >> 1 : c - c0) & 1);
    tma_store_wait_all();
  }
  if (shares) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) around += __shfl_xor_sync(0xffffffffu, around, off);
    __syncthreads();
    if (b.lane == 0) sums[b.warp] = around;
    __syncthreads();
    if (threadIdx.x == kLeaderQ) {
      float s = 0.f;
      for (int i = 0; i < kThreads / 32; ++i) s += sums[i];
      p.around[(size_t)seq * p.segments + seg] = s;
    }
  }
  b.finish(COLUMNS);
}

// ---------------------------------------------------------------- dk and dv
template <int D, int NM, bool PHI> constexpr bool kv_own_tiles() {
  return D == 64 || (NM == 1 && !PHI);
}
template <int D, int NM, bool PHI> constexpr int kv_tiles() {
  return 4 * kStages<D> + 2 * PHI + (kv_own_tiles<D, NM, PHI>() ? 2 : 0);
}
template <int D, int NM, bool PHI, bool DECAY>
__global__ void __launch_bounds__(kThreads, 1)
grad_kv_tc_kernel(const __grid_constant__ Maps maps, const ChunkBwd p, unsigned int *err) {
  // A tile of its own holds phi(k) beside k, which its derivative needs, and another phi(q)'s low part
  // (phi(k)'s would enter dv alone, where its rounding averages out).  dk and dv leave by
  // tiles of their own; where there is no room for them, by k's and v's, which then load
  // late (through the state's planes instead they kept these waiting: 256 us against 238).
  using SM = Smem<D, NM, kv_tiles<D, NM, PHI>(), 1>;
  using ST = StateTile<D>;
  constexpr bool TWO = kStages<D> == 2, OWN = kv_own_tiles<D, NM, PHI>(), EARLY_K = OWN && !PHI;
  constexpr bool SPLIT = kSplit<D, PHI, DECAY>;
  constexpr int NS = SPLIT ? 2 : NM;  // planes of the state
  // Tensor memory: K Q^T and V dO^T, dv, dk.  When the scores have been read their operands
  // take columns 0..63 and 192..255, the state's update those between.
  constexpr uint32_t T_P = 0, T_DP = 128, T_V = 256, T_K = 256 + D, COLUMNS = 512;
  constexpr uint32_t T_AP = 0, T_ADP = 192, T_U = 64;
  constexpr uint32_t id_s = idesc_bf16_f32(128, 128, false, false);
  constexpr uint32_t id_in = idesc_bf16_f32(128, D, false, false);
  constexpr uint32_t id_out = idesc_bf16_f32(128, D, false, true);
  constexpr uint32_t id_kv = idesc_bf16_f32(128, D, true, true);
  constexpr int N = D / PARTS;
  extern __shared__ __align__(1024) unsigned char smem[];
  Block b;
  b.start(smem, SM::OFF_BAR, COLUMNS, err);
  float2 *lam = reinterpret_cast<float2 *>(smem + SM::OFF_LAM);
  float *fac = reinterpret_cast<float *>(smem + SM::OFF_FAC);
  const int seq = blockIdx.x / p.segments, seg = blockIdx.x % p.segments;
  const int c0 = seg * p.per, c1 = min(c0 + p.per, p.chunks), n = c1 - c0;
  const size_t es = (size_t)p.n_k * p.n_v;
  const bool shares = NM == 3 && DECAY && p.rk;  // of ddecay
  constexpr uint32_t MORE = SM::OFF_TILES + 4 * kStages<D> * SM::TILE;
  constexpr uint32_t LOW = MORE + SM::TILE, OUT = MORE + 2 * PHI * SM::TILE;
  auto stage = [&](int c) { return TWO ? (c1 - 1 - c) & 1 : 0; };
  auto tile = [&](int c, int i) {  // q, k, v, dO
    return SM::OFF_TILES + (stage(c) * 4 + i) * SM::TILE;
  };
  auto load = [&](int c, int i, const CUtensorMap *map) {
    load_tile_tma<D>(b, tile(c, i), map, &b.full[stage(c)], c * CT, seq);
  };
  auto arm = [&](int c) { mbar_arrive_expect_tx(&b.full[stage(c)], 4 * SM::TILE); };
  auto load_q = [&](int c) { load(c, 0, &maps.q); };
  auto load_k = [&](int c) { load(c, 1, &maps.k); };
  auto load_v = [&](int c) { load(c, 2, &maps.v); };
  auto load_dO = [&](int c) { load(c, 3, &maps.dO); };
  auto prefetch = [&](int c) {
    prefetch_tile<D>(&maps.q, c * CT, seq, p.n_k);
    prefetch_tile<D>(&maps.k, c * CT, seq, p.n_k);
    prefetch_tile<D>(&maps.v, c * CT, seq, p.n_v);
    prefetch_tile<D>(&maps.dO, c * CT, seq, p.n_v);
  };
  if (threadIdx.x == kLeaderKV) {
    arm(c1 - 1);
    load_q(c1 - 1);
    load_k(c1 - 1);
    load_v(c1 - 1);
    load_dO(c1 - 1);
  }
  TokenDecay next;
  next.load(p, b, seq, c1 - 1);
  StateRow<D, NM, SPLIT> state;
  state.load(seg + 1 < p.segments ? p.W + ((size_t)seq * (p.segments - 1) + seg) * es
             : p.dSf ? p.dSf + (size_t)seq * es : nullptr, b, p);
  state.planes(b);
  int done = 0;
  for (; done < n; ++done) {
    const int c = c1 - 1 - done, t0 = c * CT, t = t0 + b.row;
    const uint32_t phase = done & 1;
    const uint32_t TQ = tile(c, 0), TK = tile(c, 1), TV = tile(c, 2), TD = tile(c, 3);
    const uint32_t TKP = PHI ? MORE : TK, TDV = OWN ? OUT : TV, TDK = OWN ? OUT + SM::TILE : TK;
    const bool more = done + 1 < n, update = more || (p.dS0 && seg == 0);
    if (DECAY && b.part == 0) {
      next.put<true>(b, lam, fac);
      if (more) next.load(p, b, seq, c - 1);
    }
    const bool keep = NM == 3 && DECAY && p.keeps(seq, c, c1);
    b.wait_full(stage(c), TWO ? done >> 1 & 1 : phase);
    if (PHI) {
      map_tile_tc<D, true>(smem + TQ, smem + TQ, smem + LOW, p.L - t0, p.n_k);
      map_tile_tc<D, false>(smem + TK, smem + TKP, nullptr, p.L - t0, p.n_k);
    }
    if (OWN && threadIdx.x == kLeaderKV) tma_store_wait_read_all();
    fence_proxy_async_smem();
    tc_fence_before();
    if (__syncthreads_or(b.failed)) break;
    if (threadIdx.x == kLeaderKV) {
      tc_fence_after();
      const Operand ak = along_row<SM::BOX>(b.base + TKP), av = along_row<SM::BOX>(b.base + TV);
      product<D>(b.tmem + T_P, ak, along_row<SM::BOX>(b.base + TQ), id_s, false);
      product<D>(b.tmem + T_DP, av, along_row<SM::BOX>(b.base + TD), id_s, false);
      mma_commit(&b.mma[0]);
      product<D>(b.tmem + T_V, ak, along_col<ST::BOX>(b.base), id_out, false);
#pragma unroll
      for (int m = NS - 1; m >= 0; --m)
        product<D>(b.tmem + T_K, av, along_row<ST::BOX>(b.base + m * ST::PLANE), id_in,
                   m < NS - 1);
      mma_commit(&b.mma[1]);
      if (more && TWO) {
        arm(c - 1);
        load_q(c - 1);
        load_k(c - 1);
        load_v(c - 1);
        load_dO(c - 1);
      } else if (more) {
        prefetch(c - 1);
      }
    }
    const float2 own = DECAY ? lam[b.row] : make_float2(0.f, 0.f);
    const float2 end = DECAY ? lam[CT - 1] : make_float2(0.f, 0.f);
    const float2 all = exp2_two(end);
    if (keep) {
      float s = state.dot_kept(p.kept + p.keep_slot(seq, c) * (D * D), b);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      float *to = p.between + p.keep_slot(seq, c) * kShares;
      if (b.lane == 0)
        for (int i = b.warp; i < kShares; i += kThreads / 32)
          to[i] = i == b.warp ? s * all.x : 0.f;
    }
    b.wait_mma(0, phase);
    // the scores as operands: row i, tokens j >= i
    uint32_t wp[16], wd[16];
    float pairs = 0.f;  // with tokens of the blocks behind
    const int block = b.part;
    const bool diagonal = block == b.quarter;
    if (block < b.quarter) {  // all in front of the warp's rows
#pragma unroll
      for (int e = 0; e < 16; ++e) wp[e] = wd[e] = 0;
    } else {
      RowDecay decay;
      if (DECAY) decay.start<true>(b, block, lam, fac, own);
#pragma unroll
      for (int y = 0; y < 32; y += 16) {
        float f[16], g[16], d[16];
        load_16(b, T_P + block * 32 + y, f);
        load_16(b, T_DP + block * 32 + y, g);
        if (DECAY) decay.get(y, d);
        if (shares && !diagonal) {
          float s[2] = {0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 16; ++e) s[e % 2] += f[e] * d[e] * g[e];
          pairs += s[0] + s[1];
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (DECAY) f[e] *= d[e], g[e] *= d[e];
          if (diagonal) {
            f[e] = y + e >= b.lane ? f[e] : 0.f;
            g[e] = y + e >= b.lane ? g[e] : 0.f;
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          wp[y / 2 + e] = la::pack_bf16(f[2 * e], f[2 * e + 1]);
          wd[y / 2 + e] = la::pack_bf16(g[2 * e], g[2 * e + 1]);
        }
      }
    }
    tc_fence_before();
    __syncthreads();  // the scores are read: their operands may take their place
    tc_fence_after();
    tmem_st16(b.at(T_AP + block * 16), wp);
    tmem_st16(b.at(T_ADP + block * 16), wd);
    b.wait_mma(1, phase);
    const float tail = decay_between(end, own);
    float dot = 0.f;
    if (DECAY) {  // the state's share, by each token's decay to the chunk's end
#pragma unroll
      for (int x = 0; x < 2 * N; x += 16) {
        const bool of_k = x >= N;
        const int col = b.part * N + x % N;
        uint32_t r[16];
        float f[16];
        load_16(b, (of_k ? T_K : T_V) + col, f);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          f[e] *= tail;
          r[e] = __float_as_uint(f[e]);
        }
        tmem_st16(b.at((of_k ? T_K : T_V) + col), r);
        if (shares && of_k) {
#pragma unroll
          for (int e = 0; e < 16; e += 8) dot = dot_8(*b.cell(TK, col + e), f + e, dot);
        }
      }
    }
    if (shares) b.leave(T_U, dot, pairs);
    tmem_st_wait();
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    const Operand q = along_col<SM::BOX>(b.base + TQ), dO = along_col<SM::BOX>(b.base + TD);
    const Operand q_low = along_col<SM::BOX>(b.base + LOW);
    if (threadIdx.x == kLeaderKV) {  // the scores' share, while the decayed Q is formed
      tc_fence_after();
      product_ta<CT>(b.tmem + T_V, b.tmem + T_AP, dO, id_out, true);
      if (PHI) product_ta<CT>(b.tmem + T_K, b.tmem + T_ADP, q_low, id_out, true);
      product_ta<CT>(b.tmem + T_K, b.tmem + T_ADP, q, id_out, true);
      mma_commit(&b.mma[2]);
      if (more && !TWO) {
        arm(c - 1);
        if (OWN) load_v(c - 1);
        if (EARLY_K) load_k(c - 1);
      }
    }
    if (shares && b.part == 0) b.gather(T_U, dot, pairs);
    if (shares && t < p.L) {
      const size_t to = (size_t)seq * p.L + t;
      if (b.part == 0) p.rk[to] = dot, p.rs[to] = pairs;
    }
    if (update && DECAY) {
      decayed_rows<D, NM, CT, PHI>(smem + TQ, smem + LOW, smem, 0,
                                   [&](int i) { return ex2_approx(lam[i].x); });
      fence_proxy_async_smem();
    }
    tc_fence_before();
    if (DECAY) __syncthreads();
    if (threadIdx.x == kLeaderKV && update) {  // the state's update, while dk and dv leave
      tc_fence_after();
      if (DECAY) {
#pragma unroll
        for (int m = NM - 1; m >= 0; --m)
          product<CT>(b.tmem + T_U, along_col<SM::BOX>(b.base + m * SM::TILE), dO, id_kv,
                      m < NM - 1);
      } else {
        constexpr bool BOTH = PHI && !SPLIT;
        if (BOTH) product<CT>(b.tmem + T_U, q_low, dO, id_kv, false);
        product<CT>(b.tmem + T_U, SPLIT ? along_cols(b.base + TQ, b.base + LOW) : q, dO, id_kv, BOTH);
      }
      mma_commit(&b.mma[3]);
    }
    b.wait_mma(2, phase);
    if (threadIdx.x == kLeaderKV && more && DECAY && !TWO) load_q(c - 1);
    __syncwarp();
#pragma unroll
    for (int x = 0; x < N; x += 16) {
      const int col = b.part * N + x;
      float f[16];
      load_16(b, T_V + col, f);
#pragma unroll
      for (int e = 0; e < 16; e += 8) stage_8<false>(b.cell(TDV, col + e), nullptr, f + e);
      load_16(b, T_K + col, f);
#pragma unroll
      for (int e = 0; e < 16; e += 8)
        stage_8<PHI>(b.cell(TDK, col + e), b.cell(TK, col + e), f + e);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == kLeaderKV) {
      store_tile_tma<D>(b, TDV, &maps.dv, t0, seq, p.n_v);
      store_tile_tma<D>(b, TDK, &maps.dk, t0, seq, p.n_k);
      tma_store_commit();
      if (OWN && !EARLY_K && more && !TWO) load_k(c - 1);
    }
    if (update) {
      b.wait_mma(3, phase);
      if (threadIdx.x == kLeaderKV && more && !TWO) {
        if (!DECAY) load_q(c - 1);
        load_dO(c - 1);
        if (!OWN) {
          tma_store_wait_read_all();
          load_k(c - 1);
          load_v(c - 1);
        }
      }
      __syncwarp();
      state.update(b, T_U, all);
      if (more) state.planes(b);
    }
  }
  if (done == n) {
    if (p.dS0 && seg == 0) state.store(p.dS0 + (size_t)seq * es, b, p);
  } else if (threadIdx.x == kLeaderKV) {
    tc::drain_wait(&b.full[stage(c1 - 1 - done)], (TWO ? done >> 1 : done) & 1);
  }
  if (threadIdx.x == kLeaderKV) tma_store_wait_all();
  b.finish(COLUMNS);
}

template <int D, int NM, bool PHI, bool DECAY>
cudaError_t launch_tc(const ChunkBwd &p, int seqs, cudaStream_t stream) {
  using SS = ShareSmem<D, NM, PHI, DECAY>;
  using SQ = Smem<D, NM, 4, kStages<D>, PHI>;
  using SK = Smem<D, NM, kv_tiles<D, NM, PHI>(), 1>;
  Maps m;
  const struct {
    CUtensorMap *map;
    const void *p;
    int width;
  } all[] = {{&m.q, p.q, p.n_k},   {&m.k, p.k, p.n_k},   {&m.v, p.v, p.n_v},  {&m.dO, p.dO, p.n_v},
             {&m.dq, p.dq, p.n_k}, {&m.dk, p.dk, p.n_k}, {&m.dv, p.dv, p.n_v}};
  for (const auto &x : all)
    if (!make_tmap_bf16_3d(x.map, x.p, x.width, p.L, seqs, 64, CT)) return cudaErrorInvalidValue;
  unsigned int *err = device_error_word();
  cudaError_t e;
  if (p.segments > 1) {
    auto share = segment_share_tc_kernel<D, NM, PHI, DECAY>;
    static int set[64];
    if ((e = tc::set_smem_once(share, SS::BYTES, set)) != cudaSuccess) return e;
    share<<<dim3((unsigned)(seqs * (p.segments - 1)), 2), kThreads, SS::BYTES, stream>>>(m, p, err);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_segment_scan(p, seqs, stream)) != cudaSuccess) return e;
  }
  auto gq = grad_q_tc_kernel<D, NM, PHI, DECAY>;
  auto gkv = grad_kv_tc_kernel<D, NM, PHI, DECAY>;
  static int set_q[64], set_kv[64];
  if ((e = tc::set_smem_once(gq, SQ::BYTES, set_q)) != cudaSuccess) return e;
  if ((e = tc::set_smem_once(gkv, SK::BYTES, set_kv)) != cudaSuccess) return e;
  gq<<<seqs * p.segments, kThreads, SQ::BYTES, stream>>>(m, p, err);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  gkv<<<seqs * p.segments, kThreads, SK::BYTES, stream>>>(m, p, err);
  return cudaGetLastError();
}

template <int D, bool DECAY>
cudaError_t launch_d(const ChunkBwd &p, int seqs, bool planes, cudaStream_t stream) {
  if (planes) return launch_tc<D, 3, false, DECAY>(p, seqs, stream);
  return p.phi == LA_PHI_ELU1 ? launch_tc<D, 1, true, DECAY>(p, seqs, stream)
                              : launch_tc<D, 1, false, DECAY>(p, seqs, stream);
}

}  // namespace

cudaError_t launch_chunk_bwd_tc(const ChunkBwd &p, int seqs, bool planes, cudaStream_t stream) {
  if (std::max(p.n_k, p.n_v) > 64)
    return p.decay_kind != LA_DECAY_NONE ? launch_d<128, true>(p, seqs, planes, stream)
                                         : launch_d<128, false>(p, seqs, planes, stream);
  return p.decay_kind != LA_DECAY_NONE ? launch_d<64, true>(p, seqs, planes, stream)
                                       : launch_d<64, false>(p, seqs, planes, stream);
}

}  // namespace la
