// la_block_norm.cu -- the norms around a block: the gated norm of a layer's
// heads on their way to the output projection, and the residual step between
// two blocks (post norm, residual scale, addition, next block's norm).
//
// Both are streams over their inputs and outputs with one or two reductions
// per row, held in fp32: a row's mean first, then the mean square about it.  A
// team of threads takes a row and keeps it in registers, so every input is read
// once: 2 to 32 lanes of a warp (rows up to 1024 wide, several to a warp) or
// a whole block.
//
// The residual step reads as many bytes of parameters as of data where the
// residual is fp32, so its teams take many rows, keep the factors of x in
// registers and load the next row meanwhile: 16384 x 4096 at 6.4 TB/s (94% of
// the measured copy).  The gated norm's teams take one row each: the same loop
// cost it more registers than it gave (4 x 16 x 4096 x 64 bf16: 23 us, 4.3 TB/s,
// against 25 to 29; 2 x 2047 x 4096 fp32: 35.5, 5.7 TB/s, against 37).  Its short
// rows are bound by instructions and latency: index arithmetic and two sums of
// shuffles for 64 values.
#include <cstdint>

#include "../../include/la_gb300.h"
#include "la_act.cuh"
#include "la_internal.h"

namespace la {
namespace {

constexpr int kTeamThreads = 256;  // threads per block of teams inside a warp

// The sum of v over the team: LANES neighbouring lanes, or the block (LANES = 0).
template <int LANES>
__device__ __forceinline__ float team_sum(float v) {
#pragma unroll
  for (int off = (LANES ? LANES : 32) / 2; off > 0; off >>= 1)
    v += __shfl_xor_sync(0xffffffffu, v, off);
  if constexpr (LANES == 0) {
    __shared__ float red[32];
    const int warp = threadIdx.x / 32, warps = blockDim.x / 32;
    __syncthreads();  // red may still be read from the sum before
    if (threadIdx.x % 32 == 0) red[warp] = v;
    __syncthreads();
    v = threadIdx.x % 32 < warps ? red[threadIdx.x % 32] : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  }
  return v;
}

// One row of width d in the team's registers, two values to a register pair:
// thread `lane` of `size` holds the vectors lane, lane + size, ... of V
// elements; places past the row hold 0.
template <int V, int LANES, int I>
struct Row {
  using Cell = CellOf<V>;
  using C = typename Cell::type;
  static constexpr int H = V > 1 ? V / 2 : 1;
  C v[I][H];

  __device__ __forceinline__ void set(int i, const float *f) {
#pragma unroll
    for (int e = 0; e < H; ++e) {
      if constexpr (V == 1) v[i][e] = f[e];
      else v[i][e] = pack2(f[2 * e], f[2 * e + 1]);
    }
  }
  __device__ __forceinline__ void get(int i, float *f) const {
#pragma unroll
    for (int e = 0; e < H; ++e) {
      if constexpr (V == 1) f[e] = v[i][e];
      else unpack2(v[i][e], f[2 * e], f[2 * e + 1]);
    }
  }
  // v <- (v - mean) / sqrt(mean square about it + eps), mean = 0 for RMS.  The
  // first vector starts `shift` places in front of the row (SHIFT; else 0).
  template <bool SHIFT = false>
  __device__ __forceinline__ void normalise(int d, int norm, float eps, int lane, int size,
                                            int shift = 0) {
    const float inv = 1.f / d;
    if (norm == LA_NORM_LAYER) {
      C s = 0;
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int e = 0; e < H; ++e) s = add2(s, v[i][e]);
      const C m = Cell::both(-team_sum<LANES>(Cell::sum(s)) * inv);
#pragma unroll
      for (int i = 0; i < I; ++i) {
        const int c = (lane + i * size) * V - shift;
        if constexpr (SHIFT) {
          float f[V];
#pragma unroll
          for (int e = 0; e < H; ++e) v[i][e] = add2(v[i][e], m);
          get(i, f);
#pragma unroll
          for (int e = 0; e < V; ++e) f[e] = c + e >= 0 && c + e < d ? f[e] : 0.f;
          set(i, f);
        } else {
#pragma unroll
          for (int e = 0; e < H; ++e) v[i][e] = c < d ? add2(v[i][e], m) : C(0);
        }
      }
    }
    C q = 0;
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int e = 0; e < H; ++e) q = fma2(v[i][e], v[i][e], q);
    const C r = Cell::both(rsqrtf(fmaf(team_sum<LANES>(Cell::sum(q)), inv, eps)));
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int e = 0; e < H; ++e) v[i][e] = mul2(v[i][e], r);
  }
};

// V fp32 parameters, 16-byte vectors where V allows them (V = 1, 2, 4 or 8).
template <int V>
__device__ __forceinline__ void load_params(const float *p, float *f) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 u = __ldg(reinterpret_cast<const float4 *>(p + i));
      f[i] = u.x, f[i + 1] = u.y, f[i + 2] = u.z, f[i + 3] = u.w;
    }
  } else if constexpr (V == 2) {
    const float2 u = __ldg(reinterpret_cast<const float2 *>(p));
    f[0] = u.x, f[1] = u.y;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = __ldg(p + i);
  }
}

// Five blocks of teams per SM (48 registers, 8 to 32 bytes of them spilled): 4 x
// 16 x 4096 x 64 takes 23.4 us, with four 23.7, with six 27.
template <typename T, int V, int LANES, int I, int ACT, int MAXT>
__global__ void __launch_bounds__(MAXT, LANES && V > 2 && I <= 2 ? 5 : 1)
gated_norm_kernel(const GatedNormArgs a, long long rows) {
  constexpr int H = Row<V, LANES, I>::H;
  const int size = LANES ? LANES : blockDim.x;
  const int lane = LANES ? threadIdx.x % size : threadIdx.x;
  long long r = LANES ? (long long)blockIdx.x * (kTeamThreads / size) + threadIdx.x / size
                      : (long long)blockIdx.x;
  const bool live = r < rows;
  if (!live) r = rows - 1;  // its lanes take part in the sums
  const long long bt = div_index(r, a.H), b = div_index(bt, a.L);
  const int h = (int)(r - bt * a.H), d = a.d;
  const T *xr = static_cast<const T *>(a.x) + b * a.x_bs + h * a.x_hs + (bt - b * a.L) * a.x_ts;
  const T *gr = static_cast<const T *>(a.gate) + (a.gate ? bt * a.gate_stride : 0) +
                (long long)h * d;
  T *y = static_cast<T *>(a.y) + bt * a.y_stride + (long long)h * d;
  const long long w0 = a.weight_heads > 1 ? (long long)h * d : 0;
  Raw<T, V> x[I], gate[I];
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int c = (lane + i * size) * V;
    x[i] = gate[i] = Raw<T, V>{};
    if (c < d) {
      x[i] = load_raw<T, V>(xr + c);
      if (a.gate) gate[i] = load_raw<T, V>(gr + c);
    }
  }
  Row<V, LANES, I> row, g;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    float f[V];
    x[i].unpack(f);
    row.set(i, f);
    gate[i].unpack(f);
    g.set(i, f);
  }
  if (a.gate) {
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int e = 0; e < H; ++e) g.v[i][e] = activate2(ACT, g.v[i][e]);
    if (a.gate_first) {
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int e = 0; e < H; ++e) row.v[i][e] = mul2(row.v[i][e], g.v[i][e]);
    }
  }
  row.normalise(d, a.norm, a.eps, lane, size);
  if (!live) return;
  const bool gate_last = a.gate && !a.gate_first;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int c = (lane + i * size) * V;
    if (c >= d) continue;
    Row<V, 1, 1> o, f;
    float p[V];
#pragma unroll
    for (int e = 0; e < H; ++e) o.v[0][e] = row.v[i][e];
    if (a.weight) {
      load_params<V>(a.weight + w0 + c, p);
      f.set(0, p);
#pragma unroll
      for (int e = 0; e < H; ++e) o.v[0][e] = mul2(o.v[0][e], f.v[0][e]);
    }
    if (a.bias) {
      load_params<V>(a.bias + w0 + c, p);
      f.set(0, p);
#pragma unroll
      for (int e = 0; e < H; ++e) o.v[0][e] = add2(o.v[0][e], f.v[0][e]);
    }
    if (gate_last) {
#pragma unroll
      for (int e = 0; e < H; ++e) o.v[0][e] = mul2(o.v[0][e], g.v[i][e]);
    }
    float out[V];
    o.get(0, out);
    store_vec<T, V>(y + c, out);
  }
}

// The elements lo <= e < hi of a vector, one by one; the others are 0.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_part(const T *p, int lo, int hi) {
  Raw<T, V> r{};
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (e >= lo && e < hi) {
      if constexpr (V == 1) r.u = p[e];
      else if constexpr (sizeof(T) == 4) r.w[e] = __float_as_uint(p[e]);
      else r.w[e / 2] |= (uint32_t)__bfloat16_as_ushort(p[e]) << (e % 2 * 16);
    }
  return r;
}

// A team takes the rows r, r + step, ...: the loads of its next row are in
// flight while it works on the present one.  The factors of x stay in registers
// for all of a team's rows: read anew for each, the three parameters of an fp32
// residual step are as many bytes as its data.
//
// SHIFT: rows whose width no vector divides start anywhere in a vector, row r
// at its element r D mod V.  A team's vectors then lie on the tensors' 16-byte
// boundaries, from `shift` elements in front of the row on, its first and last
// one read and written element by element; step is a multiple of V, so all rows of
// a team have one shift, and the weights stay in registers as well.
template <typename T, typename R, int V, int LANES, int I, int MAXT, bool SHIFT>
__global__ void __launch_bounds__(MAXT)
residual_norm_kernel(const ResidualNormArgs a) {
  using ThisRow = Row<V, LANES, I>;
  constexpr int H = ThisRow::H, RV = V < Pack16<R>::N ? V : Pack16<R>::N, RN = V / RV;
  const int size = LANES ? LANES : blockDim.x;
  const int lane = LANES ? threadIdx.x % size : threadIdx.x;
  const int teams = LANES ? kTeamThreads / size : 1;
  const long long step = (long long)gridDim.x * teams;
  long long r = (long long)blockIdx.x * teams + (LANES ? threadIdx.x / size : 0);
  const int D = a.D;
  const int shift = SHIFT ? (int)(r % V) * (D % V) % V : 0;
  auto place = [&](int i) { return (lane + i * size) * V - shift; };
  auto whole = [&](int c) { return SHIFT ? c >= 0 && c + V <= D : c < D; };
  auto partly = [&](int c) { return SHIFT && c > -V && c < D; };  // where not whole
  Row<V, LANES, I> s, wt;
  Raw<T, V> x[I];
  Raw<R, RV> res[I][RN];
  auto fetch = [&](long long at) {
    const T *xr = static_cast<const T *>(a.x) + at * D;
    const R *rr = static_cast<const R *>(a.residual) + at * D;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = place(i);
      if (whole(c)) {
        x[i] = load_raw<T, V>(xr + c);
        if (a.residual) {
#pragma unroll
          for (int k = 0; k < RN; ++k) res[i][k] = load_raw<R, RV>(rr + c + k * RV);
        }
      } else if (partly(c)) {
        x[i] = load_part<T, V>(xr + c, -c, D - c);
        if (a.residual) {
#pragma unroll
          for (int k = 0; k < RN; ++k)
            res[i][k] = load_part<R, RV>(rr + c + k * RV, -c - k * RV, D - c - k * RV);
        }
      }
    }
  };
  auto params = [&](const float *p, int i, float *f) {
    const int c = place(i);
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = 0.f;
    if constexpr (SHIFT) {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (c + e >= 0 && c + e < D) f[e] = __ldg(p + c + e);
    } else {
      if (c < D) load_params<V>(p + c, f);
    }
  };
#pragma unroll
  for (int i = 0; i < I; ++i) {
    x[i] = Raw<T, V>{};
#pragma unroll
    for (int k = 0; k < RN; ++k) res[i][k] = Raw<R, RV>{};
  }
  if (r < a.rows) fetch(r);
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int c = place(i);
    float f[V], g[V];
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = c + e >= 0 && c + e < D ? a.alpha : 0.f;
    if (a.scale) {
      params(a.scale, i, g);
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] *= g[e];
    }
    if (a.post_weight) {
      params(a.post_weight, i, g);
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] *= g[e];
    }
    s.set(i, f);
    if (SHIFT && a.weight) {
      params(a.weight, i, f);
      wt.set(i, f);
    }
  }
  // A team out of rows stays while another of its warp has one: the sums need
  // the whole warp.
  for (long long first = r - (LANES ? threadIdx.x % 32 / size : 0); first < a.rows;
       first += step, r += step) {
    const bool live = r < a.rows;
    ThisRow row, rs;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      float f[V];
      x[i].unpack(f);
      row.set(i, f);
#pragma unroll
      for (int k = 0; k < RN; ++k) res[i][k].unpack(f + k * RV);
      rs.set(i, f);
    }
    if (r + step < a.rows) fetch(r + step);
    if (a.post_weight) row.template normalise<SHIFT>(D, a.norm, a.eps, lane, size, shift);
    R *out = static_cast<R *>(a.residual_out) + r * D;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = place(i);
      if (!whole(c) && !partly(c)) continue;
#pragma unroll
      for (int e = 0; e < H; ++e) row.v[i][e] = fma2(s.v[i][e], row.v[i][e], rs.v[i][e]);
      if (live && a.residual_out) {
        float f[V];
        row.get(i, f);
        if (whole(c)) {
#pragma unroll
          for (int k = 0; k < RN; ++k) store_vec<R, RV>(out + c + k * RV, f + k * RV);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e)
            if (c + e >= 0 && c + e < D) out[c + e] = from_f32<R>(f[e]);
        }
      }
    }
    row.template normalise<SHIFT>(D, a.norm, a.eps, lane, size, shift);
    T *y = static_cast<T *>(a.y) + r * D;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = place(i);
      if ((!whole(c) && !partly(c)) || !live) continue;
      Row<V, 1, 1> p;
      float f[V];
      if (a.weight) {
        if constexpr (SHIFT) {
#pragma unroll
          for (int e = 0; e < H; ++e) row.v[i][e] = mul2(row.v[i][e], wt.v[i][e]);
        } else {
          params(a.weight, i, f);
          p.set(0, f);
#pragma unroll
          for (int e = 0; e < H; ++e) row.v[i][e] = mul2(row.v[i][e], p.v[0][e]);
        }
      }
      if (a.bias) {
        params(a.bias, i, f);
        p.set(0, f);
#pragma unroll
        for (int e = 0; e < H; ++e) row.v[i][e] = add2(row.v[i][e], p.v[0][e]);
      }
      row.get(i, f);
      if (whole(c)) {
        store_vec<T, V>(y + c, f);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (c + e >= 0 && c + e < D) y[c + e] = from_f32<T>(f[e]);
      }
    }
  }
}

// Calls f(Int<LANES>, Int<I>, threads per row) with the team for rows of
// width d in vectors of V elements: as few lanes as hold the row in two vectors
// each, up to a warp; then (FOUR) a warp with four, up to a width of 1024; then a
// block whose threads hold kBlockVecs<V> vectors.  The residual step has no
// registers for four: 16384 x 1024 bf16 with a bf16 residual takes 27.2 us with
// them, 24.4 in blocks (fp32 residual: 35.1 and 32.8).  Its blocks of more than
// 512 threads (rows above 8192) have 64 registers a thread and spill 216 to 426
// bytes: 2000 x 15001 fp32 takes 124 us, 1.8 times its bytes.
template <int V> constexpr int kBlockVecs = V == 8 ? 2 : V == 4 ? 4 : V == 2 ? 8 : 16;
template <int N> struct Int { static constexpr int value = N; };

template <int V, bool FOUR, typename F>
cudaError_t with_team(int d, F f) {
  const int vecs = (d + V - 1) / V;
  if constexpr (V > 2) {
    if (vecs <= 4) return f(Int<2>{}, Int<2>{}, 2);
    if (vecs <= 8) return f(Int<4>{}, Int<2>{}, 4);
    if (vecs <= 16) return f(Int<8>{}, Int<2>{}, 8);
    if (vecs <= 32) return f(Int<16>{}, Int<2>{}, 16);
    if (vecs <= 64) return f(Int<32>{}, Int<2>{}, 32);
    if constexpr (FOUR) {
      if (vecs <= 128) return f(Int<32>{}, Int<4>{}, 32);
    }
  } else {
    if (vecs <= 128) return f(Int<32>{}, Int<4>{}, 32);
    if (vecs <= 1024 / V) return f(Int<32>{}, Int<32 / V>{}, 32);
  }
  const int per = kBlockVecs<V>;
  const int threads = ((vecs + per - 1) / per + 31) / 32 * 32;
  return f(Int<0>{}, Int<kBlockVecs<V>>{}, threads);
}

template <typename T, int V, int ACT>
cudaError_t launch_gated_v(const GatedNormArgs &a) {
  const long long rows = (long long)a.B * a.L * a.H;
  return with_team<V, true>(a.d, [&](auto lanes, auto items, int threads) {
    constexpr int LANES = decltype(lanes)::value, I = decltype(items)::value;
    const int block = LANES ? kTeamThreads : threads;
    const long long per = LANES ? kTeamThreads / LANES : 1, blocks = (rows + per - 1) / per;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    const unsigned grid = (unsigned)blocks;
    if constexpr (LANES != 0)
      gated_norm_kernel<T, V, LANES, I, ACT, kTeamThreads><<<grid, block, 0, a.stream>>>(a, rows);
    else if (threads <= 512)
      gated_norm_kernel<T, V, 0, I, ACT, 512><<<grid, block, 0, a.stream>>>(a, rows);
    else
      gated_norm_kernel<T, V, 0, I, ACT, 1024><<<grid, block, 0, a.stream>>>(a, rows);
    return cudaGetLastError();
  });
}

template <typename T, typename R, int V, bool SHIFT>
cudaError_t launch_residual_v(const ResidualNormArgs &a) {
  return with_team<V, false>(a.D + (SHIFT ? V - 1 : 0), [&](auto lanes, auto items, int threads) {
    constexpr int LANES = decltype(lanes)::value, I = decltype(items)::value;
    const int block = LANES ? kTeamThreads : threads;
    // 512 threads an SM: 16384 x 4096 (fp32 residual, post norm, scale) takes 126
    // us, with 768 or 1024 threads 133 to 154, in blocks that end with their row 144.
    // A multiple of 8 blocks where a team takes more than one row.
    const long long per = LANES ? kTeamThreads / LANES : 1, blocks = (a.rows + per - 1) / per;
    const long long fill = 152ll * (block < 512 ? 512 / block : 1);
    const unsigned grid = (unsigned)(blocks < fill ? blocks : fill);
    if constexpr (LANES != 0)
      residual_norm_kernel<T, R, V, LANES, I, kTeamThreads, SHIFT><<<grid, block, 0, a.stream>>>(a);
    else if (threads <= 512)
      residual_norm_kernel<T, R, V, 0, I, 512, SHIFT><<<grid, block, 0, a.stream>>>(a);
    else
      residual_norm_kernel<T, R, V, 0, I, 1024, SHIFT><<<grid, block, 0, a.stream>>>(a);
    return cudaGetLastError();
  });
}

bool fits(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// The rows are read in the widest vectors that their alignment allows: 16
// bytes, two elements, or one.  2 x 1 x 2048 x 4096 bf16 takes 23.5 us; 4098 in
// pairs 35, element by element 46; 4097 46.5.  Short rows gain nothing from pairs:
// 4 x 8 x 2000 x 82 takes 23 us either way (a warp to a row in both; 80: 10.8).
template <typename T>
cudaError_t launch_gated_t(const GatedNormArgs &a) {
  auto rows_fit = [&](int v) {  // the strides of axes of one element are never used
    const int bytes = v * sizeof(T);
    return a.d % v == 0 && (a.B == 1 || a.x_bs % v == 0) && (a.H == 1 || a.x_hs % v == 0) &&
           (a.L == 1 || a.x_ts % v == 0) && a.gate_stride % v == 0 && a.y_stride % v == 0 &&
           fits(a.x, bytes) && fits(a.gate, bytes) && fits(a.y, bytes);
  };
  auto act = [&](auto v) {
    constexpr int VEC = decltype(v)::value;
    if (a.act == LA_ACT_SILU) return launch_gated_v<T, VEC, LA_ACT_SILU>(a);
    if (a.act == LA_ACT_SIGMOID) return launch_gated_v<T, VEC, LA_ACT_SIGMOID>(a);
    return launch_gated_v<T, VEC, LA_ACT_NONE>(a);
  };
  constexpr int V = Pack16<T>::N;
  return rows_fit(V) ? act(Int<V>{}) : rows_fit(2) ? act(Int<2>{}) : act(Int<1>{});
}

// Rows on 16-byte boundaries, rows anywhere in tensors that start on one, or
// element by element (16384 x 4096 bf16: 86 us, and 200 where one tensor starts
// off a boundary).
template <typename T, typename R>
cudaError_t launch_residual_t(const ResidualNormArgs &a) {
  constexpr int V = Pack16<T>::N;
  const bool base = fits(a.x, 16) && fits(a.y, 16) && fits(a.residual, 16) &&
                    fits(a.residual_out, 16);
  if (base && a.D % V == 0) return launch_residual_v<T, R, V, false>(a);
  // Shifted, a row may take a vector more than a block of 1024 threads holds.
  return base && a.D + V - 1 <= 16384 ? launch_residual_v<T, R, V, true>(a)
                                      : launch_residual_v<T, R, 1, false>(a);
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
